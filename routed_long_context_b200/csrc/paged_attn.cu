// Attention over a paged 8-bit key/value cache.
//
//   out = softmax(scale q . K) V over the cached tokens that a query token sees: those at or before its own
//   place in the sequence, and of these the listed pages where a list is given.
// One block per (token, kv head); its four warps take every fourth key, each with its own running maximum and
// sum, and are joined at the end.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace msa {
namespace {

template <int G>
__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedAttnArgs a) {
    const PagedView& v = a.v;
    const int64_t t = blockIdx.x;
    const int g = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = seq_of_token(a.tok_off, v.n_seq, t);
    SeqSpan sp;
    if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, threadIdx.x == 0 ? a.err : nullptr) || t < sp.t0 ||
        t >= sp.t0 + sp.n_new)
        return;
    const int seen = sp.len - sp.n_new + (int)(t - sp.t0) + 1;
    const int n_vis = (seen + v.page - 1) >> v.shift;
    const int n_list = a.sel ? a.k : n_vis;
    float q[G][4], acc[G][4], m[G], l[G], lc[G];   // lc: what the sum's roundings lost
#pragma unroll
    for (int h = 0; h < G; ++h) {
        m[h] = -INFINITY;
        l[h] = lc[h] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[h][i] = __bfloat162float(a.q[((t * v.hkv + g) * G + h) * kPagedD + lane * 4 + i]) * a.scale_log2e;
            acc[h][i] = 0.f;
        }
    }
    for (int i = 0; i < n_list; ++i) {
        const int p = a.sel ? a.sel[(t * v.hkv + g) * a.k + i] : i;
        if (p < 0 || p >= n_vis) {
            if (p != -1 && threadIdx.x == 0) record_device_error(a.err, MSA_DEV_BAD_INDEX);
            continue;
        }
        const int32_t pid = v.table[(int64_t)s * v.max_pages + p];
        if (pid < 0 || pid >= v.n_pages) {
            if (threadIdx.x == 0) record_device_error(a.err, MSA_DEV_BAD_INDEX);
            continue;
        }
        const int64_t slab = (int64_t)pid * 2 * v.hkv + g;
        const float sk = v.scales[slab], sv = v.scales[slab + v.hkv];
        const uint8_t* pk = v.pages + slab * v.page * kPagedD;
        const uint8_t* pv = pk + (int64_t)v.hkv * v.page * kPagedD;
        const int rows = min(v.page, seen - (p << v.shift));
        for (int r = warp; r < rows; r += 4) {
            const uint32_t uk = *reinterpret_cast<const uint32_t*>(pk + r * kPagedD + lane * 4);
            const uint32_t uv = *reinterpret_cast<const uint32_t*>(pv + r * kPagedD + lane * 4);
            const float2 k0 = e4m3x2_f32(uk & 0xFFFFu), k1 = e4m3x2_f32(uk >> 16);
            const float2 v0 = e4m3x2_f32(uv & 0xFFFFu), v1 = e4m3x2_f32(uv >> 16);
#pragma unroll
            for (int h = 0; h < G; ++h) {
                float x = (q[h][0] * k0.x + q[h][1] * k0.y) + (q[h][2] * k1.x + q[h][3] * k1.y);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                x *= sk;
                const float mn = fmaxf(m[h], x);
                const float al = exp2f(m[h] - mn), w = exp2f(x - mn);
                m[h] = mn;
                const float add = w - lc[h] * al, sum = l[h] * al + add;
                lc[h] = (sum - l[h] * al) - add;
                l[h] = sum;
                const float wv = w * sv;
                acc[h][0] = acc[h][0] * al + wv * v0.x;
                acc[h][1] = acc[h][1] * al + wv * v0.y;
                acc[h][2] = acc[h][2] * al + wv * v1.x;
                acc[h][3] = acc[h][3] * al + wv * v1.y;
            }
        }
    }
    __shared__ float s_acc[4][G][kPagedD], s_m[4][G], s_l[4][G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s_acc[warp][h][lane * 4 + i] = acc[h][i];
        if (lane == 0) {
            s_m[warp][h] = m[h];
            s_l[warp][h] = l[h];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * kPagedD; i += 128) {
        const int h = i / kPagedD, d = i % kPagedD;
        float M = -INFINITY;
        for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w][h]);
        float o = 0.f, L = 0.f;
        for (int w = 0; w < 4; ++w)
            if (s_m[w][h] != -INFINITY) {
                const float f = exp2f(s_m[w][h] - M);
                o += f * s_acc[w][h][d];
                L += f * s_l[w][h];
            }
        const int64_t row = (t * v.hkv + g) * G + h;
        a.out[row * kPagedD + d] = __float2bfloat16_rn(L > 0.f ? o / L : 0.f);
        if (a.lse && d == 0) a.lse[row] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
}

// The combine pass, a programmatic dependent of the attention kernel: block (i, y) joins rows 2 y and 2 y + 1 of
// the segment that starts in CTA i and goes on in later ones, in the CTAs' order.
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedAttnArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const OpenSegment seg = a.open[blockIdx.x];
    const int n = 2 * blockIdx.y + (threadIdx.x >> 7), d = threadIdx.x & 127;
    if (seg.n_more == 0 || n >= seg.rows) return;
    const int64_t first = ((int64_t)blockIdx.x * 2 + 1) * a.rows + n;
    float M = -INFINITY;
    for (int i = 0; i <= seg.n_more; ++i) M = fmaxf(M, a.part_ml[first + (i ? 2 * i - 1 : 0) * a.rows].x);
    float L = 0.f, x = 0.f;
#pragma unroll 4
    for (int i = 0; i <= seg.n_more; ++i) {
        const int64_t row = first + (i ? 2 * i - 1 : 0) * a.rows;    // slot 1, then slot 0 of the next CTAs
        const float2 ml = a.part_ml[row];
        const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
        L += ml.x == -INFINITY ? ml.y : w * ml.y;
        x += w * a.part_o[row * kPagedD + d];
    }
    const int64_t row = (seg.t0 + n / a.G) * (a.v.hkv * a.G) + seg.head * a.G + n % a.G;
    a.out[row * kPagedD + d] = __float2bfloat16_rn(L == 0.f ? 0.f : x * (seg.unit / L));
    if (a.lse && d == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

constexpr int kGrid = 296;        // CTAs of the few-rows kernel: two per SM

struct AttnPlan {
    bool few;                     // the few-rows kernel
    int grid, rows;
    size_t o, ml, open, bytes;    // offsets in the workspace
};
AttnPlan attn_plan(int64_t n_tok, int n_seq, int max_new, int hq, int hkv, int max_pages, int page, int k) {
    AttnPlan p{};
    const int G = hq / hkv;
    p.few = k > 0 || (int64_t)max_new * G <= kDecodeRows;
    p.rows = kDecodeRows;
    const int64_t pages = k > 0 ? n_tok * k : (int64_t)std::min<int64_t>(n_tok, n_seq) * max_pages;
    const int64_t tiles = pages * hkv * (page / kDecodeTile);
    p.grid = (int)std::max<int64_t>(1, std::min<int64_t>(kGrid, (tiles + 7) / 8));
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += align_up(n, 256);
        return was;
    };
    p.o = take((size_t)p.grid * 2 * p.rows * kPagedD * sizeof(float));
    p.ml = take((size_t)p.grid * 2 * p.rows * sizeof(float2));
    p.open = take((size_t)p.grid * sizeof(OpenSegment));
    p.bytes = at;
    return p;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_paged_attn_workspace_size(int64_t n_tok, int n_seq, int max_new, int hq, int hkv,
                                                    int max_pages, int page, int k, size_t* bytes) {
    MSA_REQUIRE(bytes != nullptr, "msa_paged_attn_workspace_size: bytes is NULL");
    MSA_REQUIRE(n_tok >= 0 && n_seq > 0 && max_new >= 0 && hkv > 0 && hq > 0 && hq % hkv == 0 && max_pages > 0 &&
                    page >= 16 && k >= 0,
                "msa_paged_attn_workspace_size: bad sizes");
    *bytes = attn_plan(n_tok, n_seq, max_new, hq, hkv, max_pages, page, k).bytes;
    return MSA_OK;
}

extern "C" msa_status msa_paged_attn(const msa_paged_kv* kv, const void* q, msa_dtype dt, int64_t n_tok, int hq,
                                     const int64_t* tok_off, int max_new, const int32_t* sel, int k, float scale,
                                     void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    PagedAttnArgs a{};
    MSA_RETURN_IF(paged_view(kv, "msa_paged_attn", &a.v));
    MSA_REQUIRE(dtype_ok(dt), "msa_paged_attn: bad dtype");
    if (dt != MSA_BF16) return set_error(MSA_ERR_UNSUPPORTED, "msa_paged_attn: bf16 queries only");
    MSA_RETURN_IF(paged_tokens_ok(kv, "msa_paged_attn", n_tok, tok_off, max_new));
    MSA_REQUIRE(hq > 0 && hq % kv->hkv == 0, "msa_paged_attn: hq must be a multiple of hkv");
    a.G = hq / kv->hkv;
    if (a.G != 1 && a.G != 2 && a.G != 4 && a.G != 8)
        return set_error(MSA_ERR_UNSUPPORTED, "msa_paged_attn: hq/hkv = %d unsupported", a.G);
    MSA_REQUIRE(sel == nullptr || k >= 1, "msa_paged_attn: k must be at least 1 with a page list");
    MSA_REQUIRE(sel == nullptr || (int64_t)k * kv->page <= (int64_t)INT32_MAX, "msa_paged_attn: k * page too large");
    if (n_tok == 0 || max_new == 0) return MSA_OK;
    MSA_REQUIRE(q && out && ws, "msa_paged_attn: NULL pointer");
    MSA_REQUIRE(aligned16(q) && aligned16(out) && aligned16(lse) && aligned16(sel) && aligned16(ws),
                "msa_paged_attn: pointers must be 16-byte aligned");
    size_t need = 0;
    MSA_RETURN_IF(msa_paged_attn_workspace_size(n_tok, kv->n_seq, max_new, hq, kv->hkv, kv->max_pages, kv->page,
                                                sel ? k : 0, &need));
    if (ws_bytes < need) return set_error(MSA_ERR_WORKSPACE, "msa_paged_attn: workspace %zu < %zu", ws_bytes, need);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.n_tok = n_tok; a.tok_off = tok_off; a.max_new = max_new; a.sel = sel; a.k = k;
    a.scale_log2e = scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.err = device_error_word();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const AttnPlan p = attn_plan(n_tok, kv->n_seq, max_new, hq, kv->hkv, kv->max_pages, kv->page, sel ? k : 0);
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.rows = p.rows;
    a.part_o = reinterpret_cast<float*>(w + p.o);
    a.part_ml = reinterpret_cast<float2*>(w + p.ml);
    a.open = reinterpret_cast<OpenSegment*>(w + p.open);
    if (p.few) {
        MSA_RETURN_IF(launch_paged_decode(a, p.grid, s));
        if (p.grid == 1) return MSA_OK;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)p.grid, (unsigned)(std::min<int64_t>(p.rows, sel ? a.G : (int64_t)max_new * a.G) + 1) / 2);
        cfg.blockDim = dim3(256);
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        MSA_CUDA_TRY(cudaLaunchKernelEx(&cfg, paged_combine_kernel, a));
        return MSA_OK;
    }
    const dim3 grid((unsigned)n_tok, (unsigned)kv->hkv);
    switch (a.G) {
        case 1: paged_attn_kernel<1><<<grid, 128, 0, s>>>(a); break;
        case 2: paged_attn_kernel<2><<<grid, 128, 0, s>>>(a); break;
        case 4: paged_attn_kernel<4><<<grid, 128, 0, s>>>(a); break;
        default: paged_attn_kernel<8><<<grid, 128, 0, s>>>(a); break;
    }
    MSA_LAUNCH_CHECK();
    return MSA_OK;
}
