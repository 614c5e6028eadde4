// Attention over a paged 8-bit key/value cache.
//
//   out = softmax(scale q . K) V over the cached tokens that a query token sees: those at or before its own
//   place in the sequence, and of these the listed pages where a list is given.
// Up to 8 rows (token, query head) of a kv head and sequence, page lists and small calls go to the few-rows kernel, which
// the bytes bound; more rows to the tcgen05 kernel, which the products bound. Both cut the keys of all sequences
// evenly over the SMs; the softmaxes that end up in several pieces are joined here.
#include <algorithm>
#include <atomic>

#include "kernels.cuh"
#include "mma.cuh"
#include "paged.cuh"

namespace msa {
namespace {

// The combine pass: warp w of block (i, y) joins row 8 y + w of the
// segment that starts in CTA i and goes on in later ones, in the CTAs' order, four columns a lane. Up to 32 pieces'
// maxima and sums come at once, a lane each, and the pieces' rows four at a time: a handful of latencies in all.
constexpr int kCombineRows = 8;
__global__ void __launch_bounds__(32 * kCombineRows) paged_combine_kernel(const PagedAttnArgs a) {
    next_may_launch();
    wait_for_earlier();
    const OpenSegment seg = a.open[blockIdx.x];
    const int n = blockIdx.y * kCombineRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (seg.n_more == 0 || n >= seg.rows) return;
    // piece 0 is in slot 1 of CTA i, piece j in slot 0 of CTA i + j
    const int64_t first = (int64_t)blockIdx.x * 2 * a.rows + n;
    auto row_of = [&](int j) -> int64_t { return first + (int64_t)(j ? 2 * j : 1) * a.rows; };
    const int pieces = seg.n_more + 1;
    float M = -INFINITY;
    for (int j = lane; j < pieces; j += 32) M = fmaxf(M, a.part_ml[row_of(j)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < pieces; j0 += 32) {
        const float2 ml = j0 + lane < pieces ? a.part_ml[row_of(j0 + lane)] : make_float2(-INFINITY, 0.f);
        const bool none = ml.x == -INFINITY;               // a sum without a maximum is 0 or NaN
        const float w = none ? 0.f : exp2f(ml.x - M), part = none ? ml.y : w * ml.y;
        const int m = min(32, pieces - j0);
#pragma unroll 4
        for (int j = 0; j < m; ++j) {
            const float4 y = reinterpret_cast<const float4*>(a.part_o + row_of(j0 + j) * kPagedD)[lane];
            const float wj = __shfl_sync(0xffffffffu, w, j);
            L += __shfl_sync(0xffffffffu, part, j);
            if (wj != 0.f) {                               // a piece without a key may hold anything
                x.x = fmaf(wj, y.x, x.x);
                x.y = fmaf(wj, y.y, x.y);
                x.z = fmaf(wj, y.z, x.z);
                x.w = fmaf(wj, y.w, x.w);
            }
        }
    }
    const int64_t row = (seg.t0 + n / a.G) * (a.v.hkv * a.G) + seg.head * a.G + n % a.G;
    const float inv = L == 0.f ? 0.f : seg.unit / L;       // NaN where a query row holds one
    uint2 u;
    u.x = pack_bf16(x.x * inv, x.y * inv);
    u.y = pack_bf16(x.z * inv, x.w * inv);
    reinterpret_cast<uint2*>(a.out + row * kPagedD)[lane] = u;
    if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

std::atomic<int> g_inject_stall{0};   // testing knob: make the next launches' waits time out
constexpr int kSms = 148;

struct AttnPlan {
    bool few;                     // the few-rows kernel
    bool uncut;                   // no segment will be cut: there is nothing to combine
    int grid, rows;
    size_t o, ml, open, bytes;    // offsets in the workspace
};
AttnPlan attn_plan(int64_t n_tok, int n_seq, int max_new, int hq, int hkv, int max_pages, int page, int k) {
    AttnPlan p{};
    const int G = hq / hkv;
    const int64_t seqs = std::min<int64_t>(n_tok, n_seq), keys = (int64_t)max_pages * page;
    // upper bounds of the segments that there can be, and of a segment's tiles
    const int64_t blocks = std::min<int64_t>(((int64_t)max_new * G + kDecodeRows - 1) / kDecodeRows * seqs,
                                             n_tok * G / kDecodeRows + seqs);
    int64_t segments = (k > 0 ? n_tok : blocks) * hkv;
    int64_t tiles = k > 0 ? (page == 16 ? ((int64_t)k + 1) / 2 : (int64_t)k * (page / kDecodeTile))
                          : (keys + kDecodeTile - 1) / kDecodeTile;
    p.few = k > 0 || (int64_t)max_new * G <= kDecodeRows;
    p.rows = kDecodeRows;
    if (!p.few) {
        // More rows take the many-rows kernel, or, where there is little to do, blocks of 8 in the few-rows kernel, which
        // starts and ends sooner. Measured, with u the units (tiles and kSegWeight a segment) that a block gets and m the
        // tiles of a segment, of which a block of the many-rows kernel takes 9 at least where there are so many:
        // 7.5 + 0.3 u against 14.7 + 1.2 m us for 128 rows and 2.4 m for 256. One sequence of 64 tokens over 2,000 of 2
        // kv heads 18.8 us (many rows 34.3), 22 of 8 heads over 242 15.1 (21.8), 4 of 9 over 33 7.4 (13.1); on the
        // border 100 over 100 17.6 (17.5); beyond it 7 of up to 41 over up to 85 22.3 (20.0).
        const int rows = (int64_t)max_new * G <= 128 ? 128 : 256;
        const int64_t many = (keys + kPromptTile - 1) / kPromptTile;
        p.few = segments * (tiles + kSegWeight) <= kSms * (24 + 4 * std::min<int64_t>(many, 9) * (rows / 128));
        if (!p.few) {
            p.rows = rows;
            segments = ((int64_t)max_new * G + rows - 1) / rows * seqs * hkv;
            tiles = many;
        }
    }
    p.grid = (int)std::max<int64_t>(1, std::min<int64_t>(kSms, segments * tiles));
    // (the kernel decides by the lengths themselves; this is what it will find whatever those are)
    p.uncut = p.few && segments <= p.grid && tiles <= kDecodeUncut && (k > 0 || n_seq <= kDecodeSeqs);
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

extern "C" msa_status msa_paged_inject_stall(int on) {
    MSA_REQUIRE(on >= 0 && on <= 1000, "msa_paged_inject_stall: on must be between 0 and 1000");
    g_inject_stall.store(on);
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
    a.stall = g_inject_stall.load();
    a.err = device_error_word();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const AttnPlan p = attn_plan(n_tok, kv->n_seq, max_new, hq, kv->hkv, kv->max_pages, kv->page, sel ? k : 0);
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.rows = p.rows;
    a.part_o = reinterpret_cast<float*>(w + p.o);
    a.part_ml = reinterpret_cast<float2*>(w + p.ml);
    a.open = reinterpret_cast<OpenSegment*>(w + p.open);
    const int64_t rows = std::min<int64_t>(p.rows, sel ? a.G : (int64_t)max_new * a.G);
    const int step = p.few ? kv->n_seq : kPromptSeqs;
    for (int first = 0; first < kv->n_seq; first += step) {
        PagedAttnArgs b = a;
        b.v.n_seq = std::min(step, kv->n_seq - first);
        b.v.table += (int64_t)first * kv->max_pages;
        b.v.len += first;
        b.tok_off += first;
        if (p.few) MSA_RETURN_IF(launch_paged_decode(b, p.grid, s));
        else MSA_RETURN_IF(launch_paged_prompt(b, p.grid, s));
        if (p.grid == 1 || p.uncut) continue;
        const dim3 grid((unsigned)p.grid, (unsigned)((rows + kCombineRows - 1) / kCombineRows));
        MSA_CUDA_TRY(launch_early(paged_combine_kernel, grid, 32 * kCombineRows, 0, s, b));
    }
    return MSA_OK;
}
