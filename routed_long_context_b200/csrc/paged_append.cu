// Appending to the paged 8-bit key/value cache: rotation, scales, rounding and key bounds in one launch.
//
// For every page that takes new tokens, and each of K (rotated to its position) and V of each kv head:
//   scale   = max(scale of the older rows, 2^ceil(log2(max|new rows| / 448)))     (a fresh page: the latter)
//   row     = rn_e4m3(row / scale);  older rows of a page whose scale grows: rn_e4m3(row * old / scale)
//   bounds  = elementwise min and max of the page's stored keys
// The scale is a power of two, so dividing by it is exact, an older row changes only where it falls below
// the smallest normal e4m3 value, and every stored value times its scale is a bf16 number. Rounding is
// monotone: the bounds of the stored keys are the rounded bounds of the keys, and those of the older rows
// the older bounds rounded to the new scale, so no older row is read for them.
//
// One block per (page that takes tokens, kv head): all of the page's new rows of K and V in registers
// (eight threads a row, 2 x 8 values of K and of V each, the two halves of a rotate-half pair in one
// thread), one block-wide max, one write; with queries, one more block per (page, kv head) rotates the
// group's query heads of the same tokens. Bound by memory: each input read once, each output written once.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace msa {

msa_status paged_view(const msa_paged_kv* kv, const char* who, PagedView* out) {
    MSA_REQUIRE(kv != nullptr, "%s: NULL cache", who);
    MSA_REQUIRE(kv->pages && kv->scales && kv->page_table && kv->seq_len, "%s: NULL pointer in the cache", who);
    MSA_REQUIRE(aligned16(kv->pages) && aligned16(kv->scales) && aligned16(kv->bounds) && aligned16(kv->page_table) &&
                    aligned16(kv->seq_len),
                "%s: cache pointers must be 16-byte aligned", who);
    MSA_REQUIRE(kv->n_pages > 0 && kv->n_seq > 0 && kv->max_pages > 0 && kv->hkv > 0 && kv->hkv <= 4096,
                "%s: bad cache sizes", who);
    if (kv->d != kPagedD) return set_error(MSA_ERR_UNSUPPORTED, "%s: head_dim must be 128, got %d", who, kv->d);
    if (kv->page != 16 && kv->page != 32 && kv->page != 64 && kv->page != 128)
        return set_error(MSA_ERR_UNSUPPORTED, "%s: page must be 16, 32, 64 or 128 tokens, got %d", who, kv->page);
    MSA_REQUIRE((int64_t)kv->max_pages * kv->page <= (int64_t)INT32_MAX - 255, "%s: max_pages * page too large", who);
    // rows of 128 bytes are addressed by 32-bit coordinates
    MSA_REQUIRE(kv->n_pages <= (int64_t)INT32_MAX / (2LL * kv->hkv * kv->page), "%s: n_pages too large", who);
    out->pages = static_cast<uint8_t*>(kv->pages);
    out->scales = kv->scales;
    out->bounds = static_cast<__nv_bfloat16*>(kv->bounds);
    out->table = kv->page_table;
    out->len = kv->seq_len;
    out->n_pages = kv->n_pages;
    out->n_seq = kv->n_seq;
    out->max_pages = kv->max_pages;
    out->page = kv->page;
    out->shift = kv->page == 16 ? 4 : kv->page == 32 ? 5 : kv->page == 64 ? 6 : 7;
    out->hkv = kv->hkv;
    return MSA_OK;
}

msa_status paged_tokens_ok(const msa_paged_kv* kv, const char* who, int64_t n_tok, const int64_t* tok_off, int max_new) {
    MSA_REQUIRE(tok_off != nullptr, "%s: NULL tok_off", who);
    MSA_REQUIRE(n_tok >= 0 && n_tok < (int64_t)INT32_MAX / 2 && max_new >= 0, "%s: bad token counts", who);
    return MSA_OK;
}

namespace {

struct AppendPagedArgs {
    PagedView v;
    const void* k;
    const void* v_in;
    const void* q;
    void* q_rot;
    int64_t n_tok;
    const int64_t* tok_off;
    int max_new, G;
    int per_seq;             // > 0: blocks per_seq * s .. are sequence s's pages; 0: by offsets (page_of_item)
    int64_t pos_offset;
    const float2* cs;
    int64_t max_pos;
    int* err;
};

// Item i of the packed layout belongs to the last sequence s with tok_off[s] / page + 2 s <= i: a sequence
// of n tokens touches at most floor(n / page) + 2 pages, which is at most how far that number grows from s
// to s + 1. A warp looks at 32 sequences at a time.
__device__ __forceinline__ int seq_of_item(const AppendPagedArgs& a, int64_t item, int64_t* first) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = a.v.n_seq;                       // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int s = lo + lane * step;
        const bool in = lane * step < n && ((a.tok_off[s] >> a.v.shift) + 2LL * s) <= item;
        const int hit = 31 - __clz(__ballot_sync(0xffffffffu, in) | 1u);
        n = min(step, n - hit * step);
        lo += hit * step;
    }
    *first = (a.tok_off[lo] >> a.v.shift) + 2LL * lo;
    return lo;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* out) {
    load16_f32(p, out);
    if constexpr (sizeof(T) == 4) load16_f32(p + 4, out + 4);
}

// 16 elements of a row: 8 at 8 c and their rotate-half partners at 64 + 8 c
template <typename T>
__device__ __forceinline__ void load_pair(const T* row, int c, float* x) {
    load8(row + 8 * c, x);
    load8(row + 64 + 8 * c, x + 8);
}

__device__ __forceinline__ void rotate_pair(float* x, const float2* cs, int c) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float4 w = *reinterpret_cast<const float4*>(cs + 8 * c + i);
        const float a0 = x[i], b0 = x[8 + i], a1 = x[i + 1], b1 = x[9 + i];
        x[i] = fmaf(a0, w.x, -(b0 * w.y));
        x[8 + i] = fmaf(b0, w.x, a0 * w.y);
        x[i + 1] = fmaf(a1, w.z, -(b1 * w.w));
        x[9 + i] = fmaf(b1, w.z, a1 * w.w);
    }
}

// Largest magnitude of 16 values; a NaN becomes 0 and an infinity keeps out of the scale (it saturates).
__device__ __forceinline__ float clean_amax(float* x, bool* bad) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float y = fabsf(x[i]);
        if (!(y <= 3.402823466e38f)) {
            *bad = true;
            if (y != y) x[i] = 0.f;
        } else {
            m = fmaxf(m, y);
        }
    }
    return m;
}

__device__ __forceinline__ void store_e4m3(uint8_t* row, int c, const float* x, float inv) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint2 u;
        const float* y = x + 8 * h;
        u.x = e4m3x2(y[0] * inv, y[1] * inv) | (e4m3x2(y[2] * inv, y[3] * inv) << 16);
        u.y = e4m3x2(y[4] * inv, y[5] * inv) | (e4m3x2(y[6] * inv, y[7] * inv) << 16);
        *reinterpret_cast<uint2*>(row + 64 * h + 8 * c) = u;
    }
}

__device__ __forceinline__ float round_to(float x, float scale, float inv) {
    return e4m3x2_f32(e4m3x2(x * inv, 0.f)).x * scale;
}

template <typename T, int PAGE>
__global__ void __launch_bounds__(4 * PAGE) paged_append_kernel(const AppendPagedArgs a) {
    constexpr int kThreads = 4 * PAGE, kPass = PAGE / 2, kWarps = kThreads / 32;
    const PagedView& v = a.v;
    const int tid = threadIdx.x, c = tid & 7;
    int s;
    int64_t j;
    if (a.per_seq > 0) {
        s = blockIdx.x / a.per_seq;
        j = blockIdx.x - s * a.per_seq;
    } else {
        int64_t first;
        s = seq_of_item(a, blockIdx.x, &first);
        j = (int64_t)blockIdx.x - first;
    }
    SeqSpan sp;
    if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, tid == 0 ? a.err : nullptr)) return;
    const int base = sp.len - sp.n_new;
    const int64_t p64 = (base >> v.shift) + j;
    if (j < 0 || p64 * PAGE >= sp.len || sp.n_new == 0) return;
    const int p = (int)p64;
    const int r0 = max(base - p * PAGE, 0), r1 = min(sp.len - p * PAGE, PAGE);
    const int64_t tok0 = sp.t0 + (p * PAGE + r0 - base);          // packed row of page row r0
    const int64_t pos0 = a.pos_offset + (int64_t)p * PAGE;        // position of page row 0

    if ((int)blockIdx.y >= v.hkv) {
        // the query heads of one group: rows (token, head), 8 threads each
        const int g = blockIdx.y - v.hkv, hq = v.hkv * a.G;
        const int rows = (r1 - r0) * a.G;
        for (int i = tid >> 3; i < rows; i += kThreads / 8) {
            const int r = i / a.G, h = g * a.G + i - r * a.G;
            const int64_t off = ((tok0 + r) * hq + h) * kPagedD;
            float x[16];
            load_pair(static_cast<const T*>(a.q) + off, c, x);
            const int64_t pos = pos0 + r0 + r;
            if (pos < a.max_pos) rotate_pair(x, a.cs + pos * (kPagedD / 2), c);
            else record_device_error(a.err, MSA_DEV_ROPE_POSITION);
            T* out = static_cast<T*>(a.q_rot) + off;
            store_f32<T, 8>(out + 8 * c, x);
            store_f32<T, 8>(out + 64 + 8 * c, x + 8);
        }
        return;
    }

    const int g = blockIdx.y;
    const int32_t pid = v.table[(int64_t)s * v.max_pages + p];
    float xk[2][16], xv[2][16];
    float mk = 0.f, mv = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * kPass + (tid >> 3);
        if (r < r1) {
            const int64_t off = ((tok0 + r - r0) * v.hkv + g) * kPagedD;
            load_pair(static_cast<const T*>(a.k) + off, c, xk[i]);
            load_pair(static_cast<const T*>(a.v_in) + off, c, xv[i]);
        }
    }
    if (pid < 0 || pid >= v.n_pages) {
        if (tid == 0) record_device_error(a.err, MSA_DEV_BAD_INDEX);
        return;
    }
    const int64_t slab = ((int64_t)pid * 2 * v.hkv + g);          // (page, K, head); V is hkv further
    const float old_k = r0 > 0 ? v.scales[slab] : 0.f, old_v = r0 > 0 ? v.scales[slab + v.hkv] : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * kPass + (tid >> 3);
        if (r < r1) {
            const int64_t pos = pos0 + r;
            if (pos < a.max_pos) rotate_pair(xk[i], a.cs + pos * (kPagedD / 2), c);
            else record_device_error(a.err, MSA_DEV_ROPE_POSITION);
            mk = fmaxf(mk, clean_amax(xk[i], &bad));
            mv = fmaxf(mv, clean_amax(xv[i], &bad));
        }
    }
    if (bad) record_device_error(a.err, MSA_DEV_NONFINITE);

    __shared__ float s_max[2][kWarps];
    __shared__ float s_lo[kWarps][kPagedD], s_hi[kWarps][kPagedD];
    const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if (lane == 0) {
        s_max[0][warp] = mk;
        s_max[1][warp] = mv;
    }
    if (v.bounds) {
        // this thread's columns over its rows, then over the four row groups of the warp
        float lo[16], hi[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            lo[e] = __int_as_float(0x7f800000);
            hi[e] = -lo[e];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (r0 + i * kPass + (tid >> 3) < r1) {
                    lo[e] = fminf(lo[e], xk[i][e]);
                    hi[e] = fmaxf(hi[e], xk[i][e]);
                }
#pragma unroll
            for (int o = 8; o <= 16; o <<= 1) {
                lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
                hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
            }
        }
        if (lane < 8) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int d = (e >> 3) * 64 + 8 * c + (e & 7);
                s_lo[warp][d] = lo[e];
                s_hi[warp][d] = hi[e];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        mk = fmaxf(mk, s_max[0][w]);
        mv = fmaxf(mv, s_max[1][w]);
    }
    int ek = scale_exponent(mk), ev = scale_exponent(mv);
    if (r0 > 0) {
        ek = max(ek, exponent_of(old_k));
        ev = max(ev, exponent_of(old_v));
    }
    const float sk = pow2f(ek), ik = pow2f(-ek), sv = pow2f(ev), iv = pow2f(-ev);
    uint8_t* pk = v.pages + slab * PAGE * kPagedD;
    uint8_t* pv = pk + (int64_t)v.hkv * PAGE * kPagedD;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * kPass + (tid >> 3);
        if (r < r1) {
            store_e4m3(pk + r * kPagedD, c, xk[i], ik);
            store_e4m3(pv + r * kPagedD, c, xv[i], iv);
        }
    }
    if (tid == 0) {
        v.scales[slab] = sk;
        v.scales[slab + v.hkv] = sv;
    }
    // older rows of a scale that grows: rounded again, 16 values a thread
    if (r0 > 0) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const float was = part ? old_v : old_k, now = part ? sv : sk;
            if (now == was) continue;
            const float ratio = was * (part ? iv : ik);
            uint4* rows = reinterpret_cast<uint4*>(part ? pv : pk);
            for (int i = tid; i < r0 * (kPagedD / 16); i += kThreads) {
                uint4 u = rows[i];
                uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 lo = e4m3x2_f32(w[e] & 0xFFFFu), hi = e4m3x2_f32(w[e] >> 16);
                    w[e] = e4m3x2(lo.x * ratio, lo.y * ratio) | (e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
                }
                rows[i] = u;
            }
        }
    }
    if (v.bounds) {
        for (int d = tid; d < kPagedD; d += kThreads) {
            float lo = s_lo[0][d], hi = s_hi[0][d];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                lo = fminf(lo, s_lo[w][d]);
                hi = fmaxf(hi, s_hi[w][d]);
            }
            __nv_bfloat16* b = v.bounds + ((int64_t)pid * v.hkv + g) * 2 * kPagedD + d;
            if (r0 > 0) {
                lo = fminf(lo, __bfloat162float(b[0]));
                hi = fmaxf(hi, __bfloat162float(b[kPagedD]));
            }
            b[0] = __float2bfloat16_rn(round_to(lo, sk, ik));
            b[kPagedD] = __float2bfloat16_rn(round_to(hi, sk, ik));
        }
    }
}

template <typename T>
void launch_paged_append(const AppendPagedArgs& a, dim3 grid, cudaStream_t s) {
    switch (a.v.page) {
        case 16: paged_append_kernel<T, 16><<<grid, 64, 0, s>>>(a); break;
        case 32: paged_append_kernel<T, 32><<<grid, 128, 0, s>>>(a); break;
        case 64: paged_append_kernel<T, 64><<<grid, 256, 0, s>>>(a); break;
        default: paged_append_kernel<T, 128><<<grid, 512, 0, s>>>(a); break;
    }
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_paged_append(const msa_paged_kv* kv, const void* k, const void* v, const void* q, msa_dtype dt,
                                       int64_t n_tok, int hq, const int64_t* tok_off, int max_new, int64_t pos_offset,
                                       const float* cos_sin, int64_t max_pos, void* q_rot, void* stream) {
    AppendPagedArgs a{};
    MSA_RETURN_IF(paged_view(kv, "msa_paged_append", &a.v));
    MSA_REQUIRE(dtype_ok(dt), "msa_paged_append: bad dtype");
    MSA_RETURN_IF(paged_tokens_ok(kv, "msa_paged_append", n_tok, tok_off, max_new));
    MSA_REQUIRE(max_pos > 0 && pos_offset >= 0 && pos_offset <= (int64_t)1 << 40, "msa_paged_append: bad positions");
    MSA_REQUIRE(q == nullptr || (q_rot != nullptr && hq > 0 && hq % kv->hkv == 0),
                "msa_paged_append: q needs q_rot and hq a multiple of hkv");
    MSA_REQUIRE(n_tok == 0 || (k && v && cos_sin), "msa_paged_append: NULL pointer");
    MSA_REQUIRE(aligned16(k) && aligned16(v) && aligned16(q) && aligned16(q_rot) && aligned16(cos_sin),
                "msa_paged_append: pointers must be 16-byte aligned");
    if (n_tok == 0 || max_new == 0) return MSA_OK;
    a.k = k; a.v_in = v; a.q = q; a.q_rot = q_rot;
    a.n_tok = n_tok; a.tok_off = tok_off; a.max_new = (int)std::min<int64_t>(max_new, n_tok);
    a.G = q ? hq / kv->hkv : 1;
    a.pos_offset = pos_offset;
    a.cs = reinterpret_cast<const float2*>(cos_sin);
    a.max_pos = max_pos;
    a.err = device_error_word();
    // blocks: max_new tokens touch at most (max_new + page - 2) / page + 1 pages of a sequence, all
    // sequences together at most n_tok / page + 2 n_seq; whichever is fewer
    const int page = kv->page;
    const int64_t per_seq = ((int64_t)a.max_new + page - 2) / page + 1;
    const int64_t packed = n_tok / page + 2LL * kv->n_seq;
    int64_t items = per_seq * kv->n_seq;
    a.per_seq = (int)per_seq;
    if (packed < items) {
        items = packed;
        a.per_seq = 0;
    }
    const dim3 grid((unsigned)items, (unsigned)(q ? 2 * kv->hkv : kv->hkv), 1);
    if (dt == MSA_BF16) launch_paged_append<__nv_bfloat16>(a, grid, static_cast<cudaStream_t>(stream));
    else launch_paged_append<float>(a, grid, static_cast<cudaStream_t>(stream));
    MSA_LAUNCH_CHECK();
    return MSA_OK;
}
