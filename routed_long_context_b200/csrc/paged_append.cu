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
// One block per page that takes tokens and K or V of a kv head, K's with the query heads of its group, which turn
// by the same angles: all of the page's new rows in registers (eight threads a row, 2 x 8 values each, the two
// halves of a rotate-half pair in one thread), one block-wide maximum, one write; the bounds are taken from the
// rounded values, two to a register. A page's blocks are neighbours in the grid, as their data is in memory.
// Bound by memory: each input is read once, each output written once. 65,536 bf16 tokens of 8 kv and 32 query
// heads in pages of 64: 279 us, 5.4 TB/s; with queries in blocks of their own 419 us, at 64 registers (which
// spill) instead of 80 332 us.
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
    int max_new, G, parts;
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

// A thread's 16 elements of a row, 8 at 8 c and their rotate-half partners at 64 + 8 c: as they are in memory,
// so that several rows may be on their way at few registers, and in fp32.
template <typename T> struct Raw {
    static constexpr int N = sizeof(T) / 2;                    // 16-byte pieces per 8 elements: 1 or 2
    uint4 u[2 * N];
    __device__ __forceinline__ void load(const T* row, int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < N; ++i) u[h * N + i] = reinterpret_cast<const uint4*>(row + 64 * h + 8 * c)[i];
    }
    __device__ __forceinline__ void f32(float* x) const {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (N == 2) {
                    x[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                    x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        }
    }
};

__device__ __forceinline__ void load_angles(float4* w, const float2* cs, int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(cs + 8 * c + 2 * i);
}
__device__ __forceinline__ void rotate_pair(float* x, const float4* w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a0 = x[2 * i], b0 = x[8 + 2 * i], a1 = x[2 * i + 1], b1 = x[9 + 2 * i];
        x[2 * i] = fmaf(a0, w[i].x, -(b0 * w[i].y));
        x[8 + 2 * i] = fmaf(b0, w[i].x, a0 * w[i].y);
        x[2 * i + 1] = fmaf(a1, w[i].z, -(b1 * w[i].w));
        x[9 + 2 * i] = fmaf(b1, w[i].z, a1 * w[i].w);
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

__device__ __forceinline__ float round_to(float x, float scale, float inv) {
    return e4m3x2_f32(e4m3x2(x * inv, 0.f)).x * scale;
}
__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

template <typename T, int PAGE>
__global__ void __launch_bounds__(4 * PAGE, PAGE == 128 ? 1 : 768 / (4 * PAGE)) paged_append_kernel(const AppendPagedArgs a) {
    constexpr int kThreads = 4 * PAGE, kPass = PAGE / 2, kWarps = kThreads / 32;
    const PagedView& v = a.v;
    const int tid = threadIdx.x, c = tid & 7;
    int s;
    int64_t j;
    // the parts of a page's tokens (K, V and groups of query heads) are neighbours, as they are in memory
    const int item = blockIdx.x / a.parts, part = blockIdx.x - item * a.parts;
    if (a.per_seq > 0) {
        s = item / a.per_seq;
        j = item - s * a.per_seq;
    } else {
        int64_t first;
        s = seq_of_item(a, item, &first);
        j = item - first;
        // where offsets decrease the search may find no item of some sequence: each is looked at by a block of its own
        SeqSpan each;
        if (part == 0 && item < v.n_seq && tid == 32) seq_span(v, a.tok_off, a.n_tok, a.max_new, item, &each, a.err);
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

    if (part < v.hkv && a.q) {
        // the query heads of one group: eight threads a row, its angles loaded once for all heads
        constexpr int kHeads = 4 / (sizeof(T) / 2);               // in flight
        const int g = part, hq = v.hkv * a.G;
        for (int r = r0 + (tid >> 3); r < r1; r += kPass) {
            const int64_t pos = pos0 + r, off = ((tok0 + r - r0) * hq + g * a.G) * kPagedD;
            const T* src = static_cast<const T*>(a.q) + off;
            T* dst = static_cast<T*>(a.q_rot) + off;
            const bool turn = pos < a.max_pos;
            if (!turn) record_device_error(a.err, MSA_DEV_ROPE_POSITION);
            float4 w[4];
            if (turn) load_angles(w, a.cs + pos * (kPagedD / 2), c);
            for (int h0 = 0; h0 < a.G; h0 += kHeads) {
                Raw<T> raw[kHeads];
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    if (h0 + h < a.G) raw[h].load(src + (h0 + h) * kPagedD, c);
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    if (h0 + h < a.G) {
                        float x[16];
                        raw[h].f32(x);
                        if (turn) rotate_pair(x, w);
                        T* out = dst + (h0 + h) * kPagedD + 8 * c;
                        store_f32<T, 8>(out, x);
                        store_f32<T, 8>(out + 64, x + 8);
                    }
            }
        }
    }

    const bool keys = part < v.hkv;
    const int g = keys ? part : part - v.hkv;
    const int32_t pid = v.table[(int64_t)s * v.max_pages + p];
    Raw<T> raw[2];
    {
        const T* src = static_cast<const T*>(keys ? a.k : a.v_in) + (tok0 * v.hkv + g) * kPagedD;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r0 + i * kPass + (tid >> 3);
            if (r < r1) raw[i].load(src + (int64_t)(r - r0) * v.hkv * kPagedD, c);
        }
    }
    if (pid < 0 || pid >= v.n_pages) {
        if (tid == 0) record_device_error(a.err, MSA_DEV_BAD_INDEX);
        return;
    }
    const int64_t slab = (int64_t)pid * 2 * v.hkv + part;         // (page, K or V, head)
    const float was = r0 > 0 ? v.scales[slab] : 0.f;
    float x[2][16], top = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * kPass + (tid >> 3);
        if (r >= r1) continue;
        raw[i].f32(x[i]);
        if (keys) {
            const int64_t pos = pos0 + r;
            if (pos < a.max_pos) {
                float4 w[4];
                load_angles(w, a.cs + pos * (kPagedD / 2), c);
                rotate_pair(x[i], w);
            } else {
                record_device_error(a.err, MSA_DEV_ROPE_POSITION);
            }
        }
        top = fmaxf(top, clean_amax(x[i], &bad));
    }
    if (bad) record_device_error(a.err, MSA_DEV_NONFINITE);

    __shared__ float s_max[kWarps];
    __shared__ uint32_t s_lo[kWarps][kPagedD / 2], s_hi[kWarps][kPagedD / 2];   // fp16 pairs
    const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_max[w]);
    int e = scale_exponent(top);
    if (r0 > 0) e = max(e, min(max(exponent_of(was), kScaleMin), kScaleMax));
    const float scale = pow2f(e), inv = pow2f(-e);
    uint8_t* rows = v.pages + slab * PAGE * kPagedD;
    const bool bounds = keys && v.bounds;
    uint32_t lo[8], hi[8];                                        // of this thread's columns, as fp16 pairs
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = 0x7C007C00u;
        hi[i] = 0xFC00FC00u;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * kPass + (tid >> 3);
        if (r >= r1) continue;
        uint32_t u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = e4m3x2(x[i][2 * k] * inv, x[i][2 * k + 1] * inv);
        *reinterpret_cast<uint2*>(rows + r * kPagedD + 8 * c) = make_uint2(u[0] | (u[1] << 16), u[2] | (u[3] << 16));
        *reinterpret_cast<uint2*>(rows + r * kPagedD + 64 + 8 * c) = make_uint2(u[4] | (u[5] << 16), u[6] | (u[7] << 16));
        if (bounds) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u[k], __NV_E4M3);
                const __half2 y = *reinterpret_cast<const __half2*>(&h);
                lo[k] = as_u32(__hmin2(as_half2(lo[k]), y));
                hi[k] = as_u32(__hmax2(as_half2(hi[k]), y));
            }
        }
    }
    if (tid == 0) v.scales[slab] = scale;
    // older rows of a scale that grows: rounded again, 16 values a thread
    if (r0 > 0 && scale != was) {
        const float ratio = was * inv;
        uint4* old = reinterpret_cast<uint4*>(rows);
        for (int i = tid; i < r0 * (kPagedD / 16); i += kThreads) {
            uint4 u = old[i];
            uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 y = e4m3x2_f32(w[k] & 0xFFFFu), z = e4m3x2_f32(w[k] >> 16);
                w[k] = e4m3x2(y.x * ratio, y.y * ratio) | (e4m3x2(z.x * ratio, z.y * ratio) << 16);
            }
            old[i] = u;
        }
    }
    if (!bounds) return;
    // over the four rows of a warp's eight threads each, then over the warps
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int o = 8; o <= 16; o <<= 1) {
            lo[k] = as_u32(__hmin2(as_half2(lo[k]), as_half2(__shfl_xor_sync(0xffffffffu, lo[k], o))));
            hi[k] = as_u32(__hmax2(as_half2(hi[k]), as_half2(__shfl_xor_sync(0xffffffffu, hi[k], o))));
        }
        if (lane < 8) {
            s_lo[warp][(k >> 2) * 32 + 4 * c + (k & 3)] = lo[k];
            s_hi[warp][(k >> 2) * 32 + 4 * c + (k & 3)] = hi[k];
        }
    }
    __syncthreads();
    if (tid < kPagedD / 2) {
        __half2 l2 = as_half2(s_lo[0][tid]), h2 = as_half2(s_hi[0][tid]);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            l2 = __hmin2(l2, as_half2(s_lo[w][tid]));
            h2 = __hmax2(h2, as_half2(s_hi[w][tid]));
        }
        float2 l = __half22float2(l2), h = __half22float2(h2);
        l = make_float2(l.x * scale, l.y * scale);
        h = make_float2(h.x * scale, h.y * scale);
        __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(v.bounds + ((int64_t)pid * v.hkv + g) * 2 * kPagedD) + tid;
        if (r0 > 0) {
            const float2 ol = __bfloat1622float2(b[0]), oh = __bfloat1622float2(b[kPagedD / 2]);
            l = make_float2(fminf(l.x, round_to(ol.x, scale, inv)), fminf(l.y, round_to(ol.y, scale, inv)));
            h = make_float2(fmaxf(h.x, round_to(oh.x, scale, inv)), fmaxf(h.y, round_to(oh.y, scale, inv)));
        }
        b[0] = __floats2bfloat162_rn(l.x, l.y);                   // exact
        b[kPagedD / 2] = __floats2bfloat162_rn(h.x, h.y);
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
    a.parts = 2 * kv->hkv;
    if (items * a.parts > INT32_MAX) return set_error(MSA_ERR_UNSUPPORTED, "msa_paged_append: too many pages a call");
    const dim3 grid((unsigned)(items * a.parts));
    if (dt == MSA_BF16) launch_paged_append<__nv_bfloat16>(a, grid, static_cast<cudaStream_t>(stream));
    else launch_paged_append<float>(a, grid, static_cast<cudaStream_t>(stream));
    MSA_LAUNCH_CHECK();
    return MSA_OK;
}
