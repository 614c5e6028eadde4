// Picking the pages of a paged cache that a query token attends over, by the bounds of their keys.
//
//   score(token, kv head, page) = max over the group's query heads of sum_d max(q_d lo_d, q_d hi_d),
// the largest logit (before the scale) that any key inside the page's bounds could give; the newest pages count
// as infinite, the k best are picked, ties to the lower page, and listed in ascending order. What is picked is
// decided by sums in 64 bits, so that it does not depend on the order of summation. Those cost 64-bit
// operations for every page, so they are done for the pages near the border alone:
//
// 1. page_score_kernel: all scores in fp32 on the tensor cores. max(q lo, q hi) = min(q, 0) lo + max(q, 0) hi
//    where lo <= hi, so the scores of 16 pages and 8 query rows are one product over 2 * 128 elements whose page
//    operand is the bounds as they lie in memory. The products of two bf16 are exact; the sums are off by at
//    most E = 2^-14 sum|q_d| max|bound|: a step adds 17 numbers, and if each is cut off at 2^-23 of the largest,
//    16 steps lose 2^-14.9 of the sum of magnitudes. Bound by the bytes of the bounds, 512 per page and kv head,
//    where there are few query rows; 64 tokens of 32 heads over 6,250 pages take 37 us from a cold
//    cache, the tensor pipe active for 39 % of it; the pick after it 33 us, passes over 6,250 scores a token and head.
// 2. page_pick_kernel: one block per (token, kv head). T = the k-th best fp32 score, by its bits from the top, two
//    at a time (counting only: no histogram, whose counters equal leading bits would all hit), among the scores
//    that reach the k-th best of the threads' maxima where k is at most 256. Pages above T + 2 E are in, those
//    below T - 2 E are out, and where more than k remain those in between are summed again in 64 bits and ranked.
#include <algorithm>
#include <mutex>

#include "kernels.cuh"
#include "mma.cuh"
#include "paged.cuh"

namespace msa {
namespace {

struct SelectArgs {
    PagedView v;
    const __nv_bfloat16* q;
    int64_t n_tok;
    const int64_t* tok_off;
    int max_new, G, k, recent;
    int32_t* sel;
    int64_t first, last;           // the packed rows of this launch
    // from `first` on: [rows][hkv][max_pages], fp32 scores in a row's first half, later 64-bit keys
    unsigned long long* rows;
    float* bmax;                   // [rows][hkv][chunks], row of a sequence's first token: largest |bound| of 128 pages
    int chunks, token_parts;       // of the scoring grid
    int scores_in_smem;
    int* err;
};

constexpr int kScorePages = 128;   // pages per block of the scoring kernel
constexpr int kGroup = 8;          // query row tiles staged together, one per warp
constexpr int kPickThreads = 256;
constexpr int kNear = kPickThreads;            // border pages that are ranked in shared memory
constexpr int kCand = 1023;                    // candidates for the k best that are kept there
constexpr size_t kPickSmem = 200 * 1024;       // of scores; more pages are all summed in 64 bits
constexpr float kNoPage = -3.402823466e38f;    // score of a page that is not there

// Of a sequence's new tokens those of this launch, as if the last of them ended the sequence.
__device__ __forceinline__ void clip(const SelectArgs& a, SeqSpan* sp) {
    const int64_t end = sp->t0 + sp->n_new, t0 = max(sp->t0, a.first), t1 = max(t0, min(end, a.last));
    sp->len -= (int)(end - t1);
    sp->n_new = (int)(t1 - t0);
    sp->t0 = t0;
}

// The larger; a NaN stays.
__device__ __forceinline__ float max_nan(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

__global__ void __launch_bounds__(256, 2) page_score_kernel(const SelectArgs a) {
    __shared__ uint4 s_q[kGroup][8][32];       // B fragments: [row tile][16-byte piece][lane]
    __shared__ float s_top[8];
    const PagedView& v = a.v;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int s = blockIdx.x / a.chunks, chunk = blockIdx.x - s * a.chunks;
    const int g = blockIdx.y / a.token_parts, part = blockIdx.y - g * a.token_parts;
    const int G = a.G, gs = 31 - __clz(G), hq = v.hkv * G;
    next_may_launch();
    SeqSpan sp;
    if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, nullptr)) return;
    clip(a, &sp);
    if (sp.n_new == 0) return;
    const int n_pages = (sp.len + v.page - 1) >> v.shift;
    const int p0 = chunk * kScorePages;
    if (p0 >= n_pages || n_pages <= a.k) return;           // every visible page is picked
    const int row_tiles = (sp.n_new * G + 7) / 8;
    const int per = (row_tiles + a.token_parts - 1) / a.token_parts;
    const int rt0 = part * per, rt1 = min(row_tiles, rt0 + per);
    if (rt0 >= rt1) return;

    // A warp lays out one tile of 8 query rows of a group; its elements are on their way while the group before is
    // multiplied.
    uint4 next[4];
    auto fetch = [&](int rt) {
        const int row = (rt + warp) * 8 + r;
        const bool valid = rt + warp < rt1 && row < sp.n_new * G;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((sp.t0 + (valid ? row >> gs : 0)) * hq + g * G + (valid ? row & (G - 1) : 0)) * kPagedD) + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = valid ? src[4 * i] : make_uint4(0, 0, 0, 0);
    };
    fetch(rt0);
    // A: bounds of pages r and r + 8 of the warp's 16; the thread's 16-byte pieces are 4 i + c
    uint4 w[2][8];
    bool there[2];
    int32_t pid[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int p = p0 + 16 * warp + 8 * h + r;
        pid[h] = p < n_pages ? v.table[(int64_t)s * v.max_pages + p] : -1;
        there[h] = pid[h] >= 0 && pid[h] < v.n_pages;
        if (p < n_pages && !there[h] && c == 0) record_device_error(a.err, MSA_DEV_BAD_INDEX);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4* b = reinterpret_cast<const uint4*>(v.bounds + ((int64_t)pid[h] * v.hkv + g) * 2 * kPagedD) + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[h][i] = there[h] ? b[4 * i] : make_uint4(0, 0, 0, 0);
    }

    for (int rt = rt0; rt < rt1; rt += kGroup) {
        const int n_rt = min(kGroup, rt1 - rt);
        __syncthreads();
        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 neg, pos;
            const uint32_t* xs = &next[i].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&xs[j]);
                const __nv_bfloat162 lo = __hmin2_nan(y, zero), hi = __hmax2_nan(y, zero);
                (&neg.x)[j] = *reinterpret_cast<const uint32_t*>(&lo);
                (&pos.x)[j] = *reinterpret_cast<const uint32_t*>(&hi);
            }
            s_q[warp][i][lane] = neg;                      // against the minima, the first 128 elements
            s_q[warp][4 + i][lane] = pos;
        }
        __syncthreads();
        if (rt + kGroup < rt1) fetch(rt + kGroup);
        // two row tiles at a time: two chains of products
        for (int t0 = 0; t0 < n_rt; t0 += 2) {
            float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 b0 = s_q[t0][i][lane], b1 = s_q[t0 + 1][i][lane];      // kGroup is even
                const uint32_t a0[4] = {w[0][i].x, w[1][i].x, w[0][i].y, w[1][i].y};
                const uint32_t a1[4] = {w[0][i].z, w[1][i].z, w[0][i].w, w[1][i].w};
                mma_bf16_16816(x[0], a0, b0.x, b0.y);
                mma_bf16_16816(x[1], a0, b1.x, b1.y);
                mma_bf16_16816(x[0], a1, b0.z, b0.w);
                mma_bf16_16816(x[1], a1, b1.z, b1.w);
            }
            // x: page r, rows 2 c and 2 c + 1; page r + 8, the same rows. The largest of a token's rows:
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int row = (rt + t0 + t) * 8 + 2 * c;
                const bool mine = t0 + t < n_rt;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = p0 + 16 * warp + 8 * h + r;
                    float y = x[t][2 * h];
                    if (G == 1) {
                        if (mine && p < n_pages && row + 1 < sp.n_new)
                            reinterpret_cast<float*>(a.rows + ((sp.t0 - a.first + row + 1) * v.hkv + g) * v.max_pages)[p] =
                                there[h] ? x[t][2 * h + 1] : kNoPage;
                    } else {
                        y = fmaxf(y, x[t][2 * h + 1]);
                        if (G >= 4) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
                        if (G >= 8) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
                    }
                    const int tok = row >> gs;
                    if (mine && (row & (G - 1)) == 0 && p < n_pages && tok < sp.n_new)
                        reinterpret_cast<float*>(a.rows + ((sp.t0 - a.first + tok) * v.hkv + g) * v.max_pages)[p] =
                            there[h] ? y : kNoPage;
                }
            }
        }
    }
    if (part == 0) {
        float top = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u[4] = {w[h][i].x, w[h][i].y, w[h][i].z, w[h][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = fabsf(__uint_as_float(u[j] << 16)), y = fabsf(__uint_as_float(u[j] & 0xFFFF0000u));
                    top = max_nan(top, max_nan(x, y));
                }
            }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) s_top[warp] = top;
        __syncthreads();
        if (tid == 0) {
            float x = 0.f;
            for (int i = 0; i < 8; ++i) x = max_nan(x, s_top[i]);
            a.bmax[((sp.t0 - a.first) * v.hkv + g) * a.chunks + chunk] = x;
        }
    }
}

// Order-preserving maps to unsigned integers (-0 counts as +0, NaN as the least).
__device__ __forceinline__ uint32_t ordered32(float x) {
    if (!(x == x)) return 0;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered32(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned long long ordered64(double x) {
    if (!(x == x)) return 0;
    const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

struct PickSmem {
    int cnt[2][3][kPickThreads / 32];
    float red[2][kPickThreads / 32];
    int near[kNear];
    unsigned long long key[kNear];
    int hist[256];
    unsigned long long prefix;
    int want, done;
    alignas(16) uint32_t top[kPickThreads], cand[kCand + 1];
    int cand_page[kCand], n_cand, n_near, n_in;
    uint32_t floor, kth;
};

// The k-th largest of v[0 .. n), n <= kPickThreads: every thread counts how many come before its own (equal ones by
// place); the one that finds k - 1 tells. One barrier; v[n ..] up to a multiple of 4 may hold anything.
__device__ __forceinline__ uint32_t block_kth(const uint32_t* v, int n, int k, uint32_t* told) {
    const int tid = threadIdx.x;
    if (tid < n) {
        const uint32_t x = v[tid];
        int before = 0;
#pragma unroll 4
        for (int i = 0; i < n; i += 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(v + i);
            before += (i < n) & (y.x > x || (y.x == x && i < tid));
            before += (i + 1 < n) & (y.y > x || (y.y == x && i + 1 < tid));
            before += (i + 2 < n) & (y.z > x || (y.z == x && i + 2 < tid));
            before += (i + 3 < n) & (y.w > x || (y.w == x && i + 3 < tid));
        }
        if (before == k - 1) *told = x;
    }
    __syncthreads();
    return *told;
}
// The k-th largest of v[0 .. n), n < 1024, by one warp: two bits at a time from the top, three counts in one sum.
__device__ __forceinline__ uint32_t warp_kth(const uint32_t* v, int n, int k) {
    const int lane = threadIdx.x & 31;
    uint32_t T = 0;
    for (int shift = 30; shift >= 0; shift -= 2) {
        const uint32_t t1 = T | (1u << shift), t2 = T | (2u << shift), t3 = T | (3u << shift);
        uint32_t c = 0;
        for (int i = lane; i < n; i += 32) {
            const uint32_t y = v[i];
            c += (y >= t1) + ((y >= t2) << 10) + ((y >= t3) << 20);
        }
        c = __reduce_add_sync(0xffffffffu, c);
        T = (int)(c >> 20) >= k ? t3 : (int)(c >> 10 & 1023) >= k ? t2 : (int)(c & 1023) >= k ? t1 : T;
    }
    return T;
}

// Sum over the block of three counts per thread; `turn` alternates, so that one barrier a call is enough.
__device__ __forceinline__ int3 block_count(PickSmem& sm, int turn, int x, int y, int z) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    z = __reduce_add_sync(0xffffffffu, z);
    if (lane == 0) {
        sm.cnt[turn][0][warp] = x;
        sm.cnt[turn][1][warp] = y;
        sm.cnt[turn][2][warp] = z;
    }
    __syncthreads();
    int3 t = make_int3(0, 0, 0);
#pragma unroll
    for (int w = 0; w < kPickThreads / 32; ++w) {
        t.x += sm.cnt[turn][0][w];
        t.y += sm.cnt[turn][1][w];
        t.z += sm.cnt[turn][2][w];
    }
    return t;
}

// Calls put(place, i) for the i in [0, n) with test(i), place counting them in ascending order.
template <typename Test, typename Put>
__device__ __forceinline__ void compact(PickSmem& sm, int n, Test test, Put put) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int before = 0;
    __syncthreads();
    for (int i0 = 0, turn = 0; i0 < n; i0 += kPickThreads, turn ^= 1) {
        const int i = i0 + tid;
        const bool yes = i < n && test(i);
        const unsigned m = __ballot_sync(0xffffffffu, yes);
        if (lane == 0) sm.cnt[turn][0][warp] = __popc(m);
        __syncthreads();
        int at = before;
#pragma unroll
        for (int w = 0; w < kPickThreads / 32; ++w) {
            const int x = sm.cnt[turn][0][w];
            if (w < warp) at += x;
            before += x;
        }
        if (yes) put(at + __popc(m & ((1u << lane) - 1)), i);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectArgs a) {
    extern __shared__ uint32_t s_score[];
    __shared__ PickSmem sm;
    const PagedView& v = a.v;
    const int64_t t = a.first + blockIdx.x;
    const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.G, hq = v.hkv * G;
    wait_for_earlier();
    if (g == 0 && warp == kPickThreads / 32 - 1) {         // sequences that no token leads to are looked at too
        SeqSpan each;
        for (int64_t i = blockIdx.x + (int64_t)lane * gridDim.x; i < v.n_seq; i += 32ll * gridDim.x)
            seq_span(v, a.tok_off, a.n_tok, a.max_new, (int)i, &each, a.err);
    }
    const int s = seq_of_token(a.tok_off, v.n_seq, t);
    SeqSpan sp;
    int32_t* sel = a.sel + (t * v.hkv + g) * a.k;
    if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, tid == 0 ? a.err : nullptr) || t < sp.t0 ||
        t >= sp.t0 + sp.n_new)
        return;
    clip(a, &sp);
    const int n = ((sp.len - sp.n_new + (int)(t - sp.t0)) >> v.shift) + 1;      // visible pages
    if (n <= a.k) {
        for (int i = tid; i < a.k; i += kPickThreads) sel[i] = i < n ? i : -1;
        return;
    }
    const int newest = max(0, n - a.recent);               // pages from here on are in
    unsigned long long* row64 = a.rows + ((int64_t)blockIdx.x * v.hkv + g) * v.max_pages;
    const __nv_bfloat16* q = a.q + (t * hq + g * G) * kPagedD;

    // a page's score in 64 bits, by one warp
    auto exact = [&](int p) -> unsigned long long {
        const int32_t pid = v.table[(int64_t)s * v.max_pages + p];
        if (pid < 0 || pid >= v.n_pages) return ordered64((double)-INFINITY);
        const __nv_bfloat16* b = v.bounds + ((int64_t)pid * v.hkv + g) * 2 * kPagedD + lane * 4;
        double lo[4], hi[4], best = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = (double)__bfloat162float(b[i]);
            hi[i] = (double)__bfloat162float(b[kPagedD + i]);
        }
        for (int h = 0; h < G; ++h) {
            double x = 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const double y = (double)__bfloat162float(q[h * kPagedD + lane * 4 + i]);
                x += fmax(y * lo[i], y * hi[i]);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            best = fmax(best, x);
        }
        return ordered64(best);
    };
    // the `want` largest of keys[0 .. m), the first of equal ones: by digits of 8 bits, to the edge's bits above
    // `shift` and the number of keys equal to it that are taken
    auto radix = [&](const unsigned long long* keys, int m, int want, int* shift_out, unsigned long long* edge, int* ties) {
        if (tid == 0) {
            sm.prefix = 0;
            sm.want = want;
            sm.done = 0;
        }
        __syncthreads();
        int shift = 56;
        for (;; shift -= 8) {
            sm.hist[tid] = 0;
            __syncthreads();
            const unsigned long long prefix = sm.prefix;
            for (int i = tid; i < m; i += kPickThreads) {
                const unsigned long long x = keys[i];
                if (shift == 56 || (x >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&sm.hist[(int)(x >> shift) & 255], 1);
            }
            __syncthreads();
            if (warp == 0) {
                int c = 0;                                 // lane l holds digits 255 - 8 l .. 248 - 8 l
#pragma unroll
                for (int i = 0; i < 8; ++i) c += sm.hist[255 - 8 * lane - i];
                int above = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, above, o);
                    if (lane >= o) above += y;
                }
                above -= c;
                const int need = sm.want;
                __syncwarp();
                if (above < need && above + c >= need) {
                    int i = 0;
                    while (above + sm.hist[255 - 8 * lane - i] < need) above += sm.hist[255 - 8 * lane - i++];
                    const int digit = 255 - 8 * lane - i;
                    sm.prefix = prefix | ((unsigned long long)digit << shift);
                    sm.want = need - above;
                    sm.done = sm.hist[digit] == need - above;          // the whole bucket is taken
                }
            }
            __syncthreads();
            if (shift == 0 || sm.done) break;
        }
        *shift_out = shift;
        *edge = sm.prefix >> shift;
        *ties = sm.want;
        __syncthreads();
    };
    // takes the `want` best of all n keys of row64
    auto take_from_row = [&](int want) {
        int shift, ties;
        unsigned long long edge;
        radix(row64, n, want, &shift, &edge, &ties);
        // equal keys are counted first, so that each knows its rank among them
        int equal = 0, at = 0;
        for (int i0 = 0, turn = 0; i0 < n; i0 += kPickThreads, turn ^= 1) {
            const int i = i0 + tid;
            const unsigned long long x = i < n ? row64[i] >> shift : 0;
            const bool gt = i < n && x > edge, eq = i < n && x == edge;
            const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
            if (lane == 0) {
                sm.cnt[turn][0][warp] = __popc(mg);
                sm.cnt[turn][1][warp] = __popc(me);
            }
            __syncthreads();
            int cg = at, ce = equal;
#pragma unroll
            for (int w = 0; w < kPickThreads / 32; ++w) {
                const int xg = sm.cnt[turn][0][w], xe = sm.cnt[turn][1][w];
                if (w < warp) {
                    cg += xg;
                    ce += xe;
                }
                at += xg;
                equal += xe;
            }
            cg += __popc(mg & ((1u << lane) - 1));
            ce += __popc(me & ((1u << lane) - 1));
            if (gt || (eq && ce < ties)) sel[cg + min(ce, ties)] = i;
        }
    };

    if (!a.scores_in_smem) {                               // the scores were not made: all pages in 64 bits
        for (int p = warp; p < n; p += kPickThreads / 32) {
            const unsigned long long x = p >= newest ? ~0ull : exact(p);
            if (lane == 0) row64[p] = x;
        }
        __syncthreads();
        take_from_row(a.k);
        return;
    }

    // the scores, and how far they may be off
    const float* score = reinterpret_cast<const float*>(row64);
    const float* bmax = a.bmax + ((sp.t0 - a.first) * v.hkv + g) * a.chunks;
    float bm = 0.f;
    uint32_t mine = 0;
#pragma unroll 8
    for (int i = tid; i < n; i += kPickThreads) {
        const uint32_t x = i >= newest ? 0xFFFFFFFFu : ordered32(score[i]);
        s_score[i] = x;
        mine = max(mine, x);
    }
    for (int i = tid; i < (n + kScorePages - 1) / kScorePages; i += kPickThreads) bm = max_nan(bm, bmax[i]);
    float qs = 0.f;
    if (warp < G) {
#pragma unroll
        for (int i = 0; i < 4; ++i) qs += fabsf(__bfloat162float(q[warp * kPagedD + lane * 4 + i]));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) qs += __shfl_xor_sync(0xffffffffu, qs, o);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) bm = max_nan(bm, __shfl_xor_sync(0xffffffffu, bm, o));
    if (lane == 0) {
        sm.red[0][warp] = qs;
        sm.red[1][warp] = bm;
    }
    __syncthreads();
    qs = bm = 0.f;
#pragma unroll
    for (int w = 0; w < kPickThreads / 32; ++w) {
        qs = max_nan(qs, sm.red[0][w]);
        bm = max_nan(bm, sm.red[1][w]);
    }
    // 2^-14, and what underflow may lose; NaN, and with it all pages near the border, where a query or a bound is
    const float E = qs * bm * 6.103515625e-05f + 1e-36f;

    // Few candidates first, where k allows: at least k scores reach the k-th best of the threads' own maxima, folded to
    // 2 k of them or a little more (about 1.4 k scores reach that; fewer maxima are quicker to rank).
    const bool few = a.k <= kPickThreads;
    if (few) {
        const int fold = a.k > 64 ? 0 : a.k > 32 ? 1 : a.k > 16 ? 2 : 3;
        for (int o = 0; o < fold; ++o) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, 1 << o));
        if ((tid & ((1 << fold) - 1)) == 0) sm.top[tid >> fold] = mine;
        if (tid == 0) sm.n_cand = 0;
        __syncthreads();
        const uint32_t t = block_kth(sm.top, kPickThreads >> fold, a.k, &sm.floor);
        const float f = unordered32(t);
        // everything near the border, wherever above it that turns out to be, and all that compares with nothing
        const uint32_t floor = t == 0xFFFFFFFFu ? t : (f - 2.f * E > -3.402823466e38f) ? ordered32(f - 2.f * E) : 0u;
        for (int i0 = 0; i0 < n; i0 += kPickThreads) {     // as many turns for every lane: all take part in the votes
            const int i = i0 + tid;
            const uint32_t x = i < n ? s_score[i] : 0;
            const bool yes = i < n && (x >= floor || x == 0);
            const unsigned m = __ballot_sync(0xffffffffu, yes);
            if (m == 0) continue;                          // of the whole warp
            int at = 0;
            if (lane == 0) at = atomicAdd(&sm.n_cand, __popc(m));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1));
            if (yes && at < kCand) {
                sm.cand[at] = x;
                sm.cand_page[at] = i;
            }
        }
        __syncthreads();
    }
    if (few && sm.n_cand <= kCand) {
        const int n_cand = sm.n_cand;
        if (tid == 0) sm.n_near = sm.n_in = 0;
        const int words = (n + 31) / 32;                   // a bit per page, in the place of the scores
        uint32_t* bits = s_score;
        for (int i = tid; i < words; i += kPickThreads) bits[i] = 0;
        uint32_t T;
        if (n_cand <= kPickThreads) {
            T = block_kth(sm.cand, n_cand, a.k, &sm.kth);
        } else {
            if (warp == 0) {
                const uint32_t t = warp_kth(sm.cand, n_cand, a.k);
                if (lane == 0) sm.kth = t;
            }
            __syncthreads();
            T = sm.kth;
        }
        const float edge = unordered32(T), low = edge - 2.f * E, high = edge + 2.f * E;
        for (int i = tid; i < n_cand; i += kPickThreads) {
            const uint32_t x = sm.cand[i];
            const float y = unordered32(x);
            const int p = sm.cand_page[i];
            if (x == 0xFFFFFFFFu || (T != 0xFFFFFFFFu && x != 0 && y > high)) {
                atomicOr(&bits[p >> 5], 1u << (p & 31));
                atomicAdd(&sm.n_in, 1);
            } else if (T != 0xFFFFFFFFu && !(x != 0 && y < low)) {
                const int at = atomicAdd(&sm.n_near, 1);
                if (at < kNear) sm.near[at] = p;
            }
        }
        __syncthreads();
        const int want = a.k - sm.n_in, n_near = sm.n_near;
        if (n_near <= kNear) {
            if (n_near > want) {
                for (int j = warp; j < n_near; j += kPickThreads / 32) {
                    const unsigned long long x = exact(sm.near[j]);
                    if (lane == 0) sm.key[j] = x;
                }
                __syncthreads();
            }
            if (tid < n_near) {
                const int p = sm.near[tid];
                int rank = 0;
                if (n_near > want) {
                    const unsigned long long x = sm.key[tid];
                    for (int j = 0; j < n_near; ++j) {
                        const unsigned long long y = sm.key[j];
                        rank += y > x || (y == x && sm.near[j] < p);
                    }
                }
                if (rank < want) atomicOr(&bits[p >> 5], 1u << (p & 31));
            }
            __syncthreads();
            // the set bits in ascending order: each thread a run of words
            const int run = (words + kPickThreads - 1) / kPickThreads;
            const int w0 = min(words, tid * run), w1 = min(words, w0 + run);
            int c = 0;
            for (int i = w0; i < w1; ++i) c += __popc(bits[i]);
            int up = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += y;
            }
            if (lane == 31) sm.cnt[0][0][warp] = up;
            __syncthreads();
            int at = up - c;
            for (int i = 0; i < warp; ++i) at += sm.cnt[0][0][i];
            for (int i = w0; i < w1; ++i)
                for (uint32_t m = bits[i]; m; m &= m - 1) sel[at++] = i * 32 + __ffs(m) - 1;
            return;
        }
        // too many: the scores again, for the passes over all of them
        __syncthreads();
        for (int i = tid; i < n; i += kPickThreads) s_score[i] = i >= newest ? 0xFFFFFFFFu : ordered32(score[i]);
        __syncthreads();
    }
    uint32_t T = 0;                                        // the k-th largest, two bits at a time
    for (int shift = 30, turn = 0; shift >= 0; shift -= 2, turn ^= 1) {
        const uint32_t t1 = T | (1u << shift), t2 = T | (2u << shift), t3 = T | (3u << shift);
        int c1 = 0, c2 = 0, c3 = 0;
        for (int i = tid; i < n; i += kPickThreads) {
            const uint32_t x = s_score[i];
            c1 += x >= t1;
            c2 += x >= t2;
            c3 += x >= t3;
        }
        const int3 c = block_count(sm, turn, c1, c2, c3);
        T = c.z >= a.k ? t3 : c.y >= a.k ? t2 : c.x >= a.k ? t1 : T;
    }
    const float edge = unordered32(T);
    const bool all_new = T == 0xFFFFFFFFu;                 // the newest pages are the k best
    const float low = edge - 2.f * E, high = edge + 2.f * E;
    // 2 in, 1 near the border, 0 out; comparisons with NaN or infinite bounds put a page near the border
    auto place = [&](int i) -> int {
        const uint32_t x = s_score[i];
        if (x == 0xFFFFFFFFu) return 2;
        if (all_new) return 0;
        const float y = unordered32(x);
        if (x != 0 && y > high) return 2;
        if (x != 0 && y < low) return 0;
        return 1;
    };
    int n_in = 0, n_near = 0;
    for (int i = tid; i < n; i += kPickThreads) {
        const int w = place(i);
        n_in += w == 2;
        n_near += w == 1;
    }
    const int3 c = block_count(sm, 0, n_in, n_near, 0);
    n_in = c.x;
    n_near = c.y;
    const int want = a.k - n_in;
    if (n_near == want) {
        compact(sm, n, [&](int i) { return place(i) > 0; }, [&](int at, int i) { sel[at] = i; });
        return;
    }
    if (n_near <= kNear) {
        compact(sm, n, [&](int i) { return place(i) == 1; }, [&](int at, int i) { sm.near[at] = i; });
        for (int j = warp; j < n_near; j += kPickThreads / 32) {
            const unsigned long long x = exact(sm.near[j]);
            if (lane == 0) sm.key[j] = x;
        }
        __syncthreads();
        if (tid < n_near) {
            const unsigned long long x = sm.key[tid];
            int rank = 0;
            for (int j = 0; j < n_near; ++j) {
                const unsigned long long y = sm.key[j];
                rank += y > x || (y == x && j < tid);
            }
            s_score[sm.near[tid]] = rank < want ? 0xFFFFFFFFu : 0xFFFFFFFEu;
        }
        __syncthreads();
        compact(sm, n, [&](int i) { return s_score[i] == 0xFFFFFFFFu || (s_score[i] != 0xFFFFFFFEu && place(i) == 2); },
                [&](int at, int i) { sel[at] = i; });
        return;
    }
    // many scores at the border (equal ones, or bounds without a finite error): the 64-bit keys take the row's place
    for (int p = warp; p < n; p += kPickThreads / 32) {
        const int w = place(p);
        const unsigned long long x = w == 2 ? ~0ull : w == 0 ? 0ull : exact(p);
        if (lane == 0) row64[p] = x;
    }
    __syncthreads();
    take_from_row(a.k);
}

// The workspace: rows of scores and maxima of bounds of as many packed rows as fit kSelectBytes, one at least; a longer
// call goes through its rows in slices of that many. (All at once, 65,536 tokens of 8 kv heads over their 1,024 pages
// would take 4 GB; a slice of them is 4,096 tokens, whose scores far outweigh reading the bounds again.)
constexpr size_t kSelectBytes = 256u << 20;
struct SelectPlan {
    int64_t slice;         // packed rows
    int chunks;
    size_t bmax, bytes;    // offset and size in the workspace
};
SelectPlan select_plan(int64_t n_tok, int hkv, int max_pages) {
    SelectPlan p{};
    p.chunks = (max_pages + kScorePages - 1) / kScorePages;
    const size_t row = (size_t)hkv * max_pages * sizeof(unsigned long long), top = (size_t)hkv * p.chunks * sizeof(float);
    p.slice = std::min<int64_t>(n_tok, std::max<int64_t>(1, (int64_t)((kSelectBytes - 512) / (row + top))));
    p.bmax = align_up(p.slice * row, 256);
    p.bytes = p.bmax + align_up(p.slice * top, 256);
    return p;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_page_select_workspace_size(int64_t n_tok, int hkv, int max_pages, size_t* bytes) {
    MSA_REQUIRE(bytes != nullptr, "msa_page_select_workspace_size: bytes is NULL");
    MSA_REQUIRE(n_tok >= 0 && n_tok < (int64_t)INT32_MAX / 2 && hkv > 0 && hkv <= 4096 && max_pages > 0,
                "msa_page_select_workspace_size: bad sizes");
    *bytes = select_plan(n_tok, hkv, max_pages).bytes;
    return MSA_OK;
}

extern "C" msa_status msa_page_select(const msa_paged_kv* kv, const void* q, msa_dtype dt, int64_t n_tok, int hq,
                                      const int64_t* tok_off, int max_new, int k, int recent, int32_t* sel, void* ws,
                                      size_t ws_bytes, void* stream) {
    SelectArgs a{};
    MSA_RETURN_IF(paged_view(kv, "msa_page_select", &a.v));
    MSA_REQUIRE(dtype_ok(dt), "msa_page_select: bad dtype");
    if (dt != MSA_BF16) return set_error(MSA_ERR_UNSUPPORTED, "msa_page_select: bf16 queries only");
    MSA_RETURN_IF(paged_tokens_ok(kv, "msa_page_select", n_tok, tok_off, max_new));
    MSA_REQUIRE(kv->bounds != nullptr, "msa_page_select: the cache has no bounds");
    MSA_REQUIRE(hq > 0 && hq % kv->hkv == 0, "msa_page_select: hq must be a multiple of hkv");
    a.G = hq / kv->hkv;
    if (a.G != 1 && a.G != 2 && a.G != 4 && a.G != 8)
        return set_error(MSA_ERR_UNSUPPORTED, "msa_page_select: hq/hkv = %d unsupported", a.G);
    MSA_REQUIRE(k >= 1 && recent >= 1 && recent <= k, "msa_page_select: need 1 <= recent <= k");
    if (n_tok == 0 || max_new == 0) return MSA_OK;
    MSA_REQUIRE(q && sel && ws, "msa_page_select: NULL pointer");
    MSA_REQUIRE(aligned16(q) && aligned16(sel) && aligned16(ws), "msa_page_select: pointers must be 16-byte aligned");
    size_t need = 0;
    MSA_RETURN_IF(msa_page_select_workspace_size(n_tok, kv->hkv, kv->max_pages, &need));
    if (ws_bytes < need) return set_error(MSA_ERR_WORKSPACE, "msa_page_select: workspace %zu < %zu", ws_bytes, need);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.n_tok = n_tok; a.tok_off = tok_off; a.max_new = max_new; a.k = k; a.recent = recent; a.sel = sel;
    a.rows = static_cast<unsigned long long*>(ws);
    const SelectPlan p = select_plan(n_tok, kv->hkv, kv->max_pages);
    a.bmax = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.bmax);
    a.err = device_error_word();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.chunks = p.chunks;
    if ((int64_t)a.chunks * kv->n_seq > INT32_MAX)
        return set_error(MSA_ERR_UNSUPPORTED, "msa_page_select: n_seq * max_pages too large");
    size_t smem = (size_t)kv->max_pages * sizeof(uint32_t);
    a.scores_in_smem = smem <= kPickSmem;
    if (!a.scores_in_smem) smem = 0;
    const bool scored = k < kv->max_pages && a.scores_in_smem;
    static std::mutex mu;
    static bool opted[64] = {false};
    int dev = 0;
    MSA_CUDA_TRY(cudaGetDevice(&dev));
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64 || !opted[dev]) {
            MSA_CUDA_TRY(cudaFuncSetAttribute(page_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPickSmem));
            if (dev >= 0 && dev < 64) opted[dev] = true;
        }
    }
    for (a.first = 0; a.first < n_tok; a.first = a.last) {
        a.last = std::min(n_tok, a.first + p.slice);
        const int64_t rows = a.last - a.first;
        if (scored) {
            // blocks for every SM: where pages and heads do not give enough, a sequence's query rows are parted too
            const int64_t blocks = (int64_t)a.chunks * kv->n_seq * kv->hkv;
            const int64_t groups = (std::min<int64_t>(max_new, rows) * a.G + 8 * kGroup - 1) / (8 * kGroup);
            a.token_parts = (int)std::max<int64_t>(1, std::min<int64_t>({groups, 592 / std::max<int64_t>(blocks, 1), 65535 / kv->hkv}));
            const dim3 grid((unsigned)(a.chunks * kv->n_seq), (unsigned)(kv->hkv * a.token_parts));
            page_score_kernel<<<grid, 256, 0, s>>>(a);
            MSA_LAUNCH_CHECK();
        }
        MSA_CUDA_TRY(launch_early(page_pick_kernel, dim3((unsigned)rows, (unsigned)kv->hkv), kPickThreads, smem, s, a));
    }
    return MSA_OK;
}
