// Attention of few query rows over a paged 8-bit cache: single tokens, a handful of drafted ones, single tokens over
// their page lists, and more tokens in blocks of 8 rows where there is little to do.
//
//   out = softmax(scale q . K) V,  up to 8 rows (token, query head) of one kv head at a time.
// Every cached byte is read once for 4 * 8 operations at most, so the bytes bound it, and what a warp spends on
// each byte decides how near it comes. A warp takes 32 keys at a time, transposed, so that all eight columns are
// rows of the softmax, on mma.sync with e4m3 operands, which take the cache's bytes as they are (the 128-row
// tiles of tcgen05.mma would be empty but for 1 to 8 rows; e4m3 mma.sync m16n8k32 measured 1.88 PFLOP/s here,
// fp16 m16n8k16 0.53):
//   S^T [32 keys x 8 rows]  = K [32 x 128] (Qhi + Qlo)^T
//   D   [128 x 8 rows]      = V^T [128 x 32] (Phi + Plo)^T,   O^T += D 2^(mt - m) scale(V)
// Q is split into two e4m3 parts of a row scaled to 224..448: eight significant bits, all that bf16 has, down to
// 2^-11 of the row's largest; what lies below is off by at most 2^-10 of the scale. P is taken against the
// tile's own maximum mt, times 2^8, and split into e4m3 and e5m2: an error of 2^-8 of the value (what one rounding
// to bf16 costs: e4m3 leaves less than 2^-4, and e5m2 an eighth of half of that), or of 2^-22 of the tile's largest
// for small ones, whose e4m3 part is a multiple of 2^-9 and leaves 2^-10 at most. O and the sum are fp32 against a
// maximum m that moves only when a tile exceeds it by 2^24. The order of d and of the keys inside the products
// is free: a thread takes the 16-byte pieces that it can read from shared memory without bank conflicts, and V
// needs no more than 4 x 4 byte transposes.
//
// One block per SM: a warp of its own looks the pages up, 20 tiles at a time, and brings keys and values by TMA in the
// 128-byte swizzle into a ring of 20 tiles of 8 KB (44 KB cover the latency of memory); another lays out the queries
// of the segment after the one in work; 10 warps take the tiles in turns.
//
// Measured, one token of 32 heads over 500,001: 198 us where the same context is read again and again, 213 to 217
// where it changes from call to call; 156 are its bytes at the copy rate. A block's tiles pass at 21 bytes a cycle and SM: no pipe
// is full (DRAM 62 %, tensor 31 %, 2.1 instructions issued a cycle); 10 warps with some 500 instructions a tile, in chains
// of shared memory, products and exponentials, set the pace. Start and merge take 10 us. 32 tokens over up to 16,384 each 122 us (89). Before:
// fp32 arithmetic 94 ms; fp16 and bf16 mma.sync with converted operands and 16-key tiles 246 us; e4m3 operands with each
// warp loading for itself 234 us; a loader warp 213 us. Where segments are short, what starting and ending one costs
// decides: 64 tokens over up to 300 each take 24 us, 52 where a segment's cost is left out of the blocks' shares and
// every warp prepares the queries.
#include <algorithm>
#include <mutex>

#include "kernels.cuh"
#include "mma.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace msa {
namespace {

constexpr int kWarps = 10, kConsumers = 32 * kWarps, kThreads = kConsumers + 64;   // and loader and query warps
constexpr int kSlots = 2 * kWarps;                         // two of its own for each warp
static_assert(kSlots <= 32, "a lane per slot");
constexpr int kTileBytes = 2 * kDecodeTile * kPagedD;      // K and V of a tile
constexpr int kWindow = kDecodeSeqs;                       // sequences looked at together
static_assert(kWindow == kConsumers, "a thread per sequence");
constexpr int kSegs = 2;                                   // segments whose queries are ready
constexpr float kSlack = 24.f;

struct __align__(16) TileInfo {      // of the tile's two halves of 16 keys
    int key[2];       // first key's place in the sequence
    int rows;         // keys that hold something, half 0 + 256 * half 1
    float vs;         // scale of V: the larger of the two
    float sk[2];      // scales of K
    float fac[2];     // scale of V over vs; below 2^-4 the halves are handled apart
};
constexpr int kFull = 16 + 256 * 16;

struct __align__(16) Segment {       // a block's piece of one
    int64_t t0;
    int head, n_rows, len, n_new;
    int end;                         // one past its last tile, counted from the block's first of the window
    int whole, starts;               // holds all tiles, the first one
};

struct DecodeSmem {
    uint8_t ring[kSlots][kTileBytes];
    float4 o[kWarps][kDecodeRows][kPagedD / 4];            // chunk i of row n at i ^ n / 2
    uint4 q[kSegs][4][32];                                 // fragments of Q^T by lane: high parts, low parts
    float f[kSegs][kDecodeRows];                           // logit factors of the rows
    Segment seg[kSegs];
    float2 ml[kWarps][kDecodeRows];
    TileInfo info[kSlots];
    uint64_t full[kSlots], empty[kSlots], seg_full[kSegs], seg_empty[kSegs], joined;
    int last[kSlots];                                      // loads of a slot so far
    long long pre[kWindow + 1], pre_u[kWindow + 1];        // tiles before each sequence of the window, and units
    int64_t t0[kWindow], first[kWindow];
    int n_new[kWindow], len[kWindow];
    long long scan[kWarps];
    int scan_live[kWarps], scan_most[kWarps];
    int abort_flag;
};

// c[4] += A [16 x 32] B [32 x 8], e4m3
__device__ __forceinline__ void mma_e4m3_16832(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c[4] = A B
__device__ __forceinline__ void mma_e4m3_16832_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                     uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// the same, B in e5m2
__device__ __forceinline__ void mma_e4m3_e5m2_16832(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e5m2.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// x0, x1 as pairs of e4m3, the nearest, and of e4m3 or e5m2, the nearest to what that leaves (all within fp16's range)
template <__nv_fp8_interpretation_t LO = __NV_E4M3>
__device__ __forceinline__ void split_e4m3(float x0, float x1, uint32_t* hi, uint32_t* lo) {
    const __half2 y = __floats2half2_rn(x0, x1);
    *hi = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)*hi, __NV_E4M3);
    *lo = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__hsub2(y, *reinterpret_cast<const __half2*>(&back)), __NV_SATFINITE, LO);
}

// x / d; the short division where it will do
__device__ __forceinline__ int quotient(long long x, int d) {
    return (unsigned long long)x >> 32 ? (int)(x / d) : (int)((unsigned)x / (unsigned)d);
}
// The last i with pre[i] <= g.
__device__ __forceinline__ int find(const long long* pre, int n, long long g) {
    int lo = 0;
    while (n > 1) {
        const int h = n / 2;
        if (pre[lo + h] <= g) {
            lo += h;
            n -= h;
        } else {
            n = h;
        }
    }
    return lo;
}

template <bool LIST>
__global__ void __launch_bounds__(kThreads, 1) paged_decode_kernel(const __grid_constant__ CUtensorMap tm,
                                                                   const PagedAttnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const PagedView& v = a.v;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.G, gs = 31 - __clz(G), hq = v.hkv * G, page = v.page;
    // tiles per page, or two pages per tile
    const bool pairs = page == 16;
    const int per_page = pairs ? 1 : page / kDecodeTile;
    const int list_tiles = !LIST ? 1 : pairs ? (a.k + 1) / 2 : a.k * per_page;
    const float ninf = -INFINITY;
    volatile int* abort_flag = &sm.abort_flag;
    next_may_launch();
    if (tid == 32) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm)) : "memory");
    if (tid == 0) sm.abort_flag = 0;
    if (tid == 0) mbar_init(smem_u32(&sm.joined), kWarps);
    if (tid < kSegs) {
        mbar_init(smem_u32(&sm.seg_full[tid]), 1);
        mbar_init(smem_u32(&sm.seg_empty[tid]), kWarps);
    }
    if (tid < kSlots) {
        mbar_init(smem_u32(&sm.full[tid]), 1);
        mbar_init(smem_u32(&sm.empty[tid]), 1);
        sm.last[tid] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    wait_for_earlier();

    // Tiles of all sequences, a thread per sequence of the window; and units, in which the blocks' shares are measured: a
    // segment's tiles and kSegWeight more, so that a block with many short segments gets fewer tiles; or whole segments,
    // where each gets a block.
    const int n_windows = LIST ? 1 : (v.n_seq + kWindow - 1) / kWindow;
    const bool at_hand = LIST && v.n_seq <= kWindow;       // the offsets and lengths of all sequences in shared memory
    struct Sums {
        long long tiles, units;
    };
    bool uncut = LIST && list_tiles <= kDecodeUncut && a.n_tok * v.hkv <= (long long)gridDim.x;
    auto load_window = [&](int w) -> Sums {
        const int s = w * kWindow + tid;
        SeqSpan sp{0, 0, 0};
        if (tid < kWindow && s < v.n_seq) seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, blockIdx.x == 0 ? a.err : nullptr);
        const int per_head = sp.n_new ? (sp.len + kDecodeTile - 1) / kDecodeTile : 0;
        int live = (sp.n_new * G + kDecodeRows - 1) / kDecodeRows, most = per_head;    // row blocks
        long long up = (long long)v.hkv * per_head * live;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, up, o);
            const int z = __shfl_up_sync(0xffffffffu, live, o);
            if (lane >= o) {
                up += y;
                live += z;
            }
        }
        most = __reduce_max_sync(0xffffffffu, most);
        __syncthreads();
        if (tid < kWindow) {
            sm.t0[tid] = sp.t0;
            if (LIST && s < v.n_seq) sm.first[tid] = a.tok_off[s];
            sm.n_new[tid] = sp.n_new;
            sm.len[tid] = sp.len;
            if (lane == 31) {
                sm.scan[warp] = up;
                sm.scan_live[warp] = live;
                sm.scan_most[warp] = most;
            }
        }
        __syncthreads();
        long long before = 0, tiles = 0;
        int before_live = 0, all_live = 0;
        most = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const long long x = sm.scan[i];
            const int y = sm.scan_live[i];
            if (i < warp) {
                before += x;
                before_live += y;
            }
            tiles += x;
            all_live += y;
            most = max(most, sm.scan_most[i]);
        }
        if (!LIST) uncut = n_windows == 1 && most <= kDecodeUncut && (long long)all_live * v.hkv <= (long long)gridDim.x;
        const long long per_seg = uncut ? 1 : kSegWeight;
        if (tid < kWindow) {
            sm.pre[tid + 1] = before + up;
            sm.pre_u[tid + 1] = (uncut ? 0 : before + up) + (before_live + live) * per_seg * v.hkv;
        }
        const Sums all{tiles, (uncut ? 0 : tiles) + all_live * per_seg * v.hkv};
        if (tid == 0) sm.pre[0] = sm.pre_u[0] = 0;
        __syncthreads();
        return all;
    };
    Sums total{0, 0}, first_total{0, 0};
    if (LIST) {
        if (at_hand) {
            load_window(0);
        } else {                                           // sequences that no token leads to are looked at too
            SeqSpan each;
            for (int64_t i = blockIdx.x + (int64_t)tid * gridDim.x; i < v.n_seq; i += (int64_t)kThreads * gridDim.x)
                seq_span(v, a.tok_off, a.n_tok, a.max_new, (int)i, &each, a.err);
            __syncthreads();
        }
        total.tiles = total.units = a.n_tok * v.hkv * (long long)list_tiles;       // all segments are alike
        first_total = total;
    } else {
        for (int w = n_windows - 1; w >= 0; --w) {
            first_total = load_window(w);
            total.tiles += first_total.tiles;
            total.units += first_total.units;
        }
    }
    // Segment i of sequence `lo` of the window: head i % hkv, row block i / hkv, which is that of a sequence that ends
    // with the block's last token. (All segments of a sequence count as many tiles as the last block's; those behind a
    // block's end are passed over.)
    auto block_of = [&](int lo, int i, int* head, int64_t* t0, int* n_new, int* len) {
        const int rb = i / v.hkv, before = rb * (kDecodeRows >> gs), all = sm.n_new[lo];
        *head = i - rb * v.hkv;
        *t0 = sm.t0[lo] + before;
        *n_new = min(kDecodeRows >> gs, all - before);
        *len = sm.len[lo] - all + before + *n_new;
    };
    // tiles of the window before its unit u
    auto tiles_before = [&](long long u, int n_win) -> long long {
        if (LIST) return u;
        if (u >= sm.pre_u[n_win]) return sm.pre[n_win];
        const int lo = find(sm.pre_u, n_win, u);
        const int per_head = (sm.len[lo] + kDecodeTile - 1) / kDecodeTile;
        if (uncut) return sm.pre[lo] + (u - sm.pre_u[lo]) * per_head;
        const int head = quotient(u - sm.pre_u[lo], per_head + kSegWeight);
        const int r = (int)(u - sm.pre_u[lo] - (long long)head * (per_head + kSegWeight));
        return sm.pre[lo] + (long long)head * per_head + min(r, per_head);
    };
    const int n_cta = (int)min((long long)gridDim.x, uncut ? total.units / (LIST ? list_tiles : 1) : total.tiles);
    if ((int)blockIdx.x >= n_cta) {
        if (tid == 0) a.open[blockIdx.x].n_more = 0;
        return;
    }
    const long long my_a = cta_first(total.units, n_cta, blockIdx.x), my_b = cta_first(total.units, n_cta, blockIdx.x + 1);

    uint32_t joins = 0;
    // the consuming warps have come this far; bounded, like every wait
    auto join = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.joined));
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.joined), joins++ & 1u, abort_flag));
    };
    int done = 0, segs = 0;                                // tiles and segments of earlier windows: slots and phases
    long long base = 0;                                    // units before the window
    OpenSegment open{0, 0, 0, 0, 1.f};                     // the query warp's
    for (int w = 0; w < n_windows; ++w) {
        const Sums in_window = (w == 0) ? first_total : load_window(w);
        const long long ua = max(my_a - base, 0LL), ub = min(my_b - base, in_window.units);
        const int n_win = LIST ? 0 : min(kWindow, v.n_seq - w * kWindow);
        const long long A = ua < ub ? tiles_before(ua, n_win) : 0, B = ua < ub ? tiles_before(ub, n_win) : 0;
        const int count = (int)(B - A);

        // the sequence of packed row t; false where there is none
        auto seq_of = [&](long long t, int* s, SeqSpan* sp, int* err) -> bool {
            int lo = 0, n = v.n_seq;
            while (n > 1) {                                // the last that starts at or before t
                const int h = n / 2;
                if ((at_hand ? sm.first[lo + h] : a.tok_off[lo + h]) <= t) {
                    lo += h;
                    n -= h;
                } else {
                    n = h;
                }
            }
            *s = lo;
            if (at_hand) {                                 // a sequence that contradicts itself has no tokens here
                sp->t0 = sm.t0[lo];
                sp->n_new = sm.n_new[lo];
                sp->len = sm.len[lo];
            } else if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, lo, sp, err)) {
                return false;
            }
            return t >= sp->t0 && t < sp->t0 + sp->n_new;
        };
        if (warp == kWarps) {
            // ------------------------------------------------------------------ loader: a lane per tile
            // as many at a time as there are slots: two lanes waiting for the same slot, a phase apart, could not
            // tell by its parity whose turn it is
            for (int i0 = 0; i0 < count; i0 += kSlots) {
                if (a.stall && done + i0 >= (a.stall - 1) * kSlots) break;
                const int i = lane < kSlots ? i0 + lane : count;
                TileInfo ti;
                int row[2] = {0, 0}, rows[2] = {0, 0};
                int64_t slabs[2] = {-1, -1};
                ti.key[0] = ti.key[1] = 0;
                int32_t listed[2] = {-1, -1};              // asked for before the sequence is looked for
                if (LIST && i < count) {
                    const long long g = A + i, seg = g / list_tiles;
                    const int at = (int)(g - seg * list_tiles), li = pairs ? 2 * at : at / per_page;
                    listed[0] = a.sel[seg * a.k + li];
                    if (pairs && li + 1 < a.k) listed[1] = a.sel[seg * a.k + li + 1];
                }
                auto look_up = [&]() {
                    const long long g = A + i;
                    int s, head, seen, at;                 // at: the tile's number in its segment
                    long long seg = 0;
                    if (LIST) {
                        seg = g / list_tiles;
                        at = (int)(g - seg * list_tiles);
                        const long long t = seg / v.hkv;
                        head = (int)(seg - t * v.hkv);
                        SeqSpan sp;
                        if (!seq_of(t, &s, &sp, a.err)) return;
                        seen = sp.len - sp.n_new + (int)(t - sp.t0) + 1;
                    } else {
                        const int lo = find(sm.pre, n_win, g);
                        s = w * kWindow + lo;
                        const int per_head = (sm.len[lo] + kDecodeTile - 1) / kDecodeTile;
                        const long long in_seq = g - sm.pre[lo];
                        const int nth = quotient(in_seq, per_head);
                        at = (int)(in_seq - (long long)nth * per_head);
                        int64_t t0;
                        int n_new;
                        block_of(lo, nth, &head, &t0, &n_new, &seen);
                    }
                    const int n_pages = (seen + page - 1) >> v.shift;
                    const int32_t* table = v.table + (int64_t)s * v.max_pages;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        int p, row0 = 0;
                        if (h == 1 && !pairs) {            // the other half of the same page's tile
                            if (rows[0] == 0) break;
                            ti.key[1] = ti.key[0] + 16;
                            rows[1] = max(0, min(16, seen - ti.key[1]));
                            break;
                        }
                        if (LIST) {
                            p = listed[h];
                            if (!pairs) row0 = (at - at / per_page * per_page) * kDecodeTile;
                            if (p == -1) continue;
                            if (p < 0 || p >= n_pages) {
                                record_device_error(a.err, MSA_DEV_BAD_INDEX);
                                continue;
                            }
                        } else {
                            const int key = at * kDecodeTile + 16 * h;
                            if (key >= seen) break;
                            p = key >> v.shift;
                            row0 = key & (page - 1);
                        }
                        const int32_t pid = table[p];
                        if (pid < 0 || pid >= v.n_pages) {
                            record_device_error(a.err, MSA_DEV_BAD_INDEX);
                            continue;
                        }
                        const int64_t slab = (int64_t)pid * 2 * v.hkv + head;
                        ti.key[h] = (p << v.shift) + row0;
                        rows[h] = max(0, min(16, seen - ti.key[h]));
                        row[h] = (int)(slab * page) + row0;
                        slabs[h] = slab;
                    }
                };
                if (i < count) look_up();
                ti.rows = rows[0] + 256 * rows[1];
                float sk[2] = {1.f, 1.f}, sv[2] = {1.f, 1.f};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (slabs[h] >= 0) {                   // used after the copies have been issued
                        sk[h] = v.scales[slabs[h]];
                        sv[h] = v.scales[slabs[h] + v.hkv];
                    }
                // each lane brings its tile in as soon as the slot is free
                const int n = done + i, slot = n % kSlots;      // distinct for the lanes with a tile
                const uint32_t full = smem_u32(&sm.full[slot]), empty = smem_u32(&sm.empty[slot]), dst = smem_u32(sm.ring[slot]);
                bool pending = i < count;
                const uint64_t t_start = globaltimer();
                for (uint32_t polls = 0; __any_sync(0xffffffffu, pending); ++polls) {
                    if (pending && mbar_test(empty, ((uint32_t)(n / kSlots) & 1u) ^ 1u)) {
                        sm.last[slot] = n / kSlots + 1;
                        // a box is 32 rows, or where pages have 16, 16
                        const bool one = rows[0] > 0, two = pairs && rows[1] > 0;
                        if (one) {
                            tma_load_2d(dst, &tm, 0, row[0], full);
                            tma_load_2d(dst + kTileBytes / 2, &tm, 0, row[0] + v.hkv * page, full);
                        }
                        if (two) {
                            tma_load_2d(dst + 2048, &tm, 0, row[1], full);
                            tma_load_2d(dst + kTileBytes / 2 + 2048, &tm, 0, row[1] + v.hkv * page, full);
                        }
                        if (!pairs) {
                            sk[1] = sk[0];
                            sv[1] = sv[0];
                        }
                        if (rows[0] == 0) sv[0] = sv[1];
                        if (rows[1] == 0) sv[1] = sv[0];
                        ti.sk[0] = sk[0];
                        ti.sk[1] = sk[1];
                        ti.vs = fmaxf(sv[0], sv[1]);
                        ti.fac[0] = sv[0] / ti.vs;
                        ti.fac[1] = sv[1] / ti.vs;
                        sm.info[slot] = ti;
                        // the arrival, without which the phase cannot end however many bytes are in
                        mbar_expect_tx(full, (one ? (pairs ? kTileBytes / 2 : kTileBytes) : 0) + (two ? kTileBytes / 2 : 0));
                        pending = false;
                    }
                    if ((polls & 63) == 63) {
                        if (lane == 0 && globaltimer() - t_start > kWaitNs) *abort_flag = 1;
                        if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
                    }
                }
                if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            }
        } else if (warp == kWarps + 1) {
            // ------------------------------------------------------------------ queries: a segment ahead
            const int r = lane >> 2, c = lane & 3;
            int n_seg = segs;
            for (long long g0 = A; g0 < B; ++n_seg) {
                Segment sg;
                long long seg_a, seg_b;
                if (LIST) {
                    const long long seg = g0 / list_tiles;
                    sg.t0 = seg / v.hkv;
                    sg.head = (int)(seg - sg.t0 * v.hkv);
                    seg_a = seg * list_tiles;
                    seg_b = seg_a + list_tiles;
                    int s;
                    SeqSpan sp;
                    const bool live = seq_of(sg.t0, &s, &sp, nullptr);
                    sg.len = sp.len - sp.n_new + (int)(sg.t0 - sp.t0) + 1;
                    sg.n_new = live ? 1 : 0;
                } else {
                    const int lo = find(sm.pre, n_win, g0);
                    const int per_head = (sm.len[lo] + kDecodeTile - 1) / kDecodeTile;
                    const int nth = quotient(g0 - sm.pre[lo], per_head);
                    block_of(lo, nth, &sg.head, &sg.t0, &sg.n_new, &sg.len);
                    seg_a = sm.pre[lo] + (long long)nth * per_head;
                    seg_b = seg_a + per_head;
                    if (seg_a == g0 && seg_b > B) {        // it goes on in other blocks: what the combine pass needs to know
                        const long long u = base + sm.pre_u[lo] + (long long)nth * (per_head + kSegWeight) + per_head - 1;
                        open = OpenSegment{sg.t0, sg.head, sg.n_new * G, cta_of_tile(total.units, n_cta, u) - (int)blockIdx.x, 1.f};
                    }
                }
                if (LIST && sg.n_new && seg_a == g0 && seg_b > B)
                    open = OpenSegment{sg.t0, sg.head, G, cta_of_tile(total.units, n_cta, seg_b - 1) - (int)blockIdx.x, 1.f};
                const long long g1 = min(B, seg_b);
                sg.n_rows = sg.n_new * G;
                sg.end = (int)(g1 - A);
                sg.starts = seg_a == g0;
                sg.whole = sg.starts && seg_b == g1;

                // the thread's part of Q^T: row n = r, elements 32 c .. 32 c + 31; the softmax scale's sign is Q's
                uint4 x[4];
                uint32_t qh[8], ql[8];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = make_uint4(0, 0, 0, 0);
                if (r < sg.n_rows) {
                    const uint4* src = reinterpret_cast<const uint4*>(
                        a.q + ((sg.t0 + (r >> gs)) * hq + sg.head * G + (r & (G - 1))) * kPagedD + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = src[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // s = 2^e with top <= 448 s; the range keeps s and 1 / s normal, and the logit factor at 2^-76 or more: times
                // any scale of K it is not 0, which would make a NaN of a masked place (zero queries or softmax scales; what
                // smaller queries lose moves no logit by 2^-20)
                const uint32_t ub = __float_as_uint(top);
                const int e_min = max(-100, -76 - exponent_of(a.scale_log2e));
                const int e = max(e_min, min(120, (int)(ub >> 23) - 127 - 8 + ((ub & 0x7FFFFFu) > 0x600000u ? 1 : 0)));
                const float inv = a.scale_log2e < 0.f ? -pow2f(-e) : pow2f(-e);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t h0, l0, h1, l1;
                        split_e4m3(__uint_as_float(u[2 * j] << 16) * inv, __uint_as_float(u[2 * j] & 0xFFFF0000u) * inv, &h0, &l0);
                        split_e4m3(__uint_as_float(u[2 * j + 1] << 16) * inv, __uint_as_float(u[2 * j + 1] & 0xFFFF0000u) * inv,
                                   &h1, &l1);
                        qh[2 * i + j] = h0 | (h1 << 16);
                        ql[2 * i + j] = l0 | (l1 << 16);
                    }
                }
                const float f = ub >= 0x7F800000u ? __int_as_float(0x7FFFFFFF) : fmaxf(fabsf(a.scale_log2e) * pow2f(e), pow2f(-76));
                const int at = n_seg % kSegs;
                if (!__all_sync(0xffffffffu,
                                mbar_wait(smem_u32(&sm.seg_empty[at]), ((uint32_t)(n_seg / kSegs) & 1u) ^ 1u, abort_flag)))
                    break;
                sm.q[at][0][lane] = make_uint4(qh[0], qh[1], qh[2], qh[3]);
                sm.q[at][1][lane] = make_uint4(qh[4], qh[5], qh[6], qh[7]);
                sm.q[at][2][lane] = make_uint4(ql[0], ql[1], ql[2], ql[3]);
                sm.q[at][3][lane] = make_uint4(ql[4], ql[5], ql[6], ql[7]);
                if (c == 0) sm.f[at][r] = f;
                if (lane == 0) sm.seg[at] = sg;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.seg_full[at]));
                g0 = g1;
            }
            segs = n_seg;
        } else {
            // ------------------------------------------------------------------ segment by segment
            const int r = lane >> 2, c = lane & 3;         // the thread's place in a fragment
            // its pieces of K (rows r and r + 8, pieces 2 c and 2 c + 1) and V (piece r of keys 2 c + {0, 8, 1, 9}): piece i
            // of row y lies at i ^ y % 8
            const int k_at = r * 128 + (((2 * c) ^ r) << 4);
            const int v_at0 = kTileBytes / 2 + 2 * c * 128 + ((r ^ (2 * c)) << 4);
            const int v_at1 = kTileBytes / 2 + (2 * c + 1) * 128 + ((r ^ (2 * c + 1)) << 4);
            // The warp's tiles are those whose number (over all windows) leaves it as remainder, and so are its slots: with
            // slots that passed from warp to warp, one that runs ahead could not tell a phase from the next but one.
            int taken = ((warp - done) % kWarps + kWarps) % kWarps;
            for (int end = 0; end < count;) {
                const int at = segs % kSegs;
                const bool ready = mbar_wait(smem_u32(&sm.seg_full[at]), (uint32_t)(segs / kSegs) & 1u, abort_flag);
                if (__any_sync(0xffffffffu, !ready)) break;
                ++segs;
                const int64_t t0 = sm.seg[at].t0;
                const int head = sm.seg[at].head, n_rows = sm.seg[at].n_rows, len = sm.seg[at].len, n_new = sm.seg[at].n_new;
                const int whole = sm.seg[at].whole, starts = sm.seg[at].starts;
                end = sm.seg[at].end;
                uint32_t qh[8], ql[8];
                {
                    const uint4 x = sm.q[at][0][lane], y = sm.q[at][1][lane], z = sm.q[at][2][lane], u = sm.q[at][3][lane];
                    qh[0] = x.x, qh[1] = x.y, qh[2] = x.z, qh[3] = x.w, qh[4] = y.x, qh[5] = y.y, qh[6] = y.z, qh[7] = y.w;
                    ql[0] = z.x, ql[1] = z.y, ql[2] = z.z, ql[3] = z.w, ql[4] = u.x, ql[5] = u.y, ql[6] = u.z, ql[7] = u.w;
                }
                const float f0 = sm.f[at][2 * c], f1 = sm.f[at][2 * c + 1];    // logit factors of rows 2 c and 2 c + 1
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.seg_empty[at]));
                const int seen0 = 2 * c < n_rows ? len - n_new + ((2 * c) >> gs) + 1 : 0;
                const int seen1 = 2 * c + 1 < n_rows ? len - n_new + ((2 * c + 1) >> gs) + 1 : 0;
                const int seen_all = len - n_new + 1;      // keys that every row sees

                float o[8][4], m0 = ninf, m1 = ninf, l0 = 0.f, l1 = 0.f, e0 = 0.f, e1 = 0.f;   // e: roundings of l
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

                for (; taken < end; taken += kWarps) {
                    const int n = done + taken, slot = n % kSlots;
                    const bool ok = __all_sync(
                        0xffffffffu, mbar_wait(smem_u32(&sm.full[slot]), (uint32_t)(n / kSlots) & 1u, abort_flag));
                    const TileInfo t = sm.info[slot];
                    if (ok && t.rows) {
                        const uint8_t* tile = sm.ring[slot];
                        // S^T: keys r and r + 8 of each half, rows 2 c and 2 c + 1
                        float s[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint4 x = *reinterpret_cast<const uint4*>(tile + 2048 * h + (k_at ^ (16 * i)));
                                const uint4 y = *reinterpret_cast<const uint4*>(tile + 2048 * h + 1024 + (k_at ^ (16 * i)));
                                if (i == 0) mma_e4m3_16832_first(s[h], x.x, y.x, x.y, y.y, qh[0], qh[1]);
                                else mma_e4m3_16832(s[h], x.x, y.x, x.y, y.y, qh[4], qh[5]);
                                mma_e4m3_16832(s[h], x.z, y.z, x.w, y.w, qh[4 * i + 2], qh[4 * i + 3]);
                                mma_e4m3_16832(s[h], x.x, y.x, x.y, y.y, ql[4 * i], ql[4 * i + 1]);
                                mma_e4m3_16832(s[h], x.z, y.z, x.w, y.w, ql[4 * i + 2], ql[4 * i + 3]);
                            }
                        }
                        uint4 w8[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w8[i] = *reinterpret_cast<const uint4*>(tile + (i >> 2) * 2048 + (i & 1) * 1024 + ((i >> 1) & 1 ? v_at1 : v_at0));
                        if (t.rows != kFull || max(t.key[0], t.key[1]) + 16 > seen_all) {
                            // keys that a row does not see, and places without a key, where anything may stand
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int rows = h ? t.rows >> 8 : t.rows & 255;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int y = r + 8 * (i >> 1);
                                    if (y >= rows || t.key[h] + y >= ((i & 1) ? seen1 : seen0)) s[h][i] = ninf;
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (2 * c + 8 * (i & 1) + (i >> 1) >= rows) w8[4 * h + i] = make_uint4(0, 0, 0, 0);
                            }
                        }
                        // halves whose scales of V lie far apart go one after the other, each against its own maximum
                        const bool apart = fminf(t.fac[0], t.fac[1]) < 0.0625f;
#pragma unroll 1
                        for (int pass = 0; pass < (apart ? 2 : 1); ++pass) {
                            float fac[2] = {t.fac[0], t.fac[1]}, vs = t.vs;
                            float y[2][4];
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int i = 0; i < 4; ++i) y[h][i] = s[h][i];
                            if (apart) {
                                vs *= fac[pass];
                                fac[0] = fac[1] = 1.f;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    if (pass == 0) y[1][i] = ninf;
                                    else y[0][i] = ninf;
                                }
                            }
                            const float k0[2] = {f0 * t.sk[0], f0 * t.sk[1]}, k1[2] = {f1 * t.sk[0], f1 * t.sk[1]};
                            float ma = fmaxf(fmaxf(y[0][0], y[0][2]) * k0[0], fmaxf(y[1][0], y[1][2]) * k0[1]);
                            float mb = fmaxf(fmaxf(y[0][1], y[0][3]) * k1[0], fmaxf(y[1][1], y[1][3]) * k1[1]);
#pragma unroll
                            for (int sh = 4; sh <= 16; sh <<= 1) {
                                ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, sh));
                                mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, sh));
                            }
                            if (__any_sync(0xffffffffu, ma > m0 + kSlack || mb > m1 + kSlack)) {
                                const float na = fmaxf(ma, m0), nb = fmaxf(mb, m1);
                                const float a0 = m0 == na ? 1.f : ex2(m0 - na), a1 = m1 == nb ? 1.f : ex2(m1 - nb);
                                m0 = na;
                                m1 = nb;
                                l0 *= a0;
                                e0 *= a0;
                                l1 *= a1;
                                e1 *= a1;
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    o[i][0] *= a0;
                                    o[i][1] *= a1;
                                    o[i][2] *= a0;
                                    o[i][3] *= a1;
                                }
                            }
                            // P times 2^8, and the weight of this tile's product
                            const float na = ma == ninf ? 0.f : 8.f - ma, nb = mb == ninf ? 0.f : 8.f - mb;
                            float wa = ma == ninf ? 0.f : ex2(-na - m0), wb = mb == ninf ? 0.f : ex2(-nb - m1);
                            uint32_t bh[2], bl[2];
                            float ta = 0.f, tb = 0.f;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float p0 = ex2(fmaf(y[h][0], k0[h], na)), p1 = ex2(fmaf(y[h][1], k1[h], nb));
                                const float p2 = ex2(fmaf(y[h][2], k0[h], na)), p3 = ex2(fmaf(y[h][3], k1[h], nb));
                                ta += p0 + p2;
                                tb += p1 + p3;
                                uint32_t ha, la, hb, lb;
                                split_e4m3<__NV_E5M2>(p0 * fac[h], p2 * fac[h], &ha, &la);
                                split_e4m3<__NV_E5M2>(p1 * fac[h], p3 * fac[h], &hb, &lb);
                                bh[h] = transpose8x8(__byte_perm(ha, hb, 0x5410));
                                bl[h] = transpose8x8(__byte_perm(la, lb, 0x5410));
                            }
                            {
                                const float d0 = fmaf(ta, wa, -e0), d1 = fmaf(tb, wb, -e1);
                                const float s0 = l0 + d0, s1 = l1 + d1;
                                e0 = (s0 - l0) - d0;
                                e1 = (s1 - l1) - d1;
                                l0 = s0;
                                l1 = s1;
                            }
                            wa *= vs;
                            wb *= vs;
                            // four elements of d of four keys are a 4 x 4 block of bytes; row r of the fragment of tile i is
                            // d = 16 r + 2 i, row r + 8 the next
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t f[2][4];
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const uint32_t u0 = (&w8[4 * h].x)[i], u1 = (&w8[4 * h + 1].x)[i];
                                    const uint32_t u2 = (&w8[4 * h + 2].x)[i], u3 = (&w8[4 * h + 3].x)[i];
                                    const uint32_t a0 = __byte_perm(u0, u1, 0x5140), a1 = __byte_perm(u2, u3, 0x5140);
                                    const uint32_t a2 = __byte_perm(u0, u1, 0x7362), a3 = __byte_perm(u2, u3, 0x7362);
                                    f[h][0] = __byte_perm(a0, a1, 0x5410);
                                    f[h][1] = __byte_perm(a0, a1, 0x7632);
                                    f[h][2] = __byte_perm(a2, a3, 0x5410);
                                    f[h][3] = __byte_perm(a2, a3, 0x7632);
                                }
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    float d[4];
                                    mma_e4m3_16832_first(d, f[0][2 * z], f[0][2 * z + 1], f[1][2 * z], f[1][2 * z + 1], bh[0], bh[1]);
                                    mma_e4m3_e5m2_16832(d, f[0][2 * z], f[0][2 * z + 1], f[1][2 * z], f[1][2 * z + 1], bl[0], bl[1]);
                                    float* oo = o[2 * i + z];
                                    oo[0] = fmaf(d[0], wa, oo[0]);
                                    oo[1] = fmaf(d[1], wb, oo[1]);
                                    oo[2] = fmaf(d[2], wa, oo[2]);
                                    oo[3] = fmaf(d[3], wb, oo[3]);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
                }

                // join the warps: row n of the segment by warp n, 32 columns at a time
#pragma unroll
                for (int sh = 4; sh <= 16; sh <<= 1) {
                    l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
                    l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
                }
                if (!join()) break;                        // the last segment's values have been read
                if (lane < 4) {
                    sm.ml[warp][2 * c] = make_float2(m0, l0);
                    sm.ml[warp][2 * c + 1] = make_float2(m1, l1);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)            // d = 16 r + 4 i
                        sm.o[warp][2 * c + j][(4 * r + i) ^ c] =
                            make_float4(o[2 * i][j], o[2 * i][2 + j], o[2 * i + 1][j], o[2 * i + 1][2 + j]);
                if (!join()) break;
                if (warp < n_rows) {
                    // lane i: warp i's maximum, sum and weight
                    const float2 ml = lane < kWarps ? sm.ml[lane][warp] : make_float2(ninf, 0.f);
                    float M = ml.x;
#pragma unroll
                    for (int sh = 8; sh >= 1; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, sh));
                    const float wt = ml.x == ninf ? 0.f : ex2(ml.x - M);
                    float L = ml.x == ninf ? ml.y : wt * ml.y;         // a sum without a maximum is 0 or NaN
#pragma unroll
                    for (int sh = 8; sh >= 1; sh >>= 1) L += __shfl_xor_sync(0xffffffffu, L, sh);
                    M = __shfl_sync(0xffffffffu, M, 0);
                    L = __shfl_sync(0xffffffffu, L, 0);
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) {
                        const float4 y = sm.o[i][warp][lane ^ (warp >> 1)];
                        const float z = __shfl_sync(0xffffffffu, wt, i);
                        x.x = fmaf(z, y.x, x.x);
                        x.y = fmaf(z, y.y, x.y);
                        x.z = fmaf(z, y.z, x.z);
                        x.w = fmaf(z, y.w, x.w);
                    }
                    if (whole) {
                        const int64_t row = (t0 + (warp >> gs)) * hq + head * G + (warp & (G - 1));
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        uint2 u;
                        u.x = pack_bf16(x.x * inv, x.y * inv);
                        u.y = pack_bf16(x.z * inv, x.w * inv);
                        reinterpret_cast<uint2*>(a.out + row * kPagedD)[lane] = u;
                        if (a.lse && lane == 0) a.lse[row] = L == 0.f ? ninf : (M + log2f(L)) * 0.6931471805599453f;
                    } else {
                        const int64_t row = ((int64_t)blockIdx.x * 2 + starts) * a.rows + warp;
                        reinterpret_cast<float4*>(a.part_o + row * kPagedD)[lane] = x;
                        if (lane == 0) a.part_ml[row] = make_float2(M, L);
                    }
                }
            }
        }
        done += count;
        base += in_window.units;
        __syncthreads();
    }
    if (tid == kConsumers + 32) a.open[blockIdx.x] = open;
    if (*abort_flag) {
        if (tid == 0) record_device_error(a.err, MSA_DEV_WAIT_TIMEOUT);
        // leave no copy in flight: each slot's last load
        if (tid < kSlots && sm.last[tid] > 0) mbar_wait_drain(smem_u32(&sm.full[tid]), (uint32_t)(sm.last[tid] - 1) & 1u);
    }
}

}  // namespace

msa_status launch_paged_decode(const PagedAttnArgs& a, int grid, cudaStream_t s) {
    constexpr int smem = (int)sizeof(DecodeSmem) + 1024;
    static_assert(smem <= 232448, "shared memory");
    static std::mutex mu;
    static bool opted[64] = {false};
    int dev = 0;
    MSA_CUDA_TRY(cudaGetDevice(&dev));
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64 || !opted[dev]) {
            MSA_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
            MSA_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
            if (dev >= 0 && dev < 64) opted[dev] = true;
        }
    }
    // the pages as rows of 128 bytes (64 two-byte elements); a box is a tile of keys or of values, or half of one
    CUtensorMap tm{};
    const uint64_t dims[2] = {64, (uint64_t)(a.v.n_pages * 2 * a.v.hkv * a.v.page)};
    const uint64_t strides[1] = {kPagedD};
    const uint32_t box[2] = {64, (uint32_t)std::min(a.v.page, kDecodeTile)};
    MSA_RETURN_IF(make_tensor_map_bf16(&tm, a.v.pages, 2, dims, strides, box));
    MSA_CUDA_TRY(launch_early(a.sel ? paged_decode_kernel<true> : paged_decode_kernel<false>, dim3((unsigned)grid), kThreads,
                              smem, s, tm, a));
    return MSA_OK;
}

}  // namespace msa
