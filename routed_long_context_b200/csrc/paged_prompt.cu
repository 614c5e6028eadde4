// Attention of many query rows over a paged 8-bit cache, on tcgen05 tensor cores.
//
//   out = softmax(scale q . K) V  for blocks of 128 or 256 rows (token, query head) of one kv head.
// Rows are TMEM lanes. Per tile of 128 keys and 128 rows:
//   S = Qhi K^T + Qlo K^T     tcgen05.mma f8f6f4, M = N = 128, K = 128 each, straight from the cache's bytes. A query row
//                             is split as q = s (hi + lo), s a power of two that brings its largest to 224..448 and hi
//                             and lo e4m3: eight significant bits, which is all that bf16 has, down to 2^-11 of the
//                             row's largest; what lies below is off by at most 2^-10 s. Two 8-bit products cost what
//                             one 16-bit product would, and K needs no conversion.
//   P = 2^(S f - m)           a thread per row; f carries the softmax scale, s and the page's scale of K (a power of two
//                             per 16 columns at least). m is a stale maximum: P is rounded to bf16, whose exponent has
//                             room, so m moves only when a tile's sum shows a logit more than 2^15 above it, and no
//                             maximum is taken otherwise. P replaces S in TMEM.
//   O += P V                  tcgen05.mma f16 (bf16), A = P from TMEM, B = V as bf16 (exact: e4m3 times its scale), put
//                             into shared memory by four warps of their own.
// Two warpgroups take the two row blocks of 256 rows in turns (their products and exponentials overlap), or, of a
// 128-row block, the even and the odd key tiles, joined at the end.
// The products cost 8 * 128^3 flops a tile and row block, 1,024 cycles at the tensor peak; 128 * 128 exponentials take
// as long on the special-function units: neither can take less, and neither bounds it. Measured, a tile of both row
// blocks takes 4,200 cycles: a warpgroup's exponentials and their reading and writing of TMEM 2,100, its products 1,300
// (shared memory feeds Q K^T no faster), and what passes between them, one after the other: S and P share a place in
// TMEM, and two row blocks do not fill the gaps (1.6 instructions issued a cycle, the tensor pipe active for 48 %).
// 2,000 tokens of 32 heads over 18,000: 593 to 621 us on four GPUs, 897 to 940 TFLOP/s. Not faster: an issuer of products
// for each warpgroup (764 us; in strict turns 655), steps of 64 keys with S ahead (738), part of the exponentials by
// arithmetic (641 and more), waits by one lane of a warp (741).
// With few tiles to a block, what starts and ends a segment is most of it: 8 sequences of up to 32 tokens over up to
// 8,096 take 42 us (before launches overlapped 45, and 57 where a segment's cost is left out of the blocks' shares).
//
// Roles of the 512 threads: warp 0 loads pages by TMA (128-byte swizzle, K three tiles deep, V two), warp 1 issues the
// products, warps 4..11 run the softmax, warps 12..15 convert V. Every wait is bounded; when one runs out the block
// records MSA_DEV_WAIT_TIMEOUT and leaves in order.
#include <algorithm>
#include <mutex>

#include "kernels.cuh"
#include "mma.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kKT = 128;                                   // keys per tile
constexpr int kRowsTile = 128;                             // MMA M
constexpr int kKStages = 3, kVStages = 2, kV16Stages = 2, kInfo = 8;
constexpr int kWin = kPromptSeqs;                          // sequences of a launch, a thread each
static_assert(kWin == kThreads, "a thread per sequence");
constexpr float kTrigger = 32768.f;                        // a tile's sum above it moves the reference maximum
constexpr float kSlack = 8.f;                              // log2 of how far logits may lie above the reference

constexpr float kUnit = 1152921504606846976.f;             // 2^60, the unit in which O is kept
// Tiles whose products are summed up in one place. The tensor cores cut a sum off instead of rounding it, so each of a
// tile's 8 steps may lose 2^-23 of O, always toward zero: 2^-11 at most over 512 tiles, but 8 % measured over the 113,000
// that a block has of 2^31 keys, with values of one sign. Longer runs are added up in the workspace, in fp32 rounded to
// nearest; no call over up to 65,536 keys has one, and 2,000 tokens over 18,000 take what they took (605 us, 603 before).
constexpr int kChain = 512;

constexpr int kBytes8 = kKT * kPagedD;                     // a tile of K or V in 8 bits: 16 KB
constexpr int kBytes16 = 2 * kBytes8;

struct PromptSmem {
    uint8_t q[2][2][kRowsTile * kPagedD];                  // [row block][hi, lo]
    uint8_t k[kKStages][kBytes8];
    uint8_t v8[kVStages][kBytes8];
    uint8_t v16[kV16Stages][kBytes16];                     // [d half][key][64]
    // per 16 keys of a tile: scale of K (0: no page there), 60 + the exponent of V's, 2^-that
    alignas(16) float sk[kInfo][8], ev[kInfo][8], iv[kInfo][8];
    uint64_t k_full[kKStages], k_empty[kKStages], v8_full[kVStages], v8_empty[kVStages];
    uint64_t v16_full[kV16Stages], v16_empty[kV16Stages];
    uint64_t q_full[2], s_full[2], p_full[2], o_done[2], drain;
    uint32_t tmem;
    int abort_flag, stop;
    long long pre[kWin + 1];                               // units before each sequence: a segment's tiles and kSegWeight more
    int64_t t0[kWin];
    int n_new[kWin], len[kWin];
    long long scan[kThreads / 32];
    float2 ml[2][kRowsTile];
    float fr[2][kRowsTile];
};

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// A from TMEM
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 TMEM columns on their way into registers, which may be used after tmem_wait32
__device__ __forceinline__ void tmem_issue32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
// two fp32 values in a register pair
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ uint64_t pair_u(uint32_t lo, uint32_t hi) { return (uint64_t)lo | ((uint64_t)hi << 32); }
__device__ __forceinline__ float first(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float second(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st16_u32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32_u32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// One run of key tiles of one segment: the block's share of it, or kChain tiles of that.
struct Piece {
    int64_t t0;            // first packed row of the block's tokens
    int head, rows;        // kv head, query rows
    int seen0;             // keys that the block's first token sees
    int len;               // keys of the sequence
    int s;                 // sequence
    int k0, n;             // first key tile, number of them
    int where;             // kStarts, kEnds: the block's share holds the segment's first tile, its last; kFirst, kLast: run of it
    long long seg_end;     // one past the unit of the segment's last tile
    static constexpr int kStarts = 1, kEnds = 2, kFirst = 4, kLast = 8;
};

__device__ __forceinline__ int seg_tiles(int base, int n_new, int tpb, int rb) {
    return (base + min(n_new, (rb + 1) * tpb) + kKT - 1) / kKT;
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) paged_prompt_kernel(const __grid_constant__ CUtensorMap tm,
                                                                   const PagedAttnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    PromptSmem& sm = *reinterpret_cast<PromptSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const PagedView& v = a.v;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.G, gs = 31 - __clz(G), hq = v.hkv * G;
    const int tpb = (SPLIT ? kRowsTile : 2 * kRowsTile) / G;       // tokens of a row block
    const float ninf = -INFINITY;
    volatile int* abort_flag = &sm.abort_flag;
    next_may_launch();
    if (tid == 32) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm)) : "memory");

    if (tid == 0) {
        for (int i = 0; i < kKStages; ++i) mbar_init(smem_u32(&sm.k_full[i]), 1), mbar_init(smem_u32(&sm.k_empty[i]), 1);
        for (int i = 0; i < kVStages; ++i) mbar_init(smem_u32(&sm.v8_full[i]), 1), mbar_init(smem_u32(&sm.v8_empty[i]), 128);
        for (int i = 0; i < kV16Stages; ++i)
            mbar_init(smem_u32(&sm.v16_full[i]), 128), mbar_init(smem_u32(&sm.v16_empty[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.q_full[i]), SPLIT ? 256 : 128);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.p_full[i]), 128);
            mbar_init(smem_u32(&sm.o_done[i]), 1);
        }
        mbar_init(smem_u32(&sm.drain), 1);
        sm.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }

    wait_for_earlier();
    const bool alloc = warp == 1;
    if (alloc) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }

    // units of all sequences: a thread per sequence
    long long total = 0;
    {
        SeqSpan sp{0, 0, 0};
        if (tid < v.n_seq) seq_span(v, a.tok_off, a.n_tok, a.max_new, tid, &sp, blockIdx.x == 0 ? a.err : nullptr);
        long long x = 0;
        for (int rb = 0; rb * tpb < sp.n_new; ++rb) x += seg_tiles(sp.len - sp.n_new, sp.n_new, tpb, rb) + kSegWeight;
        x *= v.hkv;
        long long up = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += y;
        }
        sm.t0[tid] = sp.t0;
        sm.n_new[tid] = sp.n_new;
        sm.len[tid] = sp.len;
        if (lane == 31) sm.scan[warp] = up;
        __syncthreads();
        long long before = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += sm.scan[i];
            total += sm.scan[i];
        }
        sm.pre[tid + 1] = before + up;
        if (tid == 0) sm.pre[0] = 0;
    }
    // A block for each tile with its segment's weight, rounded up: of a call with few tiles a block's share may still be a
    // weight alone, and the block finds no piece in it (a segment of 2 tiles: 10 units, two blocks of 5).
    constexpr int kMinUnits = 1 + kSegWeight;
    const int n_cta = (int)min((long long)gridDim.x, (total + kMinUnits - 1) / kMinUnits);
    if ((int)blockIdx.x >= n_cta) {
        if (tid == 0) a.open[blockIdx.x].n_more = 0;
        if (alloc) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem) : "memory");
        return;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;                         // S (and P) of warpgroup w at 128 w, O at 256 + 128 w
    const long long A = cta_first(total, n_cta, blockIdx.x), B = cta_first(total, n_cta, blockIdx.x + 1);

    // every role's own counts, which give the ring stages and phases
    int cnt = 0;                                           // tiles of earlier pieces
    int pieces = 0;                                        // pieces (softmax: those in which the warpgroup had a tile)
    int loading_k = 0, loading_v = 0;                      // loader: tiles under way or in
    // the pieces of units [A, B), in order; every role walks them for itself
    auto walk = [&](auto&& body) {
        int lo = 0, n = v.n_seq;
        while (n > 1) {
            const int h = n / 2;
            if (sm.pre[lo + h] <= A) {
                lo += h;
                n -= h;
            } else {
                n = h;
            }
        }
        int rb = 0, head = 0;
        int n_new = sm.n_new[lo], len = sm.len[lo];
        int tiles = seg_tiles(len - n_new, n_new, tpb, 0);
        long long start = sm.pre[lo];
        while (start + (long long)(tiles + kSegWeight) * v.hkv <= A) {
            start += (long long)(tiles + kSegWeight) * v.hkv;
            tiles = seg_tiles(len - n_new, n_new, tpb, ++rb);
        }
        head = (int)((A - start) / (tiles + kSegWeight));
        start += (long long)head * (tiles + kSegWeight);
        while (true) {
            Piece p;
            p.t0 = sm.t0[lo] + rb * tpb;
            p.head = head;
            p.rows = min(tpb, n_new - rb * tpb) * G;
            p.seen0 = len - n_new + rb * tpb + 1;
            p.len = len;
            p.s = lo;
            p.k0 = (int)min((long long)tiles, max(0LL, A - start));
            p.where = Piece::kFirst | (p.k0 == 0 ? Piece::kStarts : 0) | (B - start >= tiles ? Piece::kEnds : 0);
            p.seg_end = start + tiles;
            while (true) {
                const int left = (int)min((long long)tiles, B - start) - p.k0;
                if (left <= 0) break;
                p.n = min(kChain, left);
                if (left <= kChain) p.where |= Piece::kLast;
                if (!body(p)) return;
                p.k0 += kChain;
                p.where &= ~Piece::kFirst;
            }
            start += tiles + kSegWeight;
            if (start >= B) return;
            if (++head == v.hkv) {
                head = 0;
                if (++rb * tpb >= n_new) {
                    rb = 0;
                    do ++lo;
                    while (sm.n_new[lo] == 0);
                    n_new = sm.n_new[lo];
                    len = sm.len[lo];
                }
                tiles = seg_tiles(len - n_new, n_new, tpb, rb);
            }
        }
    };
    // 72 + 88 + 2 * 176 = 4 * 128 registers, what the block starts with
    if (warp < 4) {
        fewer_registers<72>();
        if (warp == 0) {
            // ------------------------------------------------------------------ loader
            // Lane 8 i + c looks up 16-key chunk c of tile i of a group of four tiles; the page ids of the group after
            // the next and the scales of the next are on their way while a group is issued.
            const int c = lane & 7, sub = lane >> 3;
            const int cps = v.shift - 4;                   // log2(chunks per page)
            walk([&](const Piece& p) -> bool {
                const int32_t* table = v.table + (int64_t)p.s * v.max_pages;
                auto exists = [&](int group) -> bool {
                    const int j = 4 * group + sub;
                    return j < p.n && (int64_t)(p.k0 + j) * kKT + 16 * c < p.len;
                };
                auto page_id = [&](int group) -> int32_t {
                    return exists(group) ? table[((p.k0 + 4 * group + sub) * 8 + c) >> cps] : -1;
                };
                auto scales = [&](int group, int32_t& id, float* sk, float* sv) {
                    *sk = 0.f;
                    *sv = 1.f;
                    if (id < 0 || id >= v.n_pages) {
                        if (exists(group)) record_device_error(a.err, MSA_DEV_BAD_INDEX);
                        id = -1;
                        return;
                    }
                    const int64_t slab = (int64_t)id * 2 * v.hkv + p.head;
                    *sk = v.scales[slab];
                    *sv = v.scales[slab + v.hkv];
                };
                int32_t id0 = page_id(0), id1 = page_id(1), id2;
                float sk0, sv0, sk1, sv1;
                scales(0, id0, &sk0, &sv0);
                for (int group = 0; 4 * group < p.n; ++group) {
                    id2 = page_id(group + 2);
                    scales(group + 1, id1, &sk1, &sv1);
                    for (int i = 0; i < 4 && 4 * group + i < p.n; ++i) {
                        const int n = cnt + 4 * group + i;
                        if (a.stall && n >= (a.stall - 1) * kKStages) return false;
                        const int ks = n % kKStages, vs = n % kVStages;
                        const bool here = sub == i;
                        const bool first = here && id0 >= 0 && (c & ((1 << cps) - 1)) == 0;
                        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, first)) * (uint32_t)(v.page * kPagedD);
                        const int row = first ? (int)(((int64_t)id0 * 2 * v.hkv + p.head) * v.page) : 0;
                        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.k_empty[ks]), ((uint32_t)(n / kKStages) & 1u) ^ 1u, abort_flag)))
                            return false;
                        if (here) {
                            const int e = exponent_of(sv0);
                            sm.sk[n % kInfo][c] = sk0;
                            sm.ev[n % kInfo][c] = (float)(60 + e);
                            sm.iv[n % kInfo][c] = pow2f(-60 - e);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_expect_tx(smem_u32(&sm.k_full[ks]), bytes);
                        __syncwarp();
                        if (first) tma_load_2d(smem_u32(sm.k[ks]) + c * 16 * kPagedD, &tm, 0, row, smem_u32(&sm.k_full[ks]));
                        loading_k = n + 1;
                        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sm.v8_empty[vs]), ((uint32_t)(n / kVStages) & 1u) ^ 1u, abort_flag)))
                            return false;
                        if (lane == 0) mbar_expect_tx(smem_u32(&sm.v8_full[vs]), bytes);
                        __syncwarp();
                        if (first)
                            tma_load_2d(smem_u32(sm.v8[vs]) + c * 16 * kPagedD, &tm, 0, row + v.hkv * v.page,
                                        smem_u32(&sm.v8_full[vs]));
                        loading_v = n + 1;
                    }
                    id0 = id1;
                    sk0 = sk1;
                    sv0 = sv1;
                    id1 = id2;
                }
                cnt += p.n;
                return true;
            });
        } else if (warp == 1) {
            // ------------------------------------------------------------------ products
            // One issuer for both warpgroups, in turns: that keeps one warpgroup's exponentials under the other's
            // products (with an issuer each they fall into step and wait together: 3,100 + 2,500 cycles a tile).
            // What a turn needs besides P is waited for before P is.
            if (lane == 0) {
                // f8f6f4: e4m3 x e4m3 -> fp32, both K-major; f16: bf16 x bf16 -> fp32, V MN-major
                const uint32_t idesc_s = (1u << 4) | ((uint32_t)(kKT >> 3) << 17) | ((uint32_t)(kRowsTile >> 4) << 24);
                const uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(kPagedD >> 3) << 17) |
                                         ((uint32_t)(kRowsTile >> 4) << 24);
                uint32_t turns = 0;                        // bit wg: parity of its P tiles
                walk([&](const Piece& p) -> bool {
                    auto wait_k = [&](int n) -> bool {
                        return mbar_wait(smem_u32(&sm.k_full[n % kKStages]), (uint32_t)(n / kKStages) & 1u, abort_flag);
                    };
                    auto issue_s = [&](int wg, int n, bool last) {
                        const uint64_t qd = sw128_desc(smem_u32(sm.q[SPLIT ? 0 : wg][0]));
                        const uint64_t kd = sw128_desc(smem_u32(sm.k[n % kKStages]));
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_f8(tmem + 128 * wg, qd + (uint64_t)(part * (kBytes8 >> 4) + kk * 2), kd + (uint64_t)(kk * 2),
                                        idesc_s, (part | kk) ? 1u : 0u);
                        umma_commit(smem_u32(&sm.s_full[wg]));
                        if (last) umma_commit(smem_u32(&sm.k_empty[n % kKStages]));
                    };
                    // turn i of the piece: tile i / 2 of warpgroup i % 2, or tile i, which warpgroup i % 2 has
                    const int n_turns = SPLIT ? p.n : 2 * p.n;
                    for (int i = 0; i < 2 && i < n_turns; ++i) {
                        if ((!SPLIT || i == 0) && !mbar_wait(smem_u32(&sm.q_full[i]), (uint32_t)pieces & 1u, abort_flag)) return false;
                        const int n = cnt + (SPLIT ? i : 0);
                        if ((SPLIT || i == 0) && !wait_k(n)) return false;
                        tc_fence_after();
                        issue_s(i, n, SPLIT || i == 1);
                    }
                    for (int i = 0; i < n_turns; ++i) {
                        const int wg = i & 1, n = cnt + (SPLIT ? i : i >> 1), vs = n % kV16Stages;
                        const bool more = i + 2 < n_turns, last = SPLIT || wg == 1;
                        if (SPLIT || wg == 0) {
                            if (!mbar_wait(smem_u32(&sm.v16_full[vs]), (uint32_t)(n / kV16Stages) & 1u, abort_flag)) return false;
                            if (more && !wait_k(SPLIT ? n + 2 : n + 1)) return false;
                        }
                        if (!mbar_wait(smem_u32(&sm.p_full[wg]), (turns >> wg) & 1u, abort_flag)) return false;
                        turns ^= 1u << wg;
                        tc_fence_after();
                        const uint64_t vd = sw128_mn_desc(smem_u32(sm.v16[vs]), kKT * 128);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)     // 16 keys: 8 columns of P, 16 rows of V
                            umma_bf16_ts(tmem + 256 + 128 * wg, tmem + 128 * wg + 8 * kk, vd + (uint64_t)(kk * (2048 >> 4)), idesc_o,
                                         (i > 1 || kk) ? 1u : 0u);
                        if (more) issue_s(wg, SPLIT ? n + 2 : n + 1, last);
                        else umma_commit(smem_u32(&sm.o_done[wg]));
                        if (last) umma_commit(smem_u32(&sm.v16_empty[vs]));
                    }
                    cnt += p.n;
                    ++pieces;
                    return true;
                });
            }
        } else if (tid == 96) {
            // what the combine pass needs to know
            OpenSegment open{0, 0, 0, 0, kUnit};
            walk([&](const Piece& p) -> bool {
                if ((p.where & ~Piece::kLast) == (Piece::kFirst | Piece::kStarts)) {
                    open.t0 = p.t0;
                    open.head = p.head;
                    open.rows = p.rows;
                    open.n_more = cta_of_tile(total, n_cta, p.seg_end - 1) - (int)blockIdx.x;
                }
                return true;
            });
            a.open[blockIdx.x] = open;
        }
    } else if (warp >= 12) {
        fewer_registers<88>();
        // ------------------------------------------------------------------ V to bf16
        // Thread (row y of 16, piece c of 8): 16 values of rows y, y + 16, ...; the 32 bytes go to two 16-byte places
        // of the swizzled bf16 tile, in an order that keeps the eight threads of a row on distinct banks.
        const int ct = tid - 384, c = ct & 7, y = ct >> 3;
        walk([&](const Piece& p) -> bool {
            for (int j = 0; j < p.n; ++j) {
                const int n = cnt + j, vs = n % kVStages, v2 = n % kV16Stages;
                const bool in = mbar_wait(smem_u32(&sm.v8_full[vs]), (uint32_t)(n / kVStages) & 1u, abort_flag) &&
                                mbar_wait(smem_u32(&sm.v16_empty[v2]), ((uint32_t)(n / kV16Stages) & 1u) ^ 1u, abort_flag);
                if (!__all_sync(0xffffffffu, in)) return false;
                const int left = p.len - (p.k0 + j) * kKT;         // keys of the tile that the sequence has
                uint8_t* dst = sm.v16[v2] + (c >> 2) * (kKT * 128);
                const int odd = c >> 2;                            // values 8 .. 15 are written first
                uint4 u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 16 * i + y;
                    u[i] = *reinterpret_cast<const uint4*>(sm.v8[vs] + row * 128 + ((c ^ (row & 7)) << 4));
                }
                const bool hole = left < kKT || sm.sk[n % kInfo][lane & 7] == 0.f;
                if (__any_sync(0xffffffffu, hole)) {               // anything may stand where no key is
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (16 * i + y >= left || sm.sk[n % kInfo][i] == 0.f) u[i] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 16 * i + y;
                    const uint32_t us[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                    uint32_t o[8];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        // high and low bytes of four bf16, sign and 0000eee, emmm0000: 2^-120 times the values
                        const uint32_t h = (us[x] & 0x80808080u) | ((us[x] >> 4) & 0x07070707u);
                        const uint32_t l = (us[x] << 4) & 0xF0F0F0F0u;
                        o[2 * x] = __byte_perm(l, h, 0x5140);
                        o[2 * x + 1] = __byte_perm(l, h, 0x7362);
                    }
                    const uint4 lo4 = make_uint4(o[0], o[1], o[2], o[3]), hi4 = make_uint4(o[4], o[5], o[6], o[7]);
                    const int at = ((2 * (c & 3) + odd) ^ (row & 7)) << 4;
                    *reinterpret_cast<uint4*>(dst + row * 128 + at) = odd ? hi4 : lo4;
                    *reinterpret_cast<uint4*>(dst + row * 128 + (at ^ 16)) = odd ? lo4 : hi4;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_u32(&sm.v16_full[v2]));
                mbar_arrive(smem_u32(&sm.v8_empty[vs]));
            }
            cnt += p.n;
            return true;
        });
    } else {
        more_registers<176>();
        // ------------------------------------------------------------------ softmax
        const int wg = (warp - 4) >> 2, rl = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * wg, to = tmem + lanes + 256 + 128 * wg;
        uint32_t taken = 0;                            // tiles of this warpgroup
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag));
            if (ok) tc_fence_after();
            return ok;
        };
        walk([&](const Piece& p) -> bool {
            const int row0 = (SPLIT ? 0 : wg * kRowsTile) + (warp & 3) * 32, row = row0 + lane;
            const bool valid = row < p.rows;
            const int seen = valid ? p.seen0 + (row >> gs) : 0;
            const int seen_warp = p.seen0 + (row0 >> gs);              // of the warp's first row: the fewest of all
            const int64_t gr = valid ? (p.t0 + (row >> gs)) * hq + p.head * G + (row & (G - 1)) : 0;

            // queries: half a warp per row, eight elements a lane, the two parts in 8-byte pieces; of a shared row block
            // each warpgroup does half
            {
                const int half = lane >> 4, piece = lane & 15;
                uint8_t* hi = sm.q[SPLIT ? 0 : wg][0];
                uint8_t* lo = sm.q[SPLIT ? 0 : wg][1];
                const int first = (warp & 3) * 32 + (SPLIT ? 16 * wg : 0);
                constexpr int kIter = SPLIT ? 8 : 16;
#pragma unroll 1
                for (int i0 = 0; i0 < kIter; i0 += 8) {
                    uint4 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = (SPLIT ? 0 : wg * kRowsTile) + first + 2 * (i0 + i) + half;
                        x[i] = make_uint4(0, 0, 0, 0);
                        if (r < p.rows)
                            x[i] = *reinterpret_cast<const uint4*>(
                                a.q + ((p.t0 + (r >> gs)) * hq + p.head * G + (r & (G - 1))) * kPagedD + 8 * piece);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                        const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(u);
                        const __nv_bfloat162 t2 = __hmax2(__hmax2(__habs2(b[0]), __habs2(b[1])), __hmax2(__habs2(b[2]), __habs2(b[3])));
                        float top = fmaxf(__low2float(t2), __high2float(t2));
#pragma unroll
                        for (int o = 8; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        // s = 2^e with top <= 448 s; the range keeps s and 1 / s normal
                        const uint32_t ub = __float_as_uint(top);
                        const int e = max(-100, min(120, (int)(ub >> 23) - 127 - 8 + ((ub & 0x7FFFFFu) > 0x600000u ? 1 : 0)));
                        const float inv = a.scale_log2e < 0.f ? -pow2f(-e) : pow2f(-e);
                        uint32_t h[4], l[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __half2 y = __floats2half2_rn(__uint_as_float(u[k] << 16) * inv,
                                                                __uint_as_float(u[k] & 0xFFFF0000u) * inv);
                            h[k] = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                            const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h[k], __NV_E4M3);
                            l[k] = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(
                                __hsub2(y, *reinterpret_cast<const __half2*>(&back)), __NV_SATFINITE, __NV_E4M3);
                        }
                        const int rr = first + 2 * (i0 + i) + half;
                        const int at = rr * kPagedD + (((piece >> 1) ^ (rr & 7)) << 4) + 8 * (piece & 1);
                        *reinterpret_cast<uint2*>(hi + at) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
                        *reinterpret_cast<uint2*>(lo + at) = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
                        if (piece == 0) sm.fr[SPLIT ? 0 : wg][rr] = ub >= 0x7F800000u ? __int_as_float(0x7FFFFFFF) : fabsf(a.scale_log2e) * pow2f(e);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_u32(&sm.q_full[SPLIT ? 0 : wg]));
                __syncwarp();
            }

            float m = valid ? ninf : 0.f, l = 0.f, le = 0.f;       // le: roundings of l
            bool any = false;                                      // O holds something
            bool ok = true;
            for (int j = SPLIT ? wg : 0; j < p.n; j += SPLIT ? 2 : 1) {
                if (!(ok = wait(&sm.s_full[wg], taken & 1u))) break;
                ++taken;
                const float fr = sm.fr[SPLIT ? 0 : wg][rl];        // written before the products that s_full reports
                const int info = (cnt + j) % kInfo;
                float f[8];                                        // logit factors, 16 columns each
                bool hole = false;                                 // a page that is not there
                {
                    const float4* sk = reinterpret_cast<const float4*>(sm.sk[info]);
                    const float4 u = sk[0], w = sk[1];
                    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = w.x, f[5] = w.y, f[6] = w.z, f[7] = w.w;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        hole |= f[i] == 0.f;
                        f[i] *= fr;
                    }
                }
                const int key0 = (p.k0 + j) * kKT;
                float sum = 0.f;
                // a new reference maximum, of sum and O, unless the old one will do for all of the warp's rows
                auto move_max = [&](float mt) {
                    if (!__any_sync(0xffffffffu, mt > m + kSlack)) return;
                    mt = fmaxf(mt, m);
                    const float al = m == mt ? 1.f : ex2(m - mt);
                    m = mt;
                    l *= al;
                    le *= al;
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_issue32(to + 32 * c, x);
                            tmem_wait32(x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * al);
                            tmem_st32_u32(to + 32 * c, x);
                        }
                    }
                };
                bool slow = hole || key0 + kKT > seen_warp;
                if (!slow) {
                    uint32_t xa[32], xb[32], pk[64];
                    if (__any_sync(0xffffffffu, m == ninf)) {      // the row's first keys
                        float mt = m;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            tmem_issue32(ts + 32 * c, xa);
                            tmem_wait32(xa);
                            float y = ninf, z = ninf;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                y = fmaxf(y, __uint_as_float(xa[i]));
                                z = fmaxf(z, __uint_as_float(xa[16 + i]));
                            }
                            mt = fmaxf(mt, fmaxf(y * (fr * sm.sk[info][2 * c]), z * (fr * sm.sk[info][2 * c + 1])));   // f > 0
                        }
                        move_max(mt);
                        if (m == ninf) m = 0.f;                    // a row of NaN: it need not come here again
                    }
                    // against the reference maximum as it is; V's scale goes into P's exponent
                    const float ref = m == ninf ? 0.f : m;
                    const float4* evs = reinterpret_cast<const float4*>(sm.ev[info]);
                    const float4* ivs = reinterpret_cast<const float4*>(sm.iv[info]);
                    const float4 e4[2] = {evs[0], evs[1]}, i4[2] = {ivs[0], ivs[1]};
                    auto part = [&](uint32_t (&x)[32], int at) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c = 2 * at + h;
                            const float ff = f[c], nm = (&e4[c >> 2].x)[c & 3] - ref;
                            uint64_t sum2 = 0;
#pragma unroll
                            for (int i = 16 * h; i < 16 * h + 16; i += 2) {
                                const uint64_t y = fma2(pair_u(x[i], x[i + 1]), pair(ff, ff), pair(nm, nm));
                                const float p0 = ex2(first(y)), p1 = ex2(second(y));
                                sum2 = add2(sum2, pair(p0, p1));
                                pk[16 * at + i / 2] = pack_bf16(p0, p1);
                            }
                            sum = fmaf(first(sum2) + second(sum2), (&i4[c >> 2].x)[c & 3], sum);
                        }
                    };
                    tmem_issue32(ts, xa);
                    tmem_wait32(xa);
                    tmem_issue32(ts + 32, xb);
                    part(xa, 0);
                    tmem_wait32(xb);
                    tmem_issue32(ts + 64, xa);
                    part(xb, 1);
                    tmem_wait32(xa);
                    tmem_issue32(ts + 96, xb);
                    part(xa, 2);
                    tmem_wait32(xb);
                    part(xb, 3);
                    slow = __any_sync(0xffffffffu, sum > kTrigger);
                    if (!slow) {
                        tmem_st32_u32(ts, pk);
                        tmem_st32_u32(ts + 32, pk + 32);
                    }
                }
                if (slow) {
                    // masked tiles, and those that move the maximum: 32 columns at a time
                    const int vis = seen - key0;
                    const float* sk = sm.sk[info];
                    float mt = m;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32];
                        tmem_issue32(ts + 32 * c, x);
                        tmem_wait32(x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float ks = sk[2 * c + (i >> 4)];
                            mt = fmaxf(mt, (32 * c + i < vis && ks != 0.f) ? __uint_as_float(x[i]) * (fr * ks) : ninf);
                        }
                    }
                    move_max(mt);
                    const float ref = m == ninf ? 0.f : m;
                    sum = 0.f;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {                  // P overwrites columns that have been read
                        uint32_t x[32], y[16];
                        tmem_issue32(ts + 32 * c, x);
                        tmem_wait32(x);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float ks = sk[2 * c + h], ff = fr * ks, nm = sm.ev[info][2 * c + h] - ref;
                            float part = 0.f;
#pragma unroll
                            for (int i = 16 * h; i < 16 * h + 16; i += 2) {
                                float q[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    q[k] = (32 * c + i + k < vis && ks != 0.f) ? ex2(fmaf(__uint_as_float(x[i + k]), ff, nm)) : 0.f;
                                    part += q[k];
                                }
                                y[i / 2] = pack_bf16(q[0], q[1]);
                            }
                            sum = fmaf(part, sm.iv[info][2 * c + h], sum);
                        }
                        tmem_st16_u32(ts + 16 * c, y);
                    }
                }
                any = true;
                {
                    const float d = sum - le, t = l + d;
                    le = (t - l) - d;
                    l = t;
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                mbar_arrive(smem_u32(&sm.p_full[wg]));
            }
            if (ok && any) ok = wait(&sm.o_done[wg], (uint32_t)pieces & 1u);
            if (any) ++pieces;
            if (!SPLIT && !ok) return false;
            cnt += p.n;

            // out, or the workspace
            constexpr int kWhole = Piece::kStarts | Piece::kEnds | Piece::kLast;
            const bool whole = (p.where & kWhole) == kWhole;
            const int64_t slot0 = ((int64_t)blockIdx.x * 2 + (p.where & Piece::kStarts)) * a.rows + row0;
            // Earlier runs of the share come back by their maximum and sum (which both warpgroups read) and by the pieces of O
            // that each thread wrote itself, with weight w_old; what this run has gets the weight returned.
            float w_old = 0.f;
            auto join_earlier = [&]() -> float {
                if (p.where & Piece::kFirst) return 1.f;
                const float2 old = valid ? a.part_ml[slot0 + lane] : make_float2(ninf, 0.f);
                const float M = fmaxf(m, old.x), w = m == ninf ? 0.f : ex2(m - M);
                w_old = old.x == ninf ? 0.f : ex2(old.x - M);
                l = (m == ninf ? l : w * l) + (old.x == ninf ? old.y : w_old * old.y);
                m = M;
                return w;
            };
            // a piece of a row: four columns from `col` on of row r of the warp's, by all lanes together
            auto put = [&](int r, int col, float4 y) {
                const int rr = row0 + r;
                const float w = __shfl_sync(0xffffffffu, w_old, r);
                if (rr >= p.rows) return;
                if (w != 0.f) {
                    const float4 z = *reinterpret_cast<const float4*>(a.part_o + slot0 * kPagedD + r * kPagedD + col);
                    y = make_float4(fmaf(w, z.x, y.x), fmaf(w, z.y, y.y), fmaf(w, z.z, y.z), fmaf(w, z.w, y.w));
                }
                if (whole) {
                    uint2 u;
                    u.x = pack_bf16(y.x, y.y);
                    u.y = pack_bf16(y.z, y.w);
                    const int off = ((rr >> gs) * hq + (rr & (G - 1))) * kPagedD + col;
                    *reinterpret_cast<uint2*>(a.out + (p.t0 * hq + p.head * G) * kPagedD + off) = u;
                } else {
                    *reinterpret_cast<float4*>(a.part_o + slot0 * kPagedD + r * kPagedD + col) = y;
                }
            };
            if (SPLIT) {
                // Both warpgroups' parts are joined, each warpgroup for half of the columns: the other half goes to the
                // other one through the place of the queries (the first row block's for columns 0 .. 63, which
                // warpgroup 1 writes). Named barrier 1 holds the two together.
                sm.ml[wg][rl] = make_float2(m, l);
                asm volatile("bar.sync 1, 256;" ::: "memory");     // no product reads the queries any more
                const float2 other = sm.ml[wg ^ 1][rl];
                const float M = fmaxf(m, other.x);
                float w0 = m == ninf ? 0.f : ex2(m - M), w1 = other.x == ninf ? 0.f : ex2(other.x - M);
                l = (m == ninf ? l : w0 * l) + (other.x == ninf ? other.y : w1 * other.y);
                m = M;
                const float w_new = join_earlier();                // before the barrier behind which wg 0 writes anew
                float x[64];
                tmem_ld64(to + 64 * (wg ^ 1), x);
                float4* theirs = reinterpret_cast<float4*>(sm.q[wg ^ 1][0]) + rl * 16;
#pragma unroll
                for (int i = 0; i < 16; ++i) theirs[i ^ (rl & 15)] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                tmem_ld64(to + 64 * wg, x);
                asm volatile("bar.sync 1, 256;" ::: "memory");
                const float f = !whole ? 1.f : l == 0.f ? 0.f : kUnit / l;
                w0 *= w_new * f;
                w1 *= w_new * f;
                w_old *= f;
                float4* mine = reinterpret_cast<float4*>(sm.q[wg][0]) + rl * 16;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 y = mine[i ^ (rl & 15)];          // a part without a key may hold anything
                    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (w0 != 0.f) z = make_float4(w0 * x[4 * i], w0 * x[4 * i + 1], w0 * x[4 * i + 2], w0 * x[4 * i + 3]);
                    if (w1 != 0.f) z = make_float4(fmaf(w1, y.x, z.x), fmaf(w1, y.y, z.y), fmaf(w1, y.z, z.z), fmaf(w1, y.w, z.w));
                    mine[i ^ (rl & 15)] = z;
                }
                __syncwarp();
                // sixteen lanes write a row's half
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int r = 2 * i + (lane >> 4), c = lane & 15;
                    put(r, 64 * wg + 4 * c, reinterpret_cast<const float4*>(sm.q[wg][0])[((warp & 3) * 32 + r) * 16 + (c ^ (r & 15))]);
                }
            } else {
                // 32 columns of the warp's rows at a time, through the place of its queries (which no product reads any
                // more), so that eight lanes write a row's piece
                const float w_new = join_earlier(), unit = !whole ? 1.f : l == 0.f ? 0.f : kUnit / l, f = w_new * unit;
                w_old *= unit;
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {
                    float x[32];
                    tmem_ld32(to + 32 * part, x);
                    float4* stage = reinterpret_cast<float4*>(sm.q[wg][part & 1] + (warp & 3) * 32 * kPagedD);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        stage[lane * 8 + (i ^ (lane & 7))] = make_float4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
                    __syncwarp();
#pragma unroll 4
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + (lane >> 3), c = lane & 7;
                        put(r, 32 * part + 4 * c, stage[r * 8 + (c ^ (r & 7))]);
                    }
                    __syncwarp();
                }
            }
            if (valid && (!SPLIT || wg == 0)) {
                if (whole) {
                    if (a.lse) a.lse[gr] = l == 0.f ? ninf : (m + log2f(l)) * 0.6931471805599453f;
                } else {
                    a.part_ml[slot0 + lane] = make_float2(m, l);
                }
            }
            tc_fence_before();
            if (SPLIT) {
                // the next piece's queries may come; both warpgroups go on, or neither
                if (wg == 0 && rl == 0) sm.stop = *abort_flag;
                asm volatile("bar.sync 1, 256;" ::: "memory");
                return sm.stop == 0;
            }
            return true;
        });
    }
    __syncthreads();
    if (*abort_flag) {
        if (tid == 0) record_device_error(a.err, MSA_DEV_WAIT_TIMEOUT);
        if (warp == 1 && lane == 0) {
            umma_commit(smem_u32(&sm.drain));
            mbar_wait_drain(smem_u32(&sm.drain), 0);
        }
        if (tid == 0) {
            // leave no copy in flight: each stage's last load
            for (int i = 0; i < kKStages; ++i)
                if (loading_k > i) mbar_wait_drain(smem_u32(&sm.k_full[i]), (uint32_t)((loading_k - 1 - i) / kKStages) & 1u);
            for (int i = 0; i < kVStages; ++i)
                if (loading_v > i) mbar_wait_drain(smem_u32(&sm.v8_full[i]), (uint32_t)((loading_v - 1 - i) / kVStages) & 1u);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <bool SPLIT>
msa_status launch(const CUtensorMap& tm, const PagedAttnArgs& a, int grid, cudaStream_t s) {
    constexpr int smem = (int)sizeof(PromptSmem) + 1024;
    static_assert(smem <= 232448, "shared memory");
    static std::mutex mu;
    static bool opted[64] = {false};
    int dev = 0;
    MSA_CUDA_TRY(cudaGetDevice(&dev));
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev < 0 || dev >= 64 || !opted[dev]) {
            MSA_CUDA_TRY(cudaFuncSetAttribute(paged_prompt_kernel<SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
            if (dev >= 0 && dev < 64) opted[dev] = true;
        }
    }
    MSA_CUDA_TRY(launch_early(paged_prompt_kernel<SPLIT>, dim3((unsigned)grid), kThreads, smem, s, tm, a));
    return MSA_OK;
}

}  // namespace

msa_status launch_paged_prompt(const PagedAttnArgs& a, int grid, cudaStream_t s) {
    // the pages as rows of 128 bytes (64 two-byte elements); a box is one page of keys or of values of a head
    CUtensorMap tm{};
    const uint64_t dims[2] = {64, (uint64_t)(a.v.n_pages * 2 * a.v.hkv * a.v.page)};
    const uint64_t strides[1] = {kPagedD};
    const uint32_t box[2] = {64, (uint32_t)a.v.page};
    MSA_RETURN_IF(make_tensor_map_bf16(&tm, a.v.pages, 2, dims, strides, box));
    return a.rows == kRowsTile ? launch<true>(tm, a, grid, s) : launch<false>(tm, a, grid, s);
}

}  // namespace msa
