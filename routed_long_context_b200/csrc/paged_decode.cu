// Attention of few query rows over a paged 8-bit cache: single tokens, a handful of drafted ones, and single
// tokens over their page lists.
//
//   out = softmax(scale q . K) V,  up to 8 rows (token, query head) of one kv head at a time.
// Every cached byte is read once for 4 * 8 operations at most, so the bytes bound it; what costs is turning
// them into operands. A warp takes 16 keys at a time, transposed, on mma.sync (the 128-row tiles of
// tcgen05.mma would be empty but for 1 to 8 rows, and want the keys' operands written back to shared memory):
//   S^T [16 keys x 8 rows]  = K [16 x 128] Q^T         K: e4m3 -> fp16 exactly; Q: fp16 times a power of two
//   O^T [128 x 8 rows]     += V^T [128 x 16] P^T       V: e4m3 -> bf16 exactly; P: bf16
// so all eight columns are rows of the softmax. The order of d inside both products is free: a thread takes
// the 16-byte pieces that it can read from shared memory without bank conflicts. Keys and values come by TMA
// in the 128-byte swizzle, three tiles of 4 KB deep for each of the 16 warps of an SM (192 KB in flight; 44 KB
// cover the latency). The running maximum moves only when a logit exceeds it by 2^8.
// P carries the page's scale of V times 2^60, V stands 2^-120 too low: an e4m3 value's bits moved to a bf16's
// place, subnormals included, need no multiplication that way.
#include <algorithm>
#include <mutex>

#include "kernels.cuh"
#include "mma.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace msa {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kTileBytes = 2 * kDecodeTile * kPagedD;      // K and V of a tile
constexpr int kWindow = 256;                               // sequences looked at together
constexpr float kSlack = 8.f;
constexpr float kUnit = 1152921504606846976.f;             // 2^60: the unit in which O is kept

struct TileInfo {
    int key;          // first key's place in the sequence
    int rows;         // keys that hold something; 0: nothing was loaded
    float sk, sv;     // scales of K and of V
};

struct DecodeSmem {
    uint8_t ring[kWarps][kStages][kTileBytes];
    float o[kWarps][kDecodeRows][32];
    float2 ml[kWarps][kDecodeRows];
    TileInfo info[kWarps][kStages];
    uint64_t bar[kWarps][kStages];
    long long pre[kWindow + 1];                            // tiles before each sequence of the window
    int64_t t0[kWindow];
    int n_new[kWindow], len[kWindow];
    long long scan[kWarps];
    int abort_flag;
};

__device__ __forceinline__ void mma_f16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t u) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u, __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
// e4m3 bytes in the high bytes of both halves -> bf16 of 2^-120 times their values
__device__ __forceinline__ uint32_t e4m3_high_bf16x2(uint32_t z) {
    return ((z >> 4) & 0x07F007F0u) | (z & 0x80008000u);
}

// Prefix sums over the block of one value per thread; returns the block's total.
__device__ __forceinline__ long long block_prefix(long long x, long long* pre, long long* scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = s;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    pre[threadIdx.x + 1] = before + s;
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
    return total;
}

template <bool LIST>
__global__ void __launch_bounds__(kThreads, 2) paged_decode_kernel(const __grid_constant__ CUtensorMap tm,
                                                                   const PagedAttnArgs a) {
    extern __shared__ uint8_t smem_raw[];
    DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const PagedView& v = a.v;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;                 // the thread's place in a fragment
    const int G = a.G, hq = v.hkv * G, page = v.page;
    const int per_page = page / kDecodeTile;
    const float ninf = -INFINITY;
    volatile int* abort_flag = &sm.abort_flag;
    if (tid == 0) sm.abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sm.bar[warp][i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }

    // tiles of all sequences
    const int n_windows = LIST ? 1 : (v.n_seq + kWindow - 1) / kWindow;
    auto load_window = [&](int w) -> long long {
        const int s = w * kWindow + tid;
        SeqSpan sp{0, 0, 0};
        if (s < v.n_seq) seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, blockIdx.x == 0 ? a.err : nullptr);
        __syncthreads();
        sm.t0[tid] = sp.t0;
        sm.n_new[tid] = sp.n_new;
        sm.len[tid] = sp.len;
        return block_prefix(sp.n_new ? (long long)v.hkv * ((sp.len + kDecodeTile - 1) / kDecodeTile) : 0, sm.pre,
                            sm.scan);
    };
    long long total = 0, first_total = 0;
    const int list_tiles = LIST ? a.k * per_page : 1;
    if (LIST) {
        total = first_total = a.n_tok * v.hkv * (long long)list_tiles;
        __syncthreads();
    } else {
        for (int w = n_windows - 1; w >= 0; --w) {
            first_total = load_window(w);
            total += first_total;
        }
    }
    const int n_cta = (int)min((long long)gridDim.x, (total + kWarps - 1) / kWarps);
    if ((int)blockIdx.x >= n_cta) {
        if (tid == 0) a.open[blockIdx.x].n_more = 0;
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        return;
    }
    const long long my_a = cta_first(total, n_cta, blockIdx.x), my_b = cta_first(total, n_cta, blockIdx.x + 1);
    OpenSegment open{0, 0, 0, 0, kUnit};

    int it = 0;                                            // tiles this warp has taken: ring stage and phase
    long long base = 0;                                    // tiles before the window
    for (int w = 0; w < n_windows; ++w) {
        const long long in_window = (w == 0) ? first_total : load_window(w);
        const long long A = max(my_a - base, 0LL), B = min(my_b - base, in_window);
        if (A >= B) {
            base += in_window;
            continue;
        }
        const int n_win = LIST ? 0 : min(kWindow, v.n_seq - w * kWindow);

        // Lane l looks up tile l of the warp's next 32; they are issued one by one as ring stages come free.
        TileInfo ti{0, 0, 0.f, 0.f};
        int ti_row = 0;                                    // tensor-map row of the tile's first key
        const int n_mine = (int)((B - A - warp + kWarps - 1) / kWarps);
        int issued = 0;
        auto look_up = [&]() {
            ti = TileInfo{0, 0, 0.f, 0.f};
            const long long g = A + warp + (long long)kWarps * (issued + lane);
            if (g >= B) return;
            int s, p, head, row0, seen;
            if (LIST) {
                const long long seg = g / list_tiles;
                const int e = (int)(g - seg * list_tiles);
                const long long t = seg / v.hkv;
                head = (int)(seg - t * v.hkv);
                int lo = 0, n = v.n_seq;                   // the last sequence that starts at or before t
                while (n > 1) {
                    const int h = n / 2;
                    if (a.tok_off[lo + h] <= t) {
                        lo += h;
                        n -= h;
                    } else {
                        n = h;
                    }
                }
                s = lo;
                SeqSpan sp;
                if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, a.err) || t < sp.t0 || t >= sp.t0 + sp.n_new) return;
                seen = sp.len - sp.n_new + (int)(t - sp.t0) + 1;
                const int li = e / per_page;
                p = a.sel[seg * a.k + li];
                row0 = (e - li * per_page) * kDecodeTile;
                if (p == -1) return;
                if (p < 0 || p >= (seen + page - 1) >> v.shift) {
                    record_device_error(a.err, MSA_DEV_BAD_INDEX);
                    return;
                }
            } else {
                int lo = 0, n = n_win;
                while (n > 1) {
                    const int h = n / 2;
                    if (sm.pre[lo + h] <= g) {
                        lo += h;
                        n -= h;
                    } else {
                        n = h;
                    }
                }
                s = w * kWindow + lo;
                seen = sm.len[lo];
                const int per_head = (seen + kDecodeTile - 1) / kDecodeTile;
                const long long at = g - sm.pre[lo];
                head = (int)(at / per_head);
                const int key = (int)(at - (long long)head * per_head) * kDecodeTile;
                p = key >> v.shift;
                row0 = key & (page - 1);
            }
            const int32_t pid = v.table[(int64_t)s * v.max_pages + p];
            if (pid < 0 || pid >= v.n_pages) {
                record_device_error(a.err, MSA_DEV_BAD_INDEX);
                return;
            }
            const int64_t slab = (int64_t)pid * 2 * v.hkv + head;
            ti.key = (p << v.shift) + row0;
            ti.rows = max(0, min(kDecodeTile, seen - ti.key));
            ti.sk = v.scales[slab];
            ti.sv = v.scales[slab + v.hkv];
            ti_row = (int)(slab * page) + row0;
        };
        auto issue = [&]() {
            if (issued >= n_mine) return;
            const int n = it + issued;                     // it counts the consumed tiles of earlier windows
            if ((issued & 31) == 0) look_up();
            const int st = n % kStages;
            if (lane == (issued & 31)) {
                const uint32_t bar = smem_u32(&sm.bar[warp][st]);
                sm.info[warp][st] = ti;
                if (ti.rows > 0) {
                    const uint32_t dst = smem_u32(sm.ring[warp][st]);
                    mbar_expect_tx(bar, kTileBytes);
                    tma_load_2d(dst, &tm, 0, ti_row, bar);
                    tma_load_2d(dst + kTileBytes / 2, &tm, 0, ti_row + v.hkv * page, bar);
                } else {
                    mbar_arrive(bar);
                }
            }
            ++issued;
            __syncwarp();
        };
        for (int i = 0; i < kStages; ++i) issue();
        int taken = 0;

        // segment by segment
        for (long long g0 = A; g0 < B;) {
            long long seg_a, seg_b;
            int64_t t0;
            int head, n_rows, len, n_new;
            bool live = true;
            if (LIST) {
                const long long seg = g0 / list_tiles;
                t0 = seg / v.hkv;
                head = (int)(seg - t0 * v.hkv);
                seg_a = seg * list_tiles;
                seg_b = seg_a + list_tiles;
                const int s = seq_of_token(a.tok_off, v.n_seq, t0);
                SeqSpan sp;
                live = seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, nullptr) && t0 >= sp.t0 && t0 < sp.t0 + sp.n_new;
                len = sp.len - sp.n_new + (int)(t0 - sp.t0) + 1;
                n_new = 1;
            } else {
                int lo = 0, n = n_win;
                while (n > 1) {
                    const int h = n / 2;
                    if (sm.pre[lo + h] <= g0) {
                        lo += h;
                        n -= h;
                    } else {
                        n = h;
                    }
                }
                t0 = sm.t0[lo];
                n_new = sm.n_new[lo];
                len = sm.len[lo];
                const int per_head = (len + kDecodeTile - 1) / kDecodeTile;
                head = (int)((g0 - sm.pre[lo]) / per_head);
                seg_a = sm.pre[lo] + (long long)head * per_head;
                seg_b = seg_a + per_head;
            }
            n_rows = live ? n_new * G : 0;
            const long long g1 = min(B, seg_b);

            // this thread's part of Q^T: row n = r, elements 32 c .. 32 c + 31, times a power of two that brings the
            // row's largest to [2^14, 2^15); what of the row is below 2^-39 of that is lost
            uint32_t qf[16];
            float f0, f1;                                  // logit factors of rows 2 c and 2 c + 1
            {
                float x[32];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
                if (r < n_rows) {
                    const __nv_bfloat16* src = a.q + ((t0 + r / G) * hq + head * G + r % G) * kPagedD + 32 * c;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) load16_f32(src + i, x + i);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = max(-112, min(127, (int)(__float_as_uint(top) >> 23) - 127));
                const float up = pow2f(14 - e > 127 ? 127 : 14 - e);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const __half2 h = __floats2half2_rn(x[2 * i] * up, x[2 * i + 1] * up);
                    qf[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
                const float f = a.scale_log2e * pow2f(e - 14);
                f0 = __shfl_sync(0xffffffffu, f, 8 * c);
                f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);
            }
            const int seen0 = 2 * c < n_rows ? len - n_new + 2 * c / G + 1 : 0;
            const int seen1 = 2 * c + 1 < n_rows ? len - n_new + (2 * c + 1) / G + 1 : 0;
            const int seen_all = len - n_new + 1;          // keys that every row sees

            float o[8][4], m0 = ninf, m1 = ninf, l0 = 0.f, l1 = 0.f, e0 = 0.f, e1 = 0.f;   // e: roundings of l
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

            for (; A + warp + (long long)kWarps * taken < g1; ++taken) {
                const int n = it + taken, st = n % kStages;
                const bool ok = __all_sync(
                    0xffffffffu, mbar_wait(smem_u32(&sm.bar[warp][st]), (uint32_t)(n / kStages) & 1u, abort_flag));
                const TileInfo t = sm.info[warp][st];
                if (ok && t.rows > 0) {
                    const uint8_t* sk = sm.ring[warp][st];
                    const uint8_t* sv = sk + kTileBytes / 2;
                    // S^T: 16-byte pieces 2 c and 2 c + 1 of key rows r and r + 8 (piece i of row y lies at i ^ y % 8)
                    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int off = r * 128 + (((2 * c + h) ^ r) << 4);
                        const uint4 x = *reinterpret_cast<const uint4*>(sk + off);
                        const uint4 y = *reinterpret_cast<const uint4*>(sk + 1024 + off);
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t f[4];
                            f[0] = e4m3x2_f16x2(xs[i] & 0xFFFFu);
                            f[1] = e4m3x2_f16x2(ys[i] & 0xFFFFu);
                            f[2] = e4m3x2_f16x2(xs[i] >> 16);
                            f[3] = e4m3x2_f16x2(ys[i] >> 16);
                            mma_f16_16816(s, f, qf[8 * h + 2 * i], qf[8 * h + 2 * i + 1]);
                        }
                    }
                    const float k0 = f0 * t.sk, k1 = f1 * t.sk;
                    float x00 = s[0] * k0, x01 = s[1] * k1, x10 = s[2] * k0, x11 = s[3] * k1;   // [key r, r + 8][row]
                    if (t.key + kDecodeTile > seen_all) {
                        const int ka = t.key + r, kb = ka + 8;
                        x00 = ka < seen0 ? x00 : ninf;
                        x01 = ka < seen1 ? x01 : ninf;
                        x10 = kb < seen0 ? x10 : ninf;
                        x11 = kb < seen1 ? x11 : ninf;
                    }
                    float t0m = fmaxf(x00, x10), t1m = fmaxf(x01, x11);
                    if (__any_sync(0xffffffffu, t0m > m0 + kSlack || t1m > m1 + kSlack)) {
#pragma unroll
                        for (int sh = 4; sh <= 16; sh <<= 1) {
                            t0m = fmaxf(t0m, __shfl_xor_sync(0xffffffffu, t0m, sh));
                            t1m = fmaxf(t1m, __shfl_xor_sync(0xffffffffu, t1m, sh));
                        }
                        t0m = fmaxf(t0m, m0);
                        t1m = fmaxf(t1m, m1);
                        const float a0 = m0 == t0m ? 1.f : ex2(m0 - t0m), a1 = m1 == t1m ? 1.f : ex2(m1 - t1m);
                        m0 = t0m;
                        m1 = t1m;
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
                    const float n0 = m0 == ninf ? 0.f : m0, n1 = m1 == ninf ? 0.f : m1;
                    x00 = ex2(x00 - n0);
                    x10 = ex2(x10 - n0);
                    x01 = ex2(x01 - n1);
                    x11 = ex2(x11 - n1);
                    {
                        const float d0 = (x00 + x10) - e0, d1 = (x01 + x11) - e1;
                        const float s0 = l0 + d0, s1 = l1 + d1;
                        e0 = (s0 - l0) - d0;
                        e1 = (s1 - l1) - d1;
                        l0 = s0;
                        l1 = s1;
                    }
                    const float pv = t.sv * kUnit;
                    const uint32_t b0 = transpose8x8(pack_bf16(x00 * pv, x01 * pv));
                    const uint32_t b1 = transpose8x8(pack_bf16(x10 * pv, x11 * pv));
                    // O^T: piece r (d = 16 r ..) of keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9; row r of the fragment of tile i is
                    // d = 16 r + 2 i, row r + 8 the next
                    uint4 w4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 2 * c + (i & 1) + 8 * (i >> 1);
                        w4[i] = *reinterpret_cast<const uint4*>(sv + key * 128 + ((r ^ (key & 7)) << 4));
                    }
                    if (t.rows < kDecodeTile) {            // rows behind the end hold anything
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (2 * c + (i & 1) + 8 * (i >> 1) >= t.rows) w4[i] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t wa = (&w4[0].x)[i], wb = (&w4[1].x)[i], wc = (&w4[2].x)[i], wd = (&w4[3].x)[i];
                        uint32_t f[4];
                        f[0] = e4m3_high_bf16x2(__byte_perm(wa, wb, 0x4000));
                        f[1] = e4m3_high_bf16x2(__byte_perm(wa, wb, 0x5010));
                        f[2] = e4m3_high_bf16x2(__byte_perm(wc, wd, 0x4000));
                        f[3] = e4m3_high_bf16x2(__byte_perm(wc, wd, 0x5010));
                        mma_bf16_16816(o[2 * i], f, b0, b1);
                        f[0] = e4m3_high_bf16x2(__byte_perm(wa, wb, 0x6020));
                        f[1] = e4m3_high_bf16x2(__byte_perm(wa, wb, 0x7030));
                        f[2] = e4m3_high_bf16x2(__byte_perm(wc, wd, 0x6020));
                        f[3] = e4m3_high_bf16x2(__byte_perm(wc, wd, 0x7030));
                        mma_bf16_16816(o[2 * i + 1], f, b0, b1);
                    }
                }
                __syncwarp();
                issue();
            }

            // join the warps: row n of the segment by warp n, 32 columns at a time
#pragma unroll
            for (int sh = 4; sh <= 16; sh <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
                l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
            }
            __syncthreads();                               // the last segment's values have been read
            if (lane < 4) {
                sm.ml[warp][2 * c] = make_float2(m0, l0);
                sm.ml[warp][2 * c + 1] = make_float2(m1, l1);
            }
            __syncthreads();
            float M = ninf, L = 0.f, wt[kWarps], res[4];
#pragma unroll
            for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm.ml[i][warp].x);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 x = sm.ml[i][warp];
                wt[i] = x.x == ninf ? 0.f : ex2(x.x - M);
                L += x.x == ninf ? x.y : wt[i] * x.y;      // a sum without a maximum is 0 or NaN
            }
#pragma unroll
            for (int part = 0; part < 4; ++part) {
                if (part) __syncthreads();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float* x = o[2 * part];
                    const float* y = o[2 * part + 1];
                    *reinterpret_cast<float4*>(&sm.o[warp][2 * c + j][4 * r]) = make_float4(x[j], x[2 + j], y[j], y[2 + j]);
                }
                __syncthreads();
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) x += wt[i] * sm.o[i][warp][lane];
                res[part] = x;                             // d = 16 (lane / 4) + 4 part + lane % 4
            }
            if (warp < n_rows) {
                const int d0 = 16 * (lane >> 2) + (lane & 3);
                if (seg_a == g0 && seg_b == g1) {
                    const int64_t row = (t0 + warp / G) * hq + head * G + warp % G;
                    const float inv = L == 0.f ? 0.f : kUnit / L;
#pragma unroll
                    for (int i = 0; i < 4; ++i) a.out[row * kPagedD + d0 + 4 * i] = __float2bfloat16_rn(res[i] * inv);
                    if (a.lse && lane == 0) a.lse[row] = L == 0.f ? ninf : (M + log2f(L)) * 0.6931471805599453f;
                } else {
                    const int64_t row = ((int64_t)blockIdx.x * 2 + (seg_a == g0 ? 1 : 0)) * a.rows + warp;
#pragma unroll
                    for (int i = 0; i < 4; ++i) a.part_o[row * kPagedD + d0 + 4 * i] = res[i];
                    if (lane == 0) a.part_ml[row] = make_float2(M, L);
                }
            }
            if (seg_a == g0 && seg_b > g1 && live) {
                open.t0 = t0;
                open.head = head;
                open.rows = n_rows;
                open.n_more = cta_of_tile(total, n_cta, base + seg_b - 1) - (int)blockIdx.x;
            }
            g0 = g1;
        }
        it += n_mine;
        base += in_window;
        __syncthreads();
    }
    if (tid == 0) a.open[blockIdx.x] = open;
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (*abort_flag && lane == 0) {
        record_device_error(a.err, MSA_DEV_WAIT_TIMEOUT);
        // leave no copy in flight: the last phase of each stage
        for (int i = 0; i < kStages; ++i)
            if (it > i) mbar_wait_drain(smem_u32(&sm.bar[warp][i]), (uint32_t)((it - 1 - i) / kStages) & 1u);
    }
}

}  // namespace

msa_status launch_paged_decode(const PagedAttnArgs& a, int grid, cudaStream_t s) {
    constexpr int smem = (int)sizeof(DecodeSmem) + 1024;
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two blocks per SM");
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
    // the pages as rows of 128 bytes (64 two-byte elements); a box is one tile of keys or of values
    CUtensorMap tm{};
    const uint64_t dims[2] = {64, (uint64_t)(a.v.n_pages * 2 * a.v.hkv * a.v.page)};
    const uint64_t strides[1] = {kPagedD};
    const uint32_t box[2] = {64, kDecodeTile};
    MSA_RETURN_IF(make_tensor_map_bf16(&tm, a.v.pages, 2, dims, strides, box));
    if (a.sel) paged_decode_kernel<true><<<grid, kThreads, smem, s>>>(tm, a);
    else paged_decode_kernel<false><<<grid, kThreads, smem, s>>>(tm, a);
    MSA_LAUNCH_CHECK();
    return MSA_OK;
}

}  // namespace msa
