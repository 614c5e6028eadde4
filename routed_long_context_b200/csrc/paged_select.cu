// Picking the pages of a paged cache that a query token attends over, by the bounds of their keys.
//
// score(token, kv head, page) = max over the group's query heads of sum_d max(q_d lo_d, q_d hi_d): the largest
// logit (before the scale) that any key inside the page's bounds could give. Sums are in 64 bits, so that
// what is picked does not depend on the order of summation. The newest pages count as infinite; the k best are
// picked, ties to the lower page, and listed in ascending order.
#include <algorithm>

#include "kernels.cuh"
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
    unsigned long long* keys;      // [n_tok][hkv][max_pages], ordered like the scores
    int keys_in_smem;
    int* err;
};

constexpr int kScorePages = 64;    // pages per block of the scoring kernel

// Order-preserving map of a double to an unsigned integer (-0 below +0, which the score never distinguishes
// because it adds +0 first).
__device__ __forceinline__ unsigned long long ordered(double x) {
    const long long b = __double_as_longlong(x);
    return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

template <int G>
__global__ void __launch_bounds__(256) page_score_kernel(const SelectArgs a) {
    const PagedView& v = a.v;
    const int64_t t = blockIdx.z;
    const int g = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = seq_of_token(a.tok_off, v.n_seq, t);
    SeqSpan sp;
    if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, nullptr) || t < sp.t0 || t >= sp.t0 + sp.n_new) return;
    const int at = sp.len - sp.n_new + (int)(t - sp.t0);
    const int last = at >> v.shift;
    const int p0 = blockIdx.x * kScorePages;
    if (p0 > last || last < a.k) return;          // every visible page is picked
    double q[G][4];
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[h][i] = (double)__bfloat162float(a.q[((t * v.hkv + g) * G + h) * kPagedD + lane * 4 + i]);
    unsigned long long* keys = a.keys + (t * v.hkv + g) * v.max_pages;
    for (int p = p0 + warp; p < min(p0 + kScorePages, last + 1); p += 8) {
        const int32_t pid = v.table[(int64_t)s * v.max_pages + p];
        double best = -INFINITY;
        if (pid < 0 || pid >= v.n_pages) {
            if (lane == 0) record_device_error(a.err, MSA_DEV_BAD_INDEX);
        } else {
            const __nv_bfloat16* b = v.bounds + ((int64_t)pid * v.hkv + g) * 2 * kPagedD + lane * 4;
            double lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = (double)__bfloat162float(b[i]);
                hi[i] = (double)__bfloat162float(b[kPagedD + i]);
            }
#pragma unroll
            for (int h = 0; h < G; ++h) {
                double x = 0.0;
#pragma unroll
                for (int i = 0; i < 4; ++i) x += fmax(q[h][i] * lo[i], q[h][i] * hi[i]);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                best = fmax(best, x);
            }
        }
        if (p > last - a.recent) best = INFINITY;
        if (lane == 0) keys[p] = ordered(best + 0.0);
    }
}

// One block per (token, kv head): the k-th largest key by radix digits from the top, then the pages above it
// and the first of those equal to it, in ascending order.
constexpr int kPickThreads = 256;
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectArgs a) {
    extern __shared__ unsigned long long s_keys[];
    __shared__ int hist[256];
    __shared__ unsigned long long s_prefix;
    __shared__ int s_want, s_done, s_run[2];
    __shared__ int s_cnt[2][kPickThreads / 32];
    const PagedView& v = a.v;
    const int64_t t = blockIdx.x;
    const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = seq_of_token(a.tok_off, v.n_seq, t);
    SeqSpan sp;
    int32_t* sel = a.sel + (t * v.hkv + g) * a.k;
    if (!seq_span(v, a.tok_off, a.n_tok, a.max_new, s, &sp, tid == 0 ? a.err : nullptr) || t < sp.t0 ||
        t >= sp.t0 + sp.n_new)
        return;
    const int n = ((sp.len - sp.n_new + (int)(t - sp.t0)) >> v.shift) + 1;      // visible pages
    if (n <= a.k) {
        for (int i = tid; i < a.k; i += kPickThreads) sel[i] = i < n ? i : -1;
        return;
    }
    const unsigned long long* keys = a.keys + (t * v.hkv + g) * v.max_pages;
    if (a.keys_in_smem) {
        for (int i = tid; i < n; i += kPickThreads) s_keys[i] = keys[i];
        keys = s_keys;
    }
    if (tid == 0) {
        s_prefix = 0;
        s_want = a.k;
        s_done = 0;
    }
    __syncthreads();
    int shift = 56;
    for (;; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        const unsigned long long prefix = s_prefix;
        for (int i = tid; i < n; i += kPickThreads) {
            const unsigned long long x = keys[i];
            if (shift == 56 || (x >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(int)(x >> shift) & 255], 1);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds digits 255 - 8 l .. 248 - 8 l: counts from the top
            int c = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) c += hist[255 - 8 * lane - i];
            int above = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += y;
            }
            above -= c;
            const int want = s_want;
            __syncwarp();
            if (above < want && above + c >= want) {
                int i = 0;
                while (above + hist[255 - 8 * lane - i] < want) above += hist[255 - 8 * lane - i++];
                const int digit = 255 - 8 * lane - i;
                s_prefix = prefix | ((unsigned long long)digit << shift);
                s_want = want - above;
                s_done = hist[digit] == want - above;        // the whole bucket is picked
            }
        }
        __syncthreads();
        if (shift == 0 || s_done) break;
    }
    // picked: keys whose digits so far are above the prefix, and the first s_want of those equal to it
    const unsigned long long edge = s_prefix >> shift;
    const int want = s_want;
    if (tid < 2) s_run[tid] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kPickThreads) {
        const int i = i0 + tid;
        const unsigned long long x = i < n ? keys[i] >> shift : 0;
        const bool gt = i < n && x > edge, eq = i < n && x == edge;
        const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            s_cnt[0][warp] = __popc(mg);
            s_cnt[1][warp] = __popc(me);
        }
        __syncthreads();
        int cg = s_run[0], ce = s_run[1];
        for (int w = 0; w < warp; ++w) {
            cg += s_cnt[0][w];
            ce += s_cnt[1][w];
        }
        cg += __popc(mg & ((1u << lane) - 1));
        ce += __popc(me & ((1u << lane) - 1));
        if (gt || (eq && ce < want)) sel[cg + min(ce, want)] = i;
        __syncthreads();
        if (tid == kPickThreads - 1) {
            s_run[0] = cg + (gt ? 1 : 0);
            s_run[1] = ce + (eq ? 1 : 0);
        }
        __syncthreads();
    }
}

constexpr size_t kPickSmem = 160 * 1024;

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" msa_status msa_page_select_workspace_size(int64_t n_tok, int hkv, int max_pages, size_t* bytes) {
    MSA_REQUIRE(bytes != nullptr, "msa_page_select_workspace_size: bytes is NULL");
    MSA_REQUIRE(n_tok >= 0 && n_tok < (int64_t)INT32_MAX / 2 && hkv > 0 && hkv <= 4096 && max_pages > 0,
                "msa_page_select_workspace_size: bad sizes");
    *bytes = align_up((size_t)n_tok * hkv * max_pages * sizeof(unsigned long long), 256);
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
    if (n_tok > 65535) return set_error(MSA_ERR_UNSUPPORTED, "msa_page_select: at most 65535 tokens a call");
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.n_tok = n_tok; a.tok_off = tok_off; a.max_new = max_new; a.k = k; a.recent = recent; a.sel = sel;
    a.keys = static_cast<unsigned long long*>(ws);
    a.err = device_error_word();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k < kv->max_pages) {
        const dim3 grid((unsigned)((kv->max_pages + kScorePages - 1) / kScorePages), (unsigned)kv->hkv, (unsigned)n_tok);
        switch (a.G) {
            case 1: page_score_kernel<1><<<grid, 256, 0, s>>>(a); break;
            case 2: page_score_kernel<2><<<grid, 256, 0, s>>>(a); break;
            case 4: page_score_kernel<4><<<grid, 256, 0, s>>>(a); break;
            default: page_score_kernel<8><<<grid, 256, 0, s>>>(a); break;
        }
        MSA_LAUNCH_CHECK();
    }
    size_t smem = (size_t)kv->max_pages * sizeof(unsigned long long);
    a.keys_in_smem = smem <= kPickSmem;
    if (!a.keys_in_smem) smem = 0;
    MSA_CUDA_TRY(cudaFuncSetAttribute(page_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPickSmem));
    page_pick_kernel<<<dim3((unsigned)n_tok, (unsigned)kv->hkv), kPickThreads, smem, s>>>(a);
    MSA_LAUNCH_CHECK();
    return MSA_OK;
}
