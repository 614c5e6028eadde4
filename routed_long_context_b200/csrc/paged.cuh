// The paged 8-bit key/value cache (msa_paged_kv): what its kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_fp16.h>

#include <cuda.h>

#include "common.cuh"

namespace msa {

constexpr int kPagedD = 128;             // head dimension
constexpr int kScaleMin = -50;           // range of the scale exponents; with both ends inside fp32's own
constexpr int kScaleMax = 50;            // range, scale and 1 / scale are exact and so is every product

struct PagedView {
    uint8_t* pages;                      // e4m3 [n_pages][2][hkv][page][128]
    float* scales;                       // [n_pages][2][hkv]
    __nv_bfloat16* bounds;               // [n_pages][hkv][2][128] or NULL
    const int32_t* table;                // [n_seq][max_pages]
    const int32_t* len;                  // [n_seq]
    int64_t n_pages;
    int n_seq, max_pages, page, shift, hkv;   // page = 1 << shift
};

// Checks what the host can see of a cache; `who` names the entry point in the message.
msa_status paged_view(const msa_paged_kv* kv, const char* who, PagedView* out);
// Checks of the arguments that every call on a cache takes.
msa_status paged_tokens_ok(const msa_paged_kv* kv, const char* who, int64_t n_tok, const int64_t* tok_off, int max_new);

// The new tokens of a sequence: rows t0 .. t0 + n_new - 1 of the packed buffers, the last n_new of its
// `len` cached tokens.
struct SeqSpan {
    int64_t t0;
    int n_new, len;
};
// False (with MSA_DEV_BAD_INDEX recorded) where offsets or length contradict the call's sizes: the sequence
// is then skipped by every kernel.
__device__ __forceinline__ bool seq_span(const PagedView& v, const int64_t* tok_off, int64_t n_tok,
                                         int max_new, int s, SeqSpan* sp, int* err) {
    const int64_t a = tok_off[s], b = tok_off[s + 1];
    const int64_t len = v.len[s];
    sp->t0 = a;
    sp->n_new = 0;
    sp->len = 0;
    if (a < 0 || b < a || b > n_tok || b - a > max_new || len < b - a || len > (int64_t)v.max_pages << v.shift) {
        record_device_error(err, MSA_DEV_BAD_INDEX);
        return false;
    }
    sp->n_new = (int)(b - a);
    sp->len = (int)len;
    return true;
}

// The sequence of packed row t: the last one that starts at or before it. Every lane of a warp takes part.
__device__ __forceinline__ int seq_of_token(const int64_t* tok_off, int n_seq, int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seq;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int s = lo + lane * step;
        const bool in = lane * step < n && tok_off[s] <= t;
        const int hit = 31 - __clz(__ballot_sync(0xffffffffu, in) | 1u);
        n = min(step, n - hit * step);
        lo += hit * step;
    }
    return lo;
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127
__device__ __forceinline__ int exponent_of(float pow2) { return (int)((__float_as_uint(pow2) >> 23) & 255u) - 127; }

// Exponent of the smallest power of two s with amax / s <= 448 = 1.75 * 2^8, by the bits of amax:
// amax = m 2^x with 1 <= m < 2 needs x - 8 where m <= 1.75 and x - 7 otherwise (also for subnormals, whose
// exponent field reads -127: they clamp to the smallest scale).
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(kScaleMin, min(kScaleMax, e));
}

// Two fp32 values to e4m3, to nearest even, saturating: the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t u) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A short kernel's launch costs as much as its work, so the attention kernels, their combine pass and the pick are
// launched while what comes before them in the stream still runs: a kernel lets the next one be launched once all of its
// own blocks have started (next_may_launch), and waits for the end of those before it where it first touches memory
// (every block does, so that an end means the end of all earlier ones too). One token over 777: 14.4 -> 13.4 us, 8
// sequences of up to 32 tokens over up to 8,096: 45 -> 42. Not so launched are the append and the page scores, nor
// what follows the pick before its end: blocks that start early pile up on the SMs that are free first (append, pick and
// attention of four tokens over 16,000 in a row 35 us so, 32 as it is).
__device__ __forceinline__ void next_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int block, size_t smem, cudaStream_t s, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- attention: how the work is cut ---------------------------------------------------------------
// A segment is one softmax: the query rows of one kv head that are handled together, over their keys. The
// segments' key tiles are numbered through (sequence, row block, kv head, tile) and the numbers cut into one
// contiguous range of equal length per CTA, so that lengths however far apart load every SM alike. A CTA that
// holds the whole of a segment writes its output; otherwise the pieces go to the workspace (slot 1 of the CTA
// in which the segment starts, slot 0 of those in which it goes on) and are joined by the combine pass.
struct PagedAttnArgs {
    PagedView v;
    const __nv_bfloat16* q;
    int64_t n_tok;
    const int64_t* tok_off;
    int max_new, G;
    const int32_t* sel;      // page lists [n_tok][hkv][k] or NULL
    int k;
    float scale_log2e;
    __nv_bfloat16* out;
    float* lse;
    int rows;                // rows of a workspace slot
    float* part_o;           // [CTA][2][rows][128], unnormalised
    float2* part_ml;         // [CTA][2][rows]: reference maximum (log2) and sum
    struct OpenSegment* open;  // [CTA]
    int stall;               // testing, where not 0: the loader brings nothing from tile (stall - 1) * one round of its slots on
    int* err;
};
struct OpenSegment {         // the segment that starts in a CTA and ends in a later one
    int64_t t0;              // first packed row
    int head, rows, n_more;  // kv head, query rows, later CTAs that hold pieces (0: there is no such segment)
    float unit;              // of the unnormalised output
};

// CTA i of n takes tiles total * i / n .. total * (i + 1) / n - 1; the one that holds tile x:
__device__ __forceinline__ int64_t cta_first(int64_t total, int n, int i) {
    if (total < (1 << 23)) return (uint32_t)total * (uint32_t)i / (uint32_t)n;       // n < 256; a 64-bit division is slow
    return total * i / n;
}
__device__ __forceinline__ int cta_of_tile(int64_t total, int n, int64_t x) {
    int i = (int)(x * n / total);
    while (cta_first(total, n, i + 1) <= x) ++i;
    while (cta_first(total, n, i) > x) --i;
    return i;
}

// The few-rows kernel (paged_decode.cu: blocks of 8 rows, tiles of 32 keys) and the many-rows kernel (paged_prompt.cu: 128
// or 256 rows, 128 keys).
constexpr int kDecodeRows = 8;
constexpr int kDecodeTile = 32;
// Few rows: where every segment can have a CTA of its own and none has more tiles than this, each has one (a segment that
// is cut costs its pieces' start and merge and the combine pass). 48 tokens of 4 heads over 194: 12 -> 9 us.
constexpr int kDecodeUncut = 32;
constexpr int kSegWeight = 8;        // what starting and ending a segment costs, in tiles, in either kernel
constexpr int kDecodeSeqs = 320;     // sequences that a CTA looks at together
constexpr int kPromptTile = 128;
constexpr int kPromptSeqs = 512;     // sequences per launch
msa_status launch_paged_decode(const PagedAttnArgs& a, int grid, cudaStream_t s);
// a.rows 128: 128-row blocks, keys shared by two warpgroups; 256: a row block of 128 each
msa_status launch_paged_prompt(const PagedAttnArgs& a, int grid, cudaStream_t s);

}  // namespace msa
