// attention.cuh -- internal launchers of the attention half of a block: appends to a paged cache with norm and rotation,
// attention over that cache, FP8 encoding and products (not part of the C ABI).
#pragma once
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "kernels.cuh"

namespace moe {

// Device status bits of these calls (the workspace header's status word).
enum : int {
    kDevBadRequest = 64,       // seg_offsets or kv_len outside its range
    kDevBadPage = 128,         // a page id outside [0, n_pages)
    kDevTimeoutGemmFp8 = 256,  // a bounded wait of the FP8 GEMM ran out
    kDevTimeoutAttention = 512,  // a bounded wait of the attention ran out
};

// ---- two FP32 values an instruction
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo); }
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct KvCache {
    void *k, *v;
    bool e4m3;
    int n_pages, page_log2, n_kv, D;
    int64_t ld_page, ld_slot, ld_head;  // elements
    const float *k_scale, *v_scale;     // nullable
};

struct Requests {
    int S;
    const int32_t *seg_offsets, *kv_len, *pages;
    int64_t ld_pages;
    int64_t max_len;  // max_pages * page_size
};

struct Request {
    int beg, n, len;  // first row, rows (0: broken or empty), tokens with them
};

// Request s of a batch of T rows. bad: it breaks the rules (then it has no rows).
__device__ __forceinline__ Request load_request(const Requests& r, int s, int T, int max_new, bool& bad)
{
    const int beg = __ldg(r.seg_offsets + s), end = __ldg(r.seg_offsets + s + 1), len = __ldg(r.kv_len + s);
    bad = beg < 0 || beg > end || end > T || (s == 0 && beg != 0) || len < 0 || len > r.max_len || end - beg > max_new;
    return Request{beg, bad ? 0 : end - beg, len};
}

// The last request whose rows begin at or before row t (-1: none), where the offsets are in order; else some request, whose
// rows may begin behind t. Warp-wide; lanes look at 32 offsets at a time.
__device__ __forceinline__ int find_request(const int32_t* off, int S, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = S + 1;  // off[lo] <= t, once that was seen for lo = 0
    bool first = true;
    while (first || hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, i < hi && __ldg(off + min(i, S)) <= t);
        const int k = __popc(m);
        if (first && k == 0) return -1;
        first = false;
        lo += (max(k, 1) - 1) * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

// ---- cache_append.cu
struct AppendArgs {
    KvCache c;
    Requests r;
    int T, n_q, rot;
    bool interleaved;
    const float* inv_freq;
    const uint16_t *w_q, *w_k;  // nullable
    float eps, w_offset;
    const uint16_t *q, *k, *v;
    int64_t ld_q, ld_k, ld_v;
    uint16_t* q_out;
    int64_t ld_q_out;
    int* status;
};
cudaError_t launch_cache_append(const AppendArgs& a, int sms, cudaStream_t stream);

// ---- paged_attention.cu
struct AttentionArgs {
    KvCache c;
    Requests r;
    int T, n_q, group, max_new, window;
    unsigned group_mul;  // ceil(2^16 / group): (row * group_mul) >> 16 is row / group for row * 63 < 2^16
    float scale;
    const uint16_t* q;
    int64_t ld_q;
    uint16_t* out;
    int64_t ld_out;
    float* lse;       // nullable
    int64_t* prefix;  // [S + 3] units before each request, their number, and how they are cut (workspace)
    float* part;      // partial sums (workspace)
    float* part_ml;   // their maxima and weights (workspace)
    int* status;
    const WsHeader* hooks;  // the workspace header whose test_* fields the first wait reads
};
namespace attention {
// The rows of a unit in eights: what max_new tokens of a key head's queries need, at most eight.
inline int row_eights(int group, int max_new)
{
    const int rows = group * max_new;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : rows <= 32 ? 4 : 8;
}

// The most CTAs of the main launch; each has two places for partial sums.
inline int ctas_most(int sms) { return sms * 3; }
}  // namespace attention
size_t attention_workspace_bytes(int S, int n_q, int n_kv, int D, int max_new, int sms);
cudaError_t launch_paged_attention(AttentionArgs a, void* ws, int sms, cudaStream_t stream);

// ---- quantize_fp8.cu
cudaError_t launch_quantize_fp8(const uint16_t* x, int64_t ld_x, int T, int K, uint8_t* codes, float* scale, int sms, cudaStream_t stream);

// ---- gemm_fp8.cu
struct GemmFp8Args {
    int T, N, K;
    const uint8_t *a, *b;
    const float *a_scale, *b_scale;
    void* out;
    bool out_f32;
    int64_t ld_out;
    int* status;
    const WsHeader* hooks;  // the workspace header whose test_* fields the first wait reads
};
cudaError_t launch_gemm_fp8(const GemmFp8Args& a, int sms, cudaStream_t stream);

// Dynamic shared memory beyond 48 KB for a kernel, asked for once on each device. done: a bit for each.
inline cudaError_t allow_smem(std::atomic<uint64_t>& done, const void* kernel, size_t bytes)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done.load(std::memory_order_relaxed) >> dev & 1)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

// ---- api.cu
// The map of an output of rows ld elements apart that is stored in boxes (128-byte swizzle).
CUresult encode_tmap_2d_out(CUtensorMap* map, void* base, bool f32, uint64_t inner, uint64_t outer, uint64_t ld, uint32_t box_inner,
                            uint32_t box_outer);

}  // namespace moe
