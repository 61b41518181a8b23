// adapters.cu -- low-rank adapters of many requests: out[t] = y[t] + scale_a B_a (A_a x[t]).
// One CTA per token: the request's adapter by a binary search of the offsets, A_a x by one warp per
// rank row into shared memory (FP32), then one thread per output column.
#include "block.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// the last s in [0, S) with off[s] <= t, or -1
__device__ __forceinline__ int segment_of(const int32_t* off, int S, int t)
{
    int lo = 0, hi = S;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (off[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

__global__ void __launch_bounds__(kThreads) k_adapter_add(const AdapterArgs p)
{
    __shared__ float h[kAdapterMaxRank];
    ptx::griddep_wait();
    if (blockIdx.x == 0) {
        bool bad = p.seg_offsets[0] != 0 || p.seg_offsets[p.S] != p.T;
        for (int i = threadIdx.x; i < p.S; i += kThreads)
            bad |= p.seg_offsets[i] > p.seg_offsets[i + 1] || p.seg_adapter[i] < -1 || p.seg_adapter[i] >= p.n;
        if (bad) record_status(p.status, kDevBadSegment);
    }
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = segment_of(p.seg_offsets, p.S, t);
    const int end = s >= 0 ? p.seg_offsets[s + 1] : 0;
    const int ad = t < end && end <= p.T && p.seg_offsets[s] >= 0 ? p.seg_adapter[s] : -2;
    if (ad < -1 || ad >= p.n) return;
    const uint16_t* x = p.x + t * p.ld_x;
    if (ad >= 0)
        for (int j = warp; j < p.r; j += kThreads / 32) {
            const uint16_t* row = p.a + (static_cast<int64_t>(ad) * p.r + j) * p.K;
            float v = 0.0f;
            for (int c = lane; c < p.K; c += 32) v += bf16_to_f32(x[c]) * bf16_to_f32(row[c]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0) h[j] = v * p.scale[ad];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < p.N; c += kThreads) {
        float v = bf16_to_f32(p.y[t * p.ld_y + c]);
        if (ad >= 0) {
            const uint16_t* row = p.b + (static_cast<int64_t>(ad) * p.N + c) * p.r;
            float d = 0.0f;
            for (int j = 0; j < p.r; ++j) d += h[j] * bf16_to_f32(row[j]);
            v += d;
        }
        p.out[t * p.ld_out + c] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
    }
}

}  // namespace

cudaError_t launch_adapter_add(const AdapterArgs& a, int, cudaStream_t stream)
{
    if (a.T <= 0) return cudaSuccess;
    return launch_pdl(k_adapter_add, dim3(a.T), dim3(kThreads), 0, stream, a);
}

}  // namespace moe
