// quantize_fp8.cu -- FP8 encoding of rows with a scale for each 128 elements: s = max |x| / 448, code = E4M3(x / s).
// A block is in the registers of 16 lanes (16 bytes of bf16 each); its maximum comes by shuffles. Bounded by memory:
// x is read once, codes and scales are written once.
#include "attention.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) k_quantize_fp8(const uint16_t* __restrict__ x, int64_t ld_x, int K, int blocks, int64_t n_blocks,
                                                           uint8_t* __restrict__ codes, float* __restrict__ scale)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int at = threadIdx.x % 16;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 16);
    // every lane of a warp runs as many turns as its first (the shuffles need them all)
    const int64_t first = blockIdx.x * static_cast<int64_t>(kThreads / 16) + threadIdx.x / 16;
    for (int64_t g = first; g - (threadIdx.x / 16) % 2 < n_blocks; g += step) {
        const int64_t t = g / blocks;
        const int b = static_cast<int>(g - t * blocks), c = b * 128 + at * 8;
        const bool in = g < n_blocks && c < K;
        const uint4 v = in ? __ldcs(reinterpret_cast<const uint4*>(x + t * ld_x + c)) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        // the largest magnitude by its bits: in their order an infinity is above all numbers and a NaN above that
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7FFF0000u, w[i] & 0x7FFF0000u));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float s = m ? __fdiv_rn(__uint_as_float(m), 448.0f) : 1.0f;
        if (in) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = ptx::cvt_e4m3x2(__fdiv_rn(__uint_as_float(w[i] << 16), s), __fdiv_rn(__uint_as_float(w[i] & 0xFFFF0000u), s));
            *reinterpret_cast<uint2*>(codes + t * K + c) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
            if (at == 0) scale[g] = s;
        }
    }
}

}  // namespace

cudaError_t launch_quantize_fp8(const uint16_t* x, int64_t ld_x, int T, int K, uint8_t* codes, float* scale, int sms, cudaStream_t stream)
{
    const int blocks = (K + 127) / 128;
    const int64_t n = static_cast<int64_t>(T) * blocks, ctas = (n + kThreads / 16 - 1) / (kThreads / 16);
    const int grid = static_cast<int>(ctas < sms * 8LL ? ctas : sms * 8LL);
    return launch_pdl(k_quantize_fp8, dim3(grid), dim3(kThreads), 0, stream, x, ld_x, K, blocks, n, codes, scale);
}

}  // namespace moe
