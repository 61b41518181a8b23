// quantize_fp8.cu -- FP8 encoding of rows with a scale for each 128 elements: s = max |x| / 448, code = E4M3(x / s).
// A block is in the registers of 16 lanes (16 bytes of bf16 each); its maximum comes by shuffles. x is read once, codes
// and scales are written once; with eight quotients a lane it is bound by instruction issue before memory.
// Measured: 16,384 x 2,064 26.4 us, 3.9 TB/s; with a division for every quotient 29, with CTAs that stay and the next blocks'
// loads in flight 34 to 46 (fewer warps); 4 x 2,048 1.7 us.
#include "attention.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256, kGroups = kThreads / 16;

__device__ __forceinline__ uint64_t pair(float lo, float hi) { return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t codes_of_pair(uint64_t v)
{
    return ptx::cvt_e4m3x2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

// 16 lanes take kBlocks blocks, kGroups apart, whose loads are in flight together. A step of kGroups blocks is step_rows
// rows and step_cols blocks, with a carry.
template <int kBlocks>
__global__ void __launch_bounds__(kThreads, 6) k_quantize_fp8(const uint16_t* __restrict__ x, int64_t ld_x, int T, int K, int blocks, int step_rows,
                                                           int step_cols, uint8_t* __restrict__ codes, float* __restrict__ scale)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int at = threadIdx.x % 16;
    const int64_t first = blockIdx.x * static_cast<int64_t>(kBlocks * kGroups) + threadIdx.x / 16;
    int64_t t;
    int b;
    if (first >> 32) {
        t = first / blocks;
        b = static_cast<int>(first - t * blocks);
    } else {  // (32 bits where they do)
        const uint32_t r = static_cast<uint32_t>(first) / static_cast<uint32_t>(blocks);
        t = r;
        b = static_cast<int>(static_cast<uint32_t>(first) - r * static_cast<uint32_t>(blocks));
    }
    uint4 v[kBlocks];
    int64_t row[kBlocks];
    int col[kBlocks];  // -1: nothing there
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int c = b * 128 + at * 8;
        const bool in = t < T && c < K;
        v[i] = in ? __ldcs(reinterpret_cast<const uint4*>(x + t * ld_x + c)) : make_uint4(0, 0, 0, 0);
        row[i] = t;
        col[i] = in ? c : -1;
        t += step_rows;
        b += step_cols;
        if (b >= blocks) {
            b -= blocks;
            ++t;
        }
    }
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        // the largest magnitude by its bits: in their order an infinity is above all numbers and a NaN above that
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max(w[j] << 16 & 0x7FFF0000u, w[j] & 0x7FFF0000u));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float s = m ? __fdiv_rn(__uint_as_float(m), 448.0f) : 1.0f;
        // Codes of RN(x / s). 1 / s less and plus 2^-21 of it are further apart than all roundings here: where the products
        // with both have one code, so has the quotient between them; else (some 4 in 1,000, on or near the middle between
        // two codes) the two are divided.
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));  // off by 2^-23 of it at most
        // the largest outside [2^-100, 2^100): s or 1 / s may leave FP32's normal numbers, and all is divided
        const float below = m - 0x0D800000u < 0x64000000u ? r * (1.0f - 0x1p-21f) : __uint_as_float(0x7FC00000u), above = r * (1.0f + 0x1p-21f);
        const uint64_t below2 = pair(below, below), above2 = pair(above, above);
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
            q[j] = codes_of_pair(mul2(pair(lo, hi), below2));
            if (q[j] != codes_of_pair(mul2(pair(lo, hi), above2))) q[j] = ptx::cvt_e4m3x2(__fdiv_rn(lo, s), __fdiv_rn(hi, s));
        }
        if (col[i] >= 0) {
            *reinterpret_cast<uint2*>(codes + row[i] * K + col[i]) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
            if (at == 0) scale[row[i] * blocks + col[i] / 128] = s;
        }
    }
}

}  // namespace

cudaError_t launch_quantize_fp8(const uint16_t* x, int64_t ld_x, int T, int K, uint8_t* codes, float* scale, int sms, cudaStream_t stream)
{
    const int blocks = (K + 127) / 128;
    const int64_t n = static_cast<int64_t>(T) * blocks;
    // four blocks in flight where all multiprocessors have some warps of them (4 x 2,048 took 3.1 us with four, 1.7 with one)
    const bool many = n >= 4LL * kGroups * 4 * sms;
    const int64_t each = (many ? 4 : 1) * kGroups, ctas = (n + each - 1) / each;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(many ? k_quantize_fp8<4> : k_quantize_fp8<1>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, x, ld_x, T, K,
                      blocks, kGroups / blocks, kGroups % blocks, codes, scale);
}

}  // namespace moe
