// quantize_fp8.cu -- FP8 encoding of rows with a scale for each 128 elements: s = max |x| / 448, code = E4M3(x / s).
// A block is in the registers of 8 or 16 lanes; its maximum comes by shuffles. x is read once, codes and scales are written
// once; for the quotients it is bound by instruction issue before memory.
// Measured: 16,384 x 2,064 23.6 us, 4.3 TB/s (29 with a division for every quotient; with CTAs that stay and the next
// blocks' loads in flight 34 to 46: fewer warps); 4 x 2,048 1.7 us.
#include "attention.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t codes_of_pair(uint64_t v)
{
    return ptx::cvt_e4m3x2(lo_of(v), hi_of(v));
}

// kLanes lanes (8 or 16) take kBlocks blocks, kGroups apart, whose loads are in flight together; a lane has two pieces or one
// of 16 bytes of each, kLanes pieces apart. A step of kGroups blocks is step_rows rows and step_cols blocks, with a carry.
template <int kLanes, int kBlocks>
__global__ void __launch_bounds__(kThreads, 6) k_quantize_fp8(const uint16_t* __restrict__ x, int64_t ld_x, int T, int K, int blocks, int step_rows,
                                                              int step_cols, uint8_t* __restrict__ codes, float* __restrict__ scale)
{
    constexpr int kGroups = kThreads / kLanes, kPieces = 16 / kLanes, kApart = kLanes * 8;  // elements between two pieces
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int at = threadIdx.x % kLanes;
    const int64_t first = blockIdx.x * static_cast<int64_t>(kBlocks * kGroups) + threadIdx.x / kLanes;
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
    uint4 v[kBlocks][kPieces];
    int64_t row[kBlocks];
    int col[kBlocks];  // the lane's first piece; K: nothing there
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        const int c = t < T ? b * 128 + at * 8 : K;
#pragma unroll
        for (int h = 0; h < kPieces; ++h)
            v[i][h] = c + h * kApart < K ? __ldcs(reinterpret_cast<const uint4*>(x + t * ld_x + c + h * kApart)) : make_uint4(0, 0, 0, 0);
        row[i] = t;
        col[i] = c;
        t += step_rows;
        b += step_cols;
        if (b >= blocks) {
            b -= blocks;
            ++t;
        }
    }
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        uint32_t w[4 * kPieces];
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            w[4 * h] = v[i][h].x;
            w[4 * h + 1] = v[i][h].y;
            w[4 * h + 2] = v[i][h].z;
            w[4 * h + 3] = v[i][h].w;
        }
        // the largest magnitude by its bits: in their order an infinity is above all numbers and a NaN above that
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4 * kPieces; ++j) m = max(m, max(w[j] << 16 & 0x7FFF0000u, w[j] & 0x7FFF0000u));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float s = m ? __fdiv_rn(__uint_as_float(m), 448.0f) : 1.0f;
        // Codes of RN(x / s). 1 / s less and plus 2^-21 of it are further apart than all roundings here: where the products
        // with both have one code, so has the quotient between them; else (some 4 in 1,000, on or near the middle between
        // two codes) the two are divided.
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));  // off by 2^-23 of it at most
        // the largest outside [2^-100, 2^100): s or 1 / s may leave FP32's normal numbers, and all is divided: products with
        // NaN and with 0 differ but of an infinity or a NaN, whose code (of x / inf, or x / NaN) is that of NaN
        const bool near = m - 0x0D800000u < 0x64000000u;
        const float below = near ? r * (1.0f - 0x1p-21f) : __uint_as_float(0x7FC00000u), above = near ? r * (1.0f + 0x1p-21f) : 0.0f;
        const uint64_t below2 = pair(below, below), above2 = pair(above, above);
        uint32_t q[4 * kPieces];
#pragma unroll
        for (int j = 0; j < 4 * kPieces; ++j) {
            const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
            q[j] = codes_of_pair(mul2(pair(lo, hi), below2));
            if (q[j] != codes_of_pair(mul2(pair(lo, hi), above2))) q[j] = ptx::cvt_e4m3x2(__fdiv_rn(lo, s), __fdiv_rn(hi, s));
        }
        uint8_t* const to = codes + row[i] * K + col[i];
#pragma unroll
        for (int h = 0; h < kPieces; ++h)
            if (col[i] + h * kApart < K) *reinterpret_cast<uint2*>(to + h * kApart) = make_uint2(q[4 * h] | q[4 * h + 1] << 16, q[4 * h + 2] | q[4 * h + 3] << 16);
        if (at == 0 && col[i] < K) scale[row[i] * blocks + col[i] / 128] = s;
    }
}

}  // namespace

cudaError_t launch_quantize_fp8(const uint16_t* x, int64_t ld_x, int T, int K, uint8_t* codes, float* scale, int sms, cudaStream_t stream)
{
    const int blocks = (K + 127) / 128;
    const int64_t n = static_cast<int64_t>(T) * blocks;
    // Many: eight lanes a block, two blocks in flight (a block's scale and shuffles then are for twice the elements a lane:
    // 16,384 x 2,064 23.6 us, 26.4 with 16 lanes); few: 16 lanes (4 x 2,048 1.7 us, 2.1 with eight).
    const bool many = n >= 64LL * 4 * sms;
    const int groups = kThreads / (many ? 8 : 16);
    const int64_t each = (many ? 2 : 1) * groups, ctas = (n + each - 1) / each;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(many ? k_quantize_fp8<8, 2> : k_quantize_fp8<16, 1>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, x, ld_x, T,
                      K, blocks, groups / blocks, groups % blocks, codes, scale);
}

}  // namespace moe
