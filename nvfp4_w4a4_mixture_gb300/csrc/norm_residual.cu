// norm_residual.cu -- the norms on both sides of a block with its gate and residual scale:
//   u = y or y * rsqrt(mean(y^2) + eps) * (off + w_post);  r' = alpha r + g u;
//   x' = r' * rsqrt(mean(r'^2) + eps) * (off + w_pre)
// One CTA per token row; the row stays in shared memory as FP32 between the steps.
#include "block.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256, kMaxH = 8192;

__device__ __forceinline__ float load_any(const void* p, int64_t i, bool f32)
{
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__device__ float block_sum(float v, float* red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += red[i];
    return s;
}

__global__ void __launch_bounds__(kThreads) k_norm_residual(const NormArgs a)
{
    __shared__ float row[kMaxH];
    __shared__ float red[kThreads / 32];
    ptx::griddep_wait();
    const int64_t t = blockIdx.x;
    float inv = 1.0f;
    if (a.w_post) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.H; c += kThreads) {
            const float v = bf16_to_f32(a.y[t * a.ld_y + c]);
            s += v * v;
        }
        inv = rsqrtf(block_sum(s, red) / a.H + a.eps);
    }
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.H; c += kThreads) {
        float r = a.res ? a.res_scale * load_any(a.res, t * a.ld_res + c, a.res_f32) : 0.0f;
        if (a.y) {
            float u = bf16_to_f32(a.y[t * a.ld_y + c]);
            if (a.w_post) u = u * inv * (a.w_offset + bf16_to_f32(a.w_post[c]));
            if (a.gate) u *= load_any(a.gate, t * a.gate_ld + (a.gate_per_channel ? c : 0), a.gate_f32);
            r += u;
        }
        row[c] = r;
        s += r * r;
    }
    inv = rsqrtf(block_sum(s, red) / a.H + a.eps);
    for (int c = threadIdx.x; c < a.H; c += kThreads) {
        if (a.res_out) {
            if (a.res_f32) static_cast<float*>(a.res_out)[t * a.ld_res_out + c] = row[c];
            else static_cast<uint16_t*>(a.res_out)[t * a.ld_res_out + c] = static_cast<uint16_t>(pack_bf16x2(row[c], 0.0f));
        }
        if (a.x_out)
            a.x_out[t * a.ld_x + c] =
                static_cast<uint16_t>(pack_bf16x2(row[c] * inv * (a.w_offset + bf16_to_f32(a.w_pre[c])), 0.0f));
    }
}

}  // namespace

cudaError_t launch_norm_residual(const NormArgs& a, cudaStream_t stream)
{
    if (a.T <= 0) return cudaSuccess;
    return launch_pdl(k_norm_residual, dim3(a.T), dim3(kThreads), 0, stream, a);
}

}  // namespace moe
