// norm_residual.cu -- the norms on both sides of a block with its gate and residual scale:
//   u = y or y * rsqrt(mean(y^2) + eps) * (off + w_post);  r' = alpha r + g u;
//   x' = r' * rsqrt(mean(r'^2) + eps) * (off + w_pre)
// Bounded by memory: y, r and a gate per element are read once, r' and x' written once. A row stays
// in the registers of kThreads threads (kVec 16-byte vectors of bf16 a thread) from its loads to its
// stores. The CTAs stay and walk the rows; a row's loads are issued before the two reductions of the
// row before it, so that they are in flight meanwhile.
// Measured: 16,384 x 2048 with a gate per channel 44.4 us, 6.05 TB/s (90 % of what a copy reaches);
// 12,365 x 2056 with a gate per element 41.6 us (91 %); 4 x 2048 1.6 us.
#include "block.cuh"

namespace moe {

namespace {

enum GateKind : int { kGateScalar = 0, kGateBF16 = 1, kGateF32 = 2 };  // scalar: one value a row, or none

// eight values: bf16 in one 16-byte vector, FP32 in two
template <bool F32>
struct Vec8 {
    uint4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t i)
    {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (F32 ? 4 : 2));
        v[0] = __ldcs(q);
        if constexpr (F32) v[1] = __ldcs(q + 1);
    }
    __device__ __forceinline__ void zero()
    {
        v[0] = make_uint4(0, 0, 0, 0);
        if constexpr (F32) v[1] = v[0];
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (F32) {
            const uint4& q = v[i / 4];
            return __uint_as_float(i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w);
        } else {
            const uint32_t w = i / 2 == 0 ? v[0].x : i / 2 == 1 ? v[0].y : i / 2 == 2 ? v[0].z : v[0].w;
            return i % 2 ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
        }
    }
};

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// The sum of v over the threads of a row; red: a slot that neither the row's other reduction nor the
// row before uses (a slower warp may still read that).
template <int kThreads>
__device__ __forceinline__ float row_sum(float v, float* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (kThreads > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) v += red[w];
    }
    return v;
}

// What a row reads.
template <int kVec, bool kResF32, int kGate>
struct Row {
    Vec8<false> y[kVec];
    Vec8<kResF32> r[kVec];
    Vec8<kGate == kGateF32> g[kGate == kGateScalar ? 1 : kVec];
    float gate;

    template <int kThreads>
    __device__ __forceinline__ void load(const NormArgs& a, int64_t t, int at)
    {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = (i * kThreads + at) * 8;
            const bool in = c < a.H;
            if (in && a.y) y[i].load(a.y, t * a.ld_y + c);
            else y[i].zero();
            if (in && a.res) r[i].load(a.res, t * a.ld_res + c);
            else r[i].zero();
            if constexpr (kGate != kGateScalar) {
                if (in) g[i].load(a.gate, t * a.gate_ld + c);
                else g[i].zero();
            }
        }
        gate = 1.0f;
        if constexpr (kGate == kGateScalar)
            if (a.gate)
                gate = a.gate_f32 ? static_cast<const float*>(a.gate)[t * a.gate_ld]
                                  : bf16_to_f32(static_cast<const uint16_t*>(a.gate)[t * a.gate_ld]);
    }
};

// kThreads threads a row; 32: four rows a CTA, one a warp.
template <int kThreads, int kVec, bool kResF32, int kGate>
__global__ void __launch_bounds__(kThreads == 32 ? 128 : kThreads) k_norm_residual(const __grid_constant__ NormArgs a)
{
    constexpr int kRows = kThreads == 32 ? 4 : 1;
    constexpr bool kKeep = kVec <= 2;  // the weights stay in registers, else they come from L1 for each row
    __shared__ float red[2][2][kThreads / 32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int at = threadIdx.x % kThreads;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kThreads;
    if (t >= a.T) return;
    const float inv_h = 1.0f / static_cast<float>(a.H);
    auto weight = [&](const uint16_t* w, int i) {
        Vec8<false> v;
        const int c = (i * kThreads + at) * 8;
        v.zero();
        if (w && c < a.H) v.v[0] = __ldg(reinterpret_cast<const uint4*>(w + c));
        return v;
    };
    Vec8<false> w_post[kKeep ? kVec : 1], w_pre[kKeep ? kVec : 1];
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            w_post[i] = weight(a.w_post, i);
            w_pre[i] = weight(a.w_pre, i);
        }
    }
    Row<kVec, kResF32, kGate> cur;
    cur.template load<kThreads>(a, t, at);
    for (int parity = 0;; parity ^= 1) {
        float post = 1.0f;
        if (a.w_post) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += cur.y[i].get(e) * cur.y[i].get(e);
            post = rsqrtf(row_sum<kThreads>(s, red[0][parity]) * inv_h + a.eps);
        }
        float r[kVec][8], s = 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const Vec8<false> w = kKeep ? w_post[kKeep ? i : 0] : weight(a.w_post, i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u = cur.y[i].get(e);
                if (a.w_post) u = u * post * (a.w_offset + w.get(e));
                if constexpr (kGate == kGateScalar) u *= cur.gate;
                else u *= cur.g[i].get(e);
                r[i][e] = a.res_scale * cur.r[i].get(e) + u;
                s += r[i][e] * r[i][e];
            }
        }
        const int64_t next = t + step;
        if (next < a.T) cur.template load<kThreads>(a, next, at);
        if (a.res_out) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int c = (i * kThreads + at) * 8;
                if (c < a.H) {
                    if constexpr (kResF32) {
                        float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + t * a.ld_res_out + c);
                        d[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
                        d[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
                    } else {
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + t * a.ld_res_out + c) = pack8(r[i]);
                    }
                }
            }
        }
        if (a.x_out) {
            const float pre = rsqrtf(row_sum<kThreads>(s, red[1][parity]) * inv_h + a.eps);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const Vec8<false> w = kKeep ? w_pre[kKeep ? i : 0] : weight(a.w_pre, i);
                const int c = (i * kThreads + at) * 8;
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = r[i][e] * pre * (a.w_offset + w.get(e));
                if (c < a.H) *reinterpret_cast<uint4*>(a.x_out + t * a.ld_x + c) = pack8(x);
            }
        }
        t = next;
        if (t >= a.T) break;
    }
}

template <int kThreads, int kVec, bool kResF32, int kGate>
cudaError_t launch(const NormArgs& a, int sms, cudaStream_t stream)
{
    constexpr int threads = kThreads == 32 ? 128 : kThreads, rows = kThreads == 32 ? 4 : 1;
    static int per_sm = 0;
    if (per_sm == 0) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_norm_residual<kThreads, kVec, kResF32, kGate>, threads, 0);
        if (e != cudaSuccess) return e;
    }
    const int64_t need = (static_cast<int64_t>(a.T) + rows - 1) / rows, room = static_cast<int64_t>(sms) * per_sm;
    return launch_pdl(k_norm_residual<kThreads, kVec, kResF32, kGate>, dim3(static_cast<unsigned>(need < room ? need : room)), dim3(threads),
                      0, stream, a);
}

template <bool kResF32, int kGate>
cudaError_t launch_h(const NormArgs& a, int sms, cudaStream_t stream)
{
    const int n = (a.H + 7) / 8;  // 16-byte vectors of a bf16 row
    if (n <= 32) return launch<32, 1, kResF32, kGate>(a, sms, stream);
    if (n <= 64) return launch<32, 2, kResF32, kGate>(a, sms, stream);
    if (a.T <= 2 * sms) {
        // Few rows: a row's own chain counts, so two vectors a thread (4 x 4096 1.8 us; 128 threads with four 2.5).
        if (n <= 128) return launch<128, 1, kResF32, kGate>(a, sms, stream);
        if (n <= 256) return launch<128, 2, kResF32, kGate>(a, sms, stream);
        if (n <= 512) return launch<256, 2, kResF32, kGate>(a, sms, stream);
        return launch<512, 2, kResF32, kGate>(a, sms, stream);
    }
    // Many rows: the bytes in flight count, so threads without a vector cost (65,536 x 512 in 32 threads with two
    // 43.0 us, in 128 with one, half of them idle, 57.6) and fewer warps wait on one another with three or four
    // vectors a thread (4096 x 8192 45.5 us in 256 threads, 54.4 in 512; 16,320 x 2056 44.6 in 96, 47.0 in 128,
    // 55.7 in 192; 52,428 x 640 44.6 in 32, 53.7 in 128). FP32 residuals gain less (8192: 68.2 against 70.1).
    if (n <= 96) return launch<32, 3, kResF32, kGate>(a, sms, stream);
    if (n <= 128) return launch<128, 1, kResF32, kGate>(a, sms, stream);
    if (n <= 160) return launch<64, 3, kResF32, kGate>(a, sms, stream);
    if (n <= 192) return launch<96, 2, kResF32, kGate>(a, sms, stream);
    if (n <= 256) return launch<128, 2, kResF32, kGate>(a, sms, stream);
    if (n <= 288) return launch<96, 3, kResF32, kGate>(a, sms, stream);
    if (n <= 384) return launch<128, 3, kResF32, kGate>(a, sms, stream);
    if (n <= 576) return launch<192, 3, kResF32, kGate>(a, sms, stream);
    if (n <= 768) return launch<256, 3, kResF32, kGate>(a, sms, stream);
    return launch<256, 4, kResF32, kGate>(a, sms, stream);
}

template <bool kResF32>
cudaError_t launch_res(const NormArgs& a, int sms, cudaStream_t stream)
{
    if (!a.gate || !a.gate_per_channel) return launch_h<kResF32, kGateScalar>(a, sms, stream);
    return a.gate_f32 ? launch_h<kResF32, kGateF32>(a, sms, stream) : launch_h<kResF32, kGateBF16>(a, sms, stream);
}

}  // namespace

cudaError_t launch_norm_residual(const NormArgs& a, int sms, cudaStream_t stream)
{
    if (a.T <= 0) return cudaSuccess;
    return a.res_f32 ? launch_res<true>(a, sms, stream) : launch_res<false>(a, sms, stream);
}

}  // namespace moe
