// select_experts.cu -- the choice of k experts per token from given logits: softmax or sigmoid
// scores, a bias for the choice alone, groups, top-k, weights.
// One warp per token, every value in FP64: scores and choice values in shared memory, the groups'
// values by one lane per group, then k rounds of a warp arg-max (lowest id first on equal values).
#include "block.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4, kMaxE = 1024;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ bool ahead(double c, int e, double d, int f) { return c > d || (c == d && e < f); }

__device__ __forceinline__ float load_logit(const SelectArgs& a, int64_t t, int e)
{
    return a.logits_f32 ? static_cast<const float*>(a.logits)[t * a.ld + e]
                        : bf16_to_f32(static_cast<const uint16_t*>(a.logits)[t * a.ld + e]);
}

__global__ void __launch_bounds__(kWarps * 32) k_select_experts(const SelectArgs a)
{
    __shared__ double c_s[kWarps][kMaxE];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.T) return;
    double* c = c_s[warp];
    const double ninf = -INFINITY, nan = NAN;

    float m = -INFINITY;
    double sum = 0.0;
    if (!a.sigmoid) {
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load_logit(a, t, e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        for (int e = lane; e < a.E; e += 32) {
            const float l = load_logit(a, t, e);
            if (l > -INFINITY) sum += l == m ? 1.0 : exp(static_cast<double>(l) - static_cast<double>(m));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    }
    auto score = [&](float l) {
        if (!(l > -INFINITY)) return 0.0;
        if (a.sigmoid) return 1.0 / (1.0 + exp(-static_cast<double>(l)));
        return (l == m ? 1.0 : exp(static_cast<double>(l) - static_cast<double>(m))) / sum;
    };
    for (int e = lane; e < a.E; e += 32) {
        const float l = load_logit(a, t, e);
        // without a bias the logits themselves give the order, also where two scores round to one number
        const double v = a.bias ? score(l) + static_cast<double>(a.bias[e]) : static_cast<double>(l);
        c[e] = l > -INFINITY && v > ninf ? v : ninf;
    }
    __syncwarp();
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
        double v1 = ninf, v2 = ninf;
        if (lane < a.n_group)
            for (int i = 0; i < size; ++i) {
                const double v = c[lane * size + i];
                if (v > v1) {
                    v2 = v1;
                    v1 = v;
                } else if (v > v2)
                    v2 = v;
            }
        double gv = v1;
        if (a.group_top2 && v1 > ninf) {
            const double s1 = a.bias ? v1 : score(static_cast<float>(v1));
            gv = v2 > ninf ? s1 + (a.bias ? v2 : score(static_cast<float>(v2))) : s1;
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const double o = __shfl_sync(kFull, gv, g);
            rank += g != lane && ahead(o, g, gv, lane);
        }
        const unsigned keep = __ballot_sync(kFull, lane < a.n_group && rank < a.topk_group);
        for (int e = lane; e < a.E; e += 32)
            if (!((keep >> (e / size)) & 1u)) c[e] = nan;
        __syncwarp();
    }
    int my_id = 0;
    double my_s = 0.0, total = 0.0;
    for (int j = 0; j < a.k; ++j) {
        double best = nan;
        int at = kMaxE;
        for (int e = lane; e < a.E; e += 32)
            if (c[e] == c[e] && (at == kMaxE || c[e] > best)) {
                best = c[e];
                at = e;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ob = __shfl_xor_sync(kFull, best, o);
            const int oa = __shfl_xor_sync(kFull, at, o);
            if (oa < kMaxE && (at == kMaxE || ahead(ob, oa, best, at))) {
                best = ob;
                at = oa;
            }
        }
        const double s = best > ninf ? score(load_logit(a, t, at)) : 0.0;
        total += s;
        if (lane == j) {
            my_id = at;
            my_s = s;
        }
        __syncwarp();
        if (lane == (at & 31)) c[at] = nan;
        __syncwarp();
    }
    if (lane < a.k) {
        if (a.renormalize) my_s = total > 0.0 ? my_s / total : 0.0;
        a.ids[t * a.k + lane] = my_id;
        a.w[t * a.k + lane] = static_cast<float>(my_s * a.scale);
    }
}

}  // namespace

cudaError_t launch_select_experts(const SelectArgs& a, cudaStream_t stream)
{
    if (a.T <= 0) return cudaSuccess;
    return launch_pdl(k_select_experts, dim3((a.T + kWarps - 1) / kWarps), dim3(kWarps * 32), 0, stream, a);
}

}  // namespace moe
