// select_experts.cu -- the choice of k experts per token from given logits: softmax or sigmoid
// scores, a bias for the choice alone, groups, top-k, weights.
//
// kL lanes a token: 16 (two tokens a warp) for many tokens and up to 256 experts, else 32.
// The E choice values c are in registers (kNper a lane). Without a bias c is the logit itself (a larger
// logit is a larger score), so the order is exact; with one, c = score + bias in FP32 with an error of
// at most eps.
//   groups   c goes to shared memory, kL / n_group lanes (a power of two) take a group's two largest
//            values, a rank count keeps topk_group groups, the others' c become -inf
//   choice   the lane maxima are sorted across the lanes; the (k + 1)-th is a lower bound of the
//            (k + 1)-th largest value, and the few values that reach it are compacted into a list
//            and ranked by (c descending, id ascending)
//   exact    where two neighbours of the ranking, or a group that stays and one that goes, are nearer
//            than their errors, the candidates or the groups are ranked again in FP64 (exact_ranking,
//            exact_groups). Only the values that can matter are computed again
//   others   rows with fewer unmasked experts than k, more candidates than the list holds (many equal
//            logits) or logits of +inf (whole_row)
// The weights are computed from the chosen logits alone, in FP32 as they are returned (off by an ulp or two: 7e-8 of
// their norm over 16,384 tokens, where one rounding from FP64 gives 3e-8).
// Bounded by instruction issue (70 % of the slots): the steps across lanes cost what they cost for one
// token or for two. Measured: 16,384 x 512, bias and 4 of 8 groups 24.7 to 26.0 us by the set of logits (1.4
// TB/s; 1,162 warp instructions a token), without both 12.4; 12,365 x 160, 3 of 8 groups 8.5; 2048 x 512 3.1; 4 x 512 3.0.
#include <cfloat>

#include "block.cuh"
#include "fp64.cuh"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;
constexpr unsigned kFull = 0xFFFFFFFFu;

// Bounds of a score's error relative to the row's largest possible score (1; softmax: the row's
// largest). Exponential 2^(x log2 e): ex2.approx is off by 2^-22, its argument by 1.5 * 2^-24 |x|
// (the softmax's x = l - m by 2^-24 |x| more). Sigmoid: that error counts s (1 - s) times (at most
// 8e-8 in all), the sum and rcp.approx add 2^-24 and 2^-23: 2.6e-7, taken as 6e-7. Softmax: a term's
// own error is at most 2.6e-7 of the largest; the sum of up to 1024 terms, 37 roundings deep, is off
// by 3.3e-6, a factor that all scores of the row share: two of them compare within 3.8e-6, two pairs
// within 7.6e-6, taken as 2 and 4 times 2.5e-6 (for groups without a bias too, which share no factor).
constexpr float kEpsSigmoid = 6e-7f, kEpsSoftmax = 2.5e-6f, kEpsAdd = 6e-8f;

__device__ __forceinline__ bool ahead(double c, int e, double d, int f) { return c > d || (c == d && e < f); }

template <bool F32>
__device__ __forceinline__ float load_logit(const SelectArgs& a, int64_t t, int e)
{
    return F32 ? static_cast<const float*>(a.logits)[t * a.ld + e]
               : bf16_to_f32(static_cast<const uint16_t*>(a.logits)[t * a.ld + e]);
}

__device__ __forceinline__ float fast_exp(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Scores in FP64. m: the row's largest logit (softmax); scale: 1 / its softmax sum, or 1 where only the
// order or ratios of scores are asked for.
struct Exact {
    bool sigmoid;
    double m, scale;
    __device__ __forceinline__ double operator()(float l) const
    {
        if (!(l > -INFINITY)) return 0.0;
        if (sigmoid) return rcp64(1.0 + exp64(-static_cast<double>(l)));
        return (l == m ? 1.0 : exp64(static_cast<double>(l) - m)) * scale;
    }
};

template <bool F32>
__device__ __noinline__ Exact exact_scores(const SelectArgs& a, int64_t t, bool need_sum)
{
    const int lane = threadIdx.x & 31;
    Exact x{a.sigmoid, 0.0, 1.0};
    if (a.sigmoid) return x;
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load_logit<F32>(a, t, e));
    x.m = warp_max(m);
    if (!need_sum) return x;
    double sum = 0.0;
    for (int e = lane; e < a.E; e += 32) sum += x(load_logit<F32>(a, t, e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    x.scale = rcp64(sum);
    return x;
}

// The groups that stay (a bit each), from FP64 values; the FP32 choice values are in c_s, off by at most
// eps_score and their last rounding. Only what lies within that of a group's second largest can be one
// of its two largest.
template <bool F32>
__device__ __noinline__ unsigned exact_groups(const SelectArgs& a, int64_t t, const float* c_s, float eps_score)
{
    const Exact score = exact_scores<F32>(a, t, a.bias != nullptr);
    const int lane = threadIdx.x & 31, size = a.group_size;
    const int lg = a.group_lanes_log2, per = 1 << lg, g = lane >> lg, j = lane & (per - 1);
    float top = -INFINITY, v2 = -INFINITY;
    if (g < a.n_group)
        for (int i = j; i < size; i += per) {
            const float v = c_s[g * size + i];
            v2 = fmaxf(v2, fminf(top, v));
            top = fmaxf(top, v);
        }
    for (int o = per >> 1; o > 0; o >>= 1) {
        const float o1 = __shfl_xor_sync(kFull, top, o), o2 = __shfl_xor_sync(kFull, v2, o);
        v2 = fmaxf(fminf(top, o1), fmaxf(v2, o2));
        top = fmaxf(top, o1);
    }
    if (!a.group_top2) v2 = top;
    const float margin = a.bias ? 2.0f * (eps_score + kEpsAdd * fmaxf(fabsf(top), fabsf(v2))) : 0.0f;
    const bool real = g < a.n_group;
    const float thr = v2 < INFINITY ? v2 - margin : v2;  // -inf where the group has one unmasked expert or none
    // this lane's values: j, j + per, ...; fewer than 64, since size <= 1024 / n_group and per > 16 / n_group
    uint64_t hits = 0;
    if (real)
        for (int i = 0; (i << lg) + j < size; ++i) {
            const float v = c_s[g * size + (i << lg) + j];
            hits |= static_cast<uint64_t>(v >= thr && v > -INFINITY) << i;
        }
    double v1 = -INFINITY, w2 = -INFINITY;
    while (__any_sync(kFull, hits != 0)) {
        if (hits) {
            const int e = g * size + ((__ffsll(static_cast<long long>(hits)) - 1) << lg) + j;
            hits &= hits - 1;
            const double v = score(load_logit<F32>(a, t, e)) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0);
            w2 = fmax(w2, fmin(v1, v));
            v1 = fmax(v1, v);
        }
    }
    for (int o = per >> 1; o > 0; o >>= 1) {
        const double o1 = __shfl_xor_sync(kFull, v1, o), o2 = __shfl_xor_sync(kFull, w2, o);
        w2 = fmax(fmin(v1, o1), fmax(w2, o2));
        v1 = fmax(v1, o1);
    }
    const double gv = a.group_top2 && w2 > -INFINITY ? v1 + w2 : v1;
    int rank = 0;
    for (int o = 0; o < a.n_group; ++o) {
        const double ov = __shfl_sync(kFull, gv, o << lg);
        rank += ov > gv || (ov == gv && o < g);
    }
    return __reduce_or_sync(kFull, real && rank < a.topk_group ? 1u << g : 0u);
}

// A candidate: its value as an order-preserving key in the high word, the complement of its id in the
// low one, so that a larger candidate goes first (larger value, then lower id).
using Cand = unsigned long long;
__device__ __forceinline__ Cand make_cand(float v, int id) { return static_cast<Cand>(order_key(v)) << 32 | static_cast<uint32_t>(~id); }
__device__ __forceinline__ int cand_id(Cand c) { return ~static_cast<int>(static_cast<uint32_t>(c)); }
__device__ __forceinline__ float cand_value(Cand c) { return key_value(static_cast<uint32_t>(c >> 32)); }

// The first k + 1 of the C candidates in sel, ordered by FP64 values (c64: scratch for C of them).
template <bool F32>
__device__ __noinline__ void exact_ranking(const SelectArgs& a, int64_t t, const Cand* cand, int C, unsigned long long* c64, Cand* sel)
{
    const Exact score = exact_scores<F32>(a, t, true);
    const int lane = threadIdx.x & 31;
    for (int q = lane; q < C; q += 32) {
        const int e = cand_id(cand[q]);
        // as an order-preserving integer (integers compare at their full rate); -0 does not arise from a sum
        const long long v = __double_as_longlong(score(load_logit<F32>(a, t, e)) + static_cast<double>(a.bias[e]));
        c64[q] = v < 0 ? ~static_cast<unsigned long long>(v) : static_cast<unsigned long long>(v) | 1ull << 63;
    }
    __syncwarp();
    for (int q = lane; q < C; q += 32) {
        const unsigned long long me = c64[q];
        const int id = cand_id(cand[q]);
        int r = 0;
        for (int o = 0; o < C; ++o) r += c64[o] > me || (c64[o] == me && cand_id(cand[o]) < id);
        if (r <= a.k) sel[r] = cand[q];
    }
    __syncwarp();
}

// One token by plain rounds of a warp arg-max over c[E] (lowest id first on equal values): rows that
// the ranking below does not hold. V: double with a bias; float without, where c is the logit.
template <bool F32, typename V>
__device__ __noinline__ void whole_row(const SelectArgs& a, int64_t t, V* c)
{
    const int lane = threadIdx.x & 31;
    const V ninf = -INFINITY, nan = NAN;
    const Exact score = exact_scores<F32>(a, t, a.bias || !a.renormalize);
    for (int e = lane; e < a.E; e += 32) {
        const float l = load_logit<F32>(a, t, e);
        const V v = a.bias ? static_cast<V>(score(l) + static_cast<double>(a.bias[e])) : static_cast<V>(l);
        c[e] = l > -INFINITY && v > ninf ? v : ninf;
    }
    __syncwarp();
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
        V v1 = ninf, v2 = ninf;
        if (lane < a.n_group)
            for (int i = 0; i < size; ++i) {
                const V v = c[lane * size + i];
                if (v > v1) {
                    v2 = v1;
                    v1 = v;
                } else if (v > v2)
                    v2 = v;
            }
        double gv = v1;
        if (a.group_top2 && v1 > ninf) {
            const double s1 = a.bias ? static_cast<double>(v1) : score(static_cast<float>(v1));
            gv = v2 > ninf ? s1 + (a.bias ? static_cast<double>(v2) : score(static_cast<float>(v2))) : s1;
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
    bool masked = true;
    for (int j = 0; j < a.k; ++j) {
        V best = nan;
        int at = 1 << 30;
        for (int e = lane; e < a.E; e += 32)
            if (c[e] == c[e] && (at == 1 << 30 || c[e] > best)) {
                best = c[e];
                at = e;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const V ob = __shfl_xor_sync(kFull, best, o);
            const int oa = __shfl_xor_sync(kFull, at, o);
            if (oa < 1 << 30 && (at == 1 << 30 || ob > best || (ob == best && oa < at))) {
                best = ob;
                at = oa;
            }
        }
        if (lane == j) {
            my_id = at;
            masked = !(best > ninf);
        }
        __syncwarp();
        if (lane == (at & 31)) c[at] = nan;
        __syncwarp();
    }
    double s = lane < a.k && !masked ? score(load_logit<F32>(a, t, my_id)) : 0.0;
    if (a.renormalize) {
        double total = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
        s = total > 0.0 ? s / total : 0.0;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = my_id;
        a.w[t * a.k + lane] = static_cast<float>(s * a.scale);
    }
}

template <bool F32>
__device__ __forceinline__ void whole_row(const SelectArgs& a, int64_t t, double* scratch)
{
    if (a.bias) whole_row<F32, double>(a, t, scratch);
    else whole_row<F32, float>(a, t, reinterpret_cast<float*>(scratch));
}

template <int kL>
__device__ __forceinline__ float lanes_max(float v)
{
#pragma unroll
    for (int o = kL / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

template <int kL>
__device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = kL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Expert held in slot i of a token's lane: 4 neighbours a 16-byte (bf16: 8-byte) load, or one.
template <int kL, bool VEC>
__device__ __forceinline__ int expert_of(int i, int lane)
{
    return VEC ? ((i >> 2) * kL + lane) * 4 + (i & 3) : i * kL + lane;
}

template <int kL, int kNper, bool F32, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, kNper < 8 || (kL == 32 && kNper <= 16) ? 8 : kNper <= 16 ? 6 : 4) k_select_experts(const __grid_constant__ SelectArgs a)
{
    constexpr int kTok = 32 / kL, kE = kNper * kL;
    constexpr int kCap = kL == 32 ? 128 : 64;  // candidates a token
    // the choice values of kTok tokens, then FP64 values of one
    __shared__ __align__(16) unsigned char scratch_s[kWarps][8 * (kE < kCap ? kCap : kE)];
    __shared__ __align__(16) Cand cand_s[kWarps][kTok][kCap];
    __shared__ Cand sel_s[kWarps][kTok][kL + 1];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / kL, sl = lane % kL;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTok;
    if (t0 >= a.T) return;
    const bool valid = kL == 32 || t0 + sub < a.T;
    const int64_t t = valid ? t0 + sub : t0;  // lanes past the last token repeat the one before and store nothing
    float* c_all = reinterpret_cast<float*>(scratch_s[warp]);
    float* c_s = c_all + sub * kE;
    Cand* cand = cand_s[warp][sub];
    Cand* sel = sel_s[warp][sub];
    const int E = a.E, k = a.k;
    bool whole = false;  // this token goes to whole_row

    // logits; what is masked or no expert is -inf (or NaN until it is cleaned)
    float c[kNper];
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kNper; i += 4) {
            const int e = expert_of<kL, true>(i, sl);
            c[i] = c[i + 1] = c[i + 2] = c[i + 3] = -INFINITY;
            if (e < E) {
                if constexpr (F32) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + t * a.ld + e));
                    c[i] = v.x, c[i + 1] = v.y, c[i + 2] = v.z, c[i + 3] = v.w;
                } else {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + t * a.ld + e));
                    c[i] = bf16_to_f32(v.x & 0xFFFFu), c[i + 1] = bf16_to_f32(v.x >> 16);
                    c[i + 2] = bf16_to_f32(v.y & 0xFFFFu), c[i + 3] = bf16_to_f32(v.y >> 16);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kNper; ++i) {
            const int e = expert_of<kL, false>(i, sl);
            c[i] = e < E ? load_logit<F32>(a, t, e) : -INFINITY;
        }
    }

    // the row's maximum and the softmax's sum, where anything needs them
    const bool groups = a.n_group > 1 && a.topk_group < a.n_group;
    const bool need_sum = !a.sigmoid && (a.bias || !a.renormalize);
    float m = 0.0f, inv_sum = 1.0f, smax = 1.0f;
    const bool have_m = !a.sigmoid && (need_sum || groups);
    if (have_m || groups) {  // elsewhere a NaN fails every comparison that it meets, as a masked value does
#pragma unroll
        for (int i = 0; i < kNper; ++i) c[i] = fmaxf(c[i], -INFINITY);
    }
    if (have_m) {
        m = c[0];
#pragma unroll
        for (int i = 1; i < kNper; ++i) m = fmaxf(m, c[i]);
        m = lanes_max<kL>(m);
        if (!(fabsf(m) < INFINITY)) {  // nothing but masked experts, or logits of +inf
            if (kL == 32) {  // a warp with one token may leave at once
                whole_row<F32>(a, t0, reinterpret_cast<double*>(scratch_s[warp]));
                return;
            }
            whole = true;
            m = 0.0f;
        }
        if (need_sum) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kNper; ++i) sum += fast_exp(c[i] - m);
            inv_sum = 1.0f / lanes_sum<kL>(sum);
            if (a.bias) smax = inv_sum;  // without one, groups are compared by exp(l - m), which the sum does not divide
        }
    }
    if (a.bias) {
        constexpr int kStep = VEC ? 4 : 1;
        float b[kNper];
#pragma unroll
        for (int i = 0; i < kNper; i += kStep) {
            const int e = expert_of<kL, VEC>(i, sl);
            if constexpr (VEC) {
                const float4 v = e < E ? __ldg(reinterpret_cast<const float4*>(a.bias + e)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
            } else {
                b[i] = e < E ? __ldg(a.bias + e) : 0.0f;
            }
        }
        // Whether every logit and bias is finite: products with 0 add up to 0 then (on the FMA pipe, which has
        // room; the comparisons that masks need run on the other, which has none). False, too, where there are
        // fewer experts than slots.
        float chk = 0.0f;
#pragma unroll
        for (int i = 0; i < kNper; ++i) chk = fmaf(c[i], 0.0f, fmaf(b[i], 0.0f, chk));
        const bool finite = __all_sync(kFull, chk == 0.0f);
        auto scores = [&](auto score) {
            if (finite) {
#pragma unroll
                for (int i = 0; i < kNper; ++i) c[i] = score(c[i]) + b[i];
            } else {
                // a masked logit stays -inf; a NaN of the logit or the bias becomes -inf
#pragma unroll
                for (int i = 0; i < kNper; ++i) c[i] = c[i] > -INFINITY ? fmaxf(score(c[i]) + b[i], -INFINITY) : -INFINITY;
            }
        };
        if (a.sigmoid) scores([](float l) { return fast_rcp(1.0f + fast_exp(-l)); });
        else scores([&](float l) { return fast_exp(l - m) * inv_sum; });
    }
    const float eps_score = (a.sigmoid ? kEpsSigmoid : kEpsSoftmax) * smax;

    if (groups) {
        // the values in order of their experts, so that a few lanes can take a group
#pragma unroll
        for (int i = 0; i < kNper; ++i) {
            const int e = expert_of<kL, VEC>(i, sl);
            if (VEC && i % 4 == 0)
                *reinterpret_cast<float4*>(c_s + e) = make_float4(c[i], c[(i + 1) % kNper], c[(i + 2) % kNper], c[(i + 3) % kNper]);
            if (!VEC) c_s[e] = c[i];
        }
        __syncwarp();
        const int size = a.group_size, lg = a.group_lanes_log2 - (kL == 16 ? 1 : 0), per = 1 << lg;
        const int g = sl >> lg, j = sl & (per - 1);
        float v1 = -INFINITY, v2 = -INFINITY;
        auto take = [&](float v) {
            v2 = fmaxf(v2, fminf(v1, v));
            v1 = fmaxf(v1, v);
        };
        if (g < a.n_group) {
            // the groups start at different places, so that their lanes read different banks
            if constexpr (VEC) {  // groups are multiples of four there
                const int n = (size / 4 - j + per - 1) >> lg;  // this lane's pieces of four: j, j + per, ...
                int i = max(min(g, n - 1), 0);
                for (int q = 0; q < n; ++q) {
                    const float4 v = *reinterpret_cast<const float4*>(c_s + g * size + ((i << lg) + j) * 4);
                    take(v.x), take(v.y), take(v.z), take(v.w);
                    if (++i == n) i = 0;
                }
            } else {
                const int n = (size - j + per - 1) >> lg;
                int i = max(min(g, n - 1), 0);
                for (int q = 0; q < n; ++q) {
                    take(c_s[g * size + (i << lg) + j]);
                    if (++i == n) i = 0;
                }
            }
        }
        for (int o = per >> 1; o > 0; o >>= 1) {
            const float o1 = __shfl_xor_sync(kFull, v1, o), o2 = __shfl_xor_sync(kFull, v2, o);
            v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
            v1 = fmaxf(v1, o1);
        }
        float gv = v1;
        if (a.group_top2 && v1 > -INFINITY) {
            auto score = [&](float l) { return a.sigmoid ? fast_rcp(1.0f + fast_exp(-l)) : fast_exp(l - m); };
            const float s1 = a.bias ? v1 : score(v1);
            gv = v2 > -INFINITY ? s1 + (a.bias ? v2 : score(v2)) : s1;
        }
        int rank = 0;
        for (int o = 0; o < a.n_group; ++o) {
            const float ov = __shfl_sync(kFull, gv, o << lg, kL);
            rank += ov > gv || (ov == gv && o < g);
        }
        const bool real = g < a.n_group;
        // a group's bit is that of its first lane
        unsigned keep = __ballot_sync(kFull, real && j == 0 && rank < a.topk_group) >> (sub * kL);
        if (a.bias || a.group_top2) {
            // The lowest that a group that stays can be against the highest that one that goes can be. Both of a
            // group's values have a score's error and a rounding of their own size, which may cancel in the sum; the
            // sum is rounded once more. (The roundings of lo and hi themselves keep their order.)
            const float size = !a.bias ? gv : a.group_top2 && v2 > -INFINITY ? fabsf(v1) + fabsf(v2) : fabsf(v1);
            const bool inexact = a.bias ? fabsf(v1) < INFINITY : v1 > -INFINITY;  // a masked group and an infinite bias are exact
            const float err = inexact ? 2.0f * (eps_score + kEpsAdd * size) : 0.0f;
            const bool range = err < INFINITY;  // a sum that left it says nothing
            float lo = real && rank < a.topk_group ? (range ? gv - err : -INFINITY) : INFINITY;
            float hi = real && rank >= a.topk_group ? (range ? gv + err : INFINITY) : -INFINITY;
            if constexpr (kL == 32) {
                asm volatile("redux.sync.min.f32 %0, %0, 0xFFFFFFFF;" : "+f"(lo));
                asm volatile("redux.sync.max.f32 %0, %0, 0xFFFFFFFF;" : "+f"(hi));
            } else {
                for (int o = per; o < kL; o <<= 1) {
                    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
                    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
                }
            }
            const bool near = valid && !whole && hi > -INFINITY && lo <= hi;
            auto decide = [&](int h, float eps) {
                const unsigned stay = exact_groups<F32>(a, t0 + h, c_all + h * kE, eps);
                if (sub == h) {
                    keep = 0;
                    for (int o = 0; o < a.n_group; ++o) keep |= ((stay >> o) & 1u) << (o << lg);
                }
            };
            if constexpr (kL == 32) {
                if (near) decide(0, eps_score);
            } else {
#pragma unroll 1
                for (unsigned n = __ballot_sync(kFull, near && sl == 0); n; n &= n - 1)
                    decide((__ffs(n) - 1) / kL, __shfl_sync(kFull, eps_score, __ffs(n) - 1));
            }
        }
        bool in = false;
#pragma unroll
        for (int i = 0; i < kNper; ++i) {
            if (!VEC || i % 4 == 0) {
                const unsigned ge = (static_cast<unsigned>(expert_of<kL, VEC>(i, sl)) * a.group_of_mul) >> 21;
                in = (keep >> ((ge << lg) & 31u)) & 1u;
            }
            if (!in) c[i] = -INFINITY;
        }
    }

    // the (k + 1)-th largest lane maximum (k = 32: the smallest), by a bitonic sort across the lanes
    float tau = c[0];
#pragma unroll
    for (int i = 1; i < kNper; ++i) tau = fmaxf(tau, c[i]);
    tau = fmaxf(tau, -INFINITY);  // a lane of NaN
    // descending runs everywhere: where a stage wants an ascending one, the values change their sign for it
#pragma unroll
    for (int s = 2; s <= kL; s <<= 1) {
        const float flip = ((sl & s) != 0) != ((sl & (s >> 1)) != 0 && s > 2) ? -1.0f : 1.0f;
        tau *= flip;
#pragma unroll
        for (int o = s >> 1; o > 0; o >>= 1) {
            const float v = __shfl_xor_sync(kFull, tau, o);
            tau = (sl & o) == 0 ? fmaxf(tau, v) : fminf(tau, v);
        }
    }
    tau = __shfl_sync(kFull, tau, k < kL ? k : kL - 1, kL);
    // what can be among the k largest in exact arithmetic has a value of at least tau less two errors
    if (a.bias) tau -= 2.0f * (eps_score + kEpsAdd * fabsf(tau));
    tau = fmaxf(tau, -FLT_MAX);  // a masked value is none

    // the values that reach it
    unsigned mine = 0;
#pragma unroll
    for (int i = 0; i < kNper; ++i) mine |= c[i] >= tau ? 1u << i : 0u;
    int pos = __popc(mine);
#pragma unroll
    for (int o = 1; o < kL; o <<= 1) {
        const int v = __shfl_up_sync(kFull, pos, o, kL);
        if (sl >= o) pos += v;
    }
    int C = __shfl_sync(kFull, pos, kL - 1, kL);
    pos -= __popc(mine);
    whole = whole || C < k || C > kCap;
    if (whole) {
        if (kL == 32) {
            __syncwarp();
            whole_row<F32>(a, t0, reinterpret_cast<double*>(scratch_s[warp]));
            return;
        }
        C = 0;
        mine = 0;
    }
    // Straight-line stores: a loop over a lane's bits was 1 us faster for 16,384 x 512, but where a lane has two slots it
    // left candidates of lanes without a bit in the list; why was not found.
    Cand* list = cand + pos;
#pragma unroll
    for (int i = 0; i < kNper; ++i)
        if ((mine >> i) & 1u) *list++ = static_cast<Cand>(__float_as_uint(c[i])) << 32 | static_cast<uint32_t>(expert_of<kL, VEC>(i, sl));
    __syncwarp();
    for (int q = sl; q < C; q += kL) {
        const Cand v = cand[q];
        cand[q] = make_cand(__uint_as_float(static_cast<uint32_t>(v >> 32)), static_cast<int>(static_cast<uint32_t>(v)));
    }
    __syncwarp();
    if (kL == 32 && C <= 16) {  // two lanes a candidate
        const Cand me = cand[lane >> 1];
        int r = 0;
#pragma unroll 4
        for (int o = lane & 1; o < C; o += 2) r += cand[o] > me;
        r += __shfl_xor_sync(kFull, r, 1);
        if (lane < 2 * C && r <= k) sel[r] = me;
    } else {
        for (int q = sl; q < C; q += kL) {
            const Cand me = cand[q];
            int r = 0;
#pragma unroll 4
            for (int o = 0; o < C; ++o) r += cand[o] > me;
            if (r <= k) sel[r] = me;
        }
    }
    __syncwarp();
    const Cand none = make_cand(0.0f, 0);
    Cand me = whole ? none : sel[sl < k ? sl : 0];
    if (a.bias) {
        const float v = cand_value(me), next = sl < k && sl + 1 < C ? cand_value(sel[sl + 1]) : -INFINITY;
        const bool near = valid && next > -INFINITY && v - next <= 2.0f * eps_score + kEpsAdd * (fabsf(v) + fabsf(next));
        const unsigned who = __ballot_sync(kFull, near);
        if (who) {
#pragma unroll 1
            for (int h = 0; h < kTok; ++h) {
                const unsigned all = kL == 32 ? kFull : 0xFFFFu << (h * 16);
                if (who & all) {
                    __syncwarp();
                    exact_ranking<F32>(a, t0 + h, cand_s[warp][h], __shfl_sync(kFull, C, h * kL),
                                       reinterpret_cast<unsigned long long*>(scratch_s[warp]), sel_s[warp][h]);
                }
            }
            if (!whole) me = sel[sl < k ? sl : 0];
        }
    }
    const int id = cand_id(me);
    const float l = a.bias ? load_logit<F32>(a, t, id) : cand_value(me);
    float s;
    if (a.renormalize) {
        // the scores divided by exp(largest chosen logit), or for sigmoid by no less than that: a factor
        // that the sum divides out, so that small scores keep their ratios
        const float top = a.bias ? lanes_max<kL>(sl < k ? l : -INFINITY) : __shfl_sync(kFull, l, 0, kL);
        whole = whole || (a.sigmoid ? top : have_m ? top - m : 0.0f) < -80.0f;  // scores that underflow here: in FP64
        if (kL == 32 && whole) {
            whole_row<F32>(a, t0, reinterpret_cast<double*>(scratch_s[warp]));
            return;
        }
        const float f = a.sigmoid ? fminf(top, 0.0f) : top;
        s = l == f ? 1.0f : expf(l - f);
        if (a.sigmoid) s = l < 0.0f ? s / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));  // f is 0 there
        s /= lanes_sum<kL>(sl < k ? s : 0.0f);
    } else {
        s = a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - m) * inv_sum;
    }
    if (kL == 32 ? sl < k : valid && !whole && sl < k) {
        a.ids[t * k + sl] = id;
        a.w[t * k + sl] = s * a.scale;
    }
    if constexpr (kL < 32) {
#pragma unroll 1
        for (unsigned n = __ballot_sync(kFull, whole && valid && sl == 0); n; n &= n - 1) {
            __syncwarp();
            whole_row<F32>(a, t0 + (__ffs(n) - 1) / kL, reinterpret_cast<double*>(scratch_s[warp]));
        }
    }
}

template <int kL, int kNper, bool F32>
cudaError_t launch(const SelectArgs& a, bool vec, cudaStream_t stream)
{
    constexpr int per_cta = kWarps * (32 / kL);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) + per_cta - 1) / per_cta)), block(kWarps * 32);
    if constexpr (kNper >= 4) {
        if (vec) return launch_pdl(k_select_experts<kL, kNper, F32, true>, grid, block, 0, stream, a);
    }
    return launch_pdl(k_select_experts<kL, kNper, F32, false>, grid, block, 0, stream, a);
}

template <bool F32>
cudaError_t launch_type(const SelectArgs& a, cudaStream_t stream)
{
    // four experts a load where every row, the bias and the groups allow it and there are enough for all
    // lanes
    constexpr int bytes = F32 ? 4 : 2;
    const bool vec = a.E % (4 * a.n_group) == 0 && reinterpret_cast<uintptr_t>(a.logits) % (4 * bytes) == 0 &&
                     (a.ld % 4 == 0 || a.T == 1) && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    // Two tokens a warp where there are several for every multiprocessor (12,365 x 160, 3 of 8 groups: 9.3 us
    // against 11.1; of 512 experts a lane would hold 32 values, whose registers cost more than the shared steps
    // save: 16,384 x 512 14.0 us against 12.4). k + 1 of 16 lane maxima still leave a short list of candidates.
    if (a.E <= 256 && a.k <= 12 && a.n_group <= 16 && a.T >= 16 * device_sm_count()) {
        if (a.E <= 32) return launch<16, 2, F32>(a, vec, stream);
        if (a.E <= 64) return launch<16, 4, F32>(a, vec && a.E >= 64, stream);
        if (a.E <= 128) return launch<16, 8, F32>(a, vec, stream);
        if (a.E <= 192) return launch<16, 12, F32>(a, vec, stream);
        return launch<16, 16, F32>(a, vec, stream);
    }
    if (a.E <= 32) return launch<32, 1, F32>(a, vec, stream);
    if (a.E <= 128) return launch<32, 4, F32>(a, vec && a.E >= 128, stream);
    if (a.E <= 256) return launch<32, 8, F32>(a, vec, stream);
    if (a.E <= 512) return launch<32, 16, F32>(a, vec, stream);
    return launch<32, 32, F32>(a, vec, stream);
}

}  // namespace

cudaError_t launch_select_experts(const SelectArgs& a, cudaStream_t stream)
{
    if (a.T <= 0) return cudaSuccess;
    SelectArgs b = a;
    b.group_size = a.E / a.n_group;
    b.group_lanes_log2 = 0;
    while ((2 << b.group_lanes_log2) * a.n_group <= 32) ++b.group_lanes_log2;
    // e / size for e < 1024 as a product: exact, since 1023 * size <= 2^20 < 2^21
    b.group_of_mul = ((1u << 21) + b.group_size - 1) / b.group_size;
    return a.logits_f32 ? launch_type<true>(b, stream) : launch_type<false>(b, stream);
}

}  // namespace moe
