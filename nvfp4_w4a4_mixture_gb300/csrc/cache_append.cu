// cache_append.cu -- norm, rotation by position and append to the paged cache, one launch:
//   u = x rsqrt(mean(x^2) + eps) (off + w);  (a, b) -> (a cos - b sin, a sin + b cos), angle p inv_freq[i]
// A head of D elements is in the registers of D / 8 lanes (16 bytes each) from its load to its store: the norm's sum and
// the rotation's partner come by shuffles. The angle is a 64-bit fraction of a turn: inv_freq / 2 pi in 2^-64 turns
// (one FP64 product, off by 2^-54 of it), times the position modulo 2^64, which drops whole turns exactly, so the
// angle of position 2^20 is as good as that of position 1; sine and cosine of what is left are FP32's.
#include "attention.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_at(const uint4& v, int i)
{
    const uint32_t w = i / 2 == 0 ? v.x : i / 2 == 1 ? v.y : i / 2 == 2 ? v.z : v.w;
    return i % 2 ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
}

template <int kD, bool kE4M3>
__global__ void __launch_bounds__(kThreads) k_cache_append(const __grid_constant__ AppendArgs p, int heads_per_cta)
{
    constexpr int kLanes = kD / 8, kHeads = kThreads / kLanes;  // lanes a head, heads a pass
    __shared__ float2 turn[kD / 2];
    const int tid = threadIdx.x, at = tid % kLanes, c0 = at * 8, half = p.rot / 2;
    const int n_all = p.n_q + 2 * p.c.n_kv;
    const int64_t t = blockIdx.x;
    const int h0 = blockIdx.y * heads_per_cta, h1 = min(n_all, h0 + heads_per_cta);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    auto load = [&](int h) -> uint4 {
        if (h >= h1) return make_uint4(0, 0, 0, 0);
        const uint16_t* x = h < p.n_q                ? p.q + t * p.ld_q + h * kD
                            : h < p.n_q + p.c.n_kv ? p.k + t * p.ld_k + (h - p.n_q) * kD
                                                     : p.v + t * p.ld_v + (h - p.n_q - p.c.n_kv) * kD;
        return *reinterpret_cast<const uint4*>(x + c0);
    };
    int h = h0 + tid / kLanes;
    uint4 x = load(h);

    // the requests' rules, by the first CTA
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int s = tid; s < p.r.S; s += kThreads) {
            bool bad;
            load_request(p.r, s, p.T, p.T, bad);
            if (bad) record_status(p.status, kDevBadRequest);
        }
    const int s = find_request(p.r.seg_offsets, p.r.S, static_cast<int>(t));
    if (s < 0 || s >= p.r.S) return;  // behind the last request
    bool bad;
    const Request r = load_request(p.r, s, p.T, p.T, bad);
    const int pos = r.len - r.n + static_cast<int>(t - r.beg);
    if (r.n == 0 || t >= r.beg + r.n || pos < 0) return;
    int64_t page = __ldg(p.r.pages + s * p.r.ld_pages + (pos >> p.c.page_log2));
    if (page < 0 || page >= p.c.n_pages) {
        page = -1;
        if (tid == 0) record_status(p.status, kDevBadPage);
    }
    const int64_t place = page * p.c.ld_page + (pos & ((1 << p.c.page_log2) - 1)) * p.c.ld_slot;

    if (tid < half) {
        double f = static_cast<double>(__ldg(p.inv_freq + tid)) * 0.15915494309189533577;  // turns a position
        f -= floor(f);
        const uint64_t phase = static_cast<uint64_t>(f * 18446744073709551616.0) * static_cast<uint64_t>(pos);
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int64_t>(phase)) * 0x1p-63f, &sn, &cs);
        turn[tid] = make_float2(cs, sn);
    }
    __syncthreads();
    float2 cs[8];  // of this lane's elements (interleaved: of its four pairs)
    const bool turns = c0 < p.rot;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = c0 + i, f = p.interleaved ? c / 2 : c < half ? c : c - half;
        cs[i] = turns ? turn[f] : make_float2(1.0f, 0.0f);
    }
    const bool low = c0 < half;
    const int partner = !turns || p.interleaved ? at : low ? at + half / 8 : at - half / 8;

    for (; h - tid / kLanes < h1; h += kHeads) {
        const uint4 cur = x;
        x = load(h + kHeads);
        const bool is_q = h < p.n_q, is_v = h >= p.n_q + p.c.n_kv;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = bf16_at(cur, i);
        const uint16_t* w = is_q ? p.w_q : p.w_k;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (!is_v && w) {
            const float rs = rsqrtf(sum * (1.0f / kD) + p.eps);
            const uint4 wv = __ldg(reinterpret_cast<const uint4*>(w + c0));
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * rs * (p.w_offset + bf16_at(wv, i));
        }
        float o[8];
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                o[i] = f[i] * cs[i].x - f[i + 1] * cs[i].y;
                o[i + 1] = f[i] * cs[i].y + f[i + 1] * cs[i].x;
            }
        } else {
            const int lane = (tid & 31) - at + partner;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float other = __shfl_sync(0xFFFFFFFFu, f[i], lane);
                o[i] = low ? f[i] * cs[i].x - other * cs[i].y : other * cs[i].y + f[i] * cs[i].x;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!turns || is_v) o[i] = f[i];
        if (h >= h1) continue;
        if (is_q) {
            const uint4 v = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
            *reinterpret_cast<uint4*>(p.q_out + t * p.ld_q_out + h * kD + c0) = v;
        } else if (page >= 0) {
            const int kv = is_v ? h - p.n_q - p.c.n_kv : h - p.n_q;
            const int64_t e = place + kv * p.c.ld_head + c0;
            void* base = is_v ? p.c.v : p.c.k;
            if constexpr (kE4M3) {
                const float* sc = is_v ? p.c.v_scale : p.c.k_scale;
                const float d = sc ? __ldg(sc + kv) : 1.0f;
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = ptx::cvt_e4m3x2(__fdiv_rn(o[2 * i], d), __fdiv_rn(o[2 * i + 1], d));
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + e) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
            } else {
                const uint4 v = is_v ? cur
                                     : make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e) = v;
            }
        }
    }
}

template <int kD, bool kE4M3>
cudaError_t launch(const AppendArgs& a, int sms, cudaStream_t stream)
{
    constexpr int kHeads = kThreads / (kD / 8);
    const int n_all = a.n_q + 2 * a.c.n_kv, passes = (n_all + kHeads - 1) / kHeads;
    // few tokens: their heads over more CTAs, a pass each
    const int per = a.T * static_cast<int64_t>(passes) <= sms * 4LL ? kHeads : n_all;
    return launch_pdl(k_cache_append<kD, kE4M3>, dim3(a.T, (n_all + per - 1) / per), dim3(kThreads), 0, stream, a, per);
}

template <bool kE4M3>
cudaError_t launch_d(const AppendArgs& a, int sms, cudaStream_t stream)
{
    switch (a.c.D) {
    case 64: return launch<64, kE4M3>(a, sms, stream);
    case 128: return launch<128, kE4M3>(a, sms, stream);
    case 256: return launch<256, kE4M3>(a, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int sms, cudaStream_t stream)
{
    return a.c.e4m3 ? launch_d<true>(a, sms, stream) : launch_d<false>(a, sms, stream);
}

}  // namespace moe
