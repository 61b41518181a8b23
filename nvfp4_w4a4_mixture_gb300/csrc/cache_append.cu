// cache_append.cu -- norm, rotation by position and append to the paged cache, one launch:
//   u = x rsqrt(mean(x^2) + eps) (off + w);  (a, b) -> (a cos - b sin, a sin + b cos), angle p inv_freq[i]
// A warp takes the heads of one token (of few tokens, some of them), 256 elements a pass: a head of D elements is in the
// registers of D / 8 lanes (16 bytes each) from its load to its store, the norm's sum and the rotation's partner come by
// shuffles. The angle is a 64-bit fraction of a turn: inv_freq / 2 pi in 2^-64 turns (a product of integers, off by less
// than one of them), times the position modulo 2^64, which drops whole turns exactly, so the angle of position 2^20 is as
// good as that of position 1. What is left is rounded to FP32 (2^-26 turns at the most) for FP32's sine and cosine.
// Measured: 16,384 tokens, 16 + 2 heads of 256, 60 us, 5.6 TB/s (84 % of what a copy reaches), into an 8-bit cache 67 us (4.8);
// 12,365 tokens of 37 requests, 14 + 2 heads of 64, 19 us, 3.0 TB/s: a token's loads come one after the other (its request,
// length and page, then keys and values behind the queries' stores); 4 tokens 3.4 us, that chain.
#include "attention.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;

// two bf16 values as FP32
__device__ __forceinline__ uint64_t widen(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// f / 2 pi modulo one turn, in 2^-64 turns, for a finite f: its 24 bits times 2^96 / 2 pi (94 bits), shifted. Cut, not
// rounded: off by less than 2^-64 turns. (In integers: a multiprocessor has few units for FP64.)
__device__ __forceinline__ uint64_t turns_of(float f)
{
    constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f4ull;  // floor(2^96 / 2 pi)
    const uint32_t bits = __float_as_uint(f), e = bits >> 23 & 0xFFu;
    const uint64_t m = e ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;  // |f| = m 2^(max(e, 1) - 150)
    const uint64_t low = m * kLow, mid = m * kHigh;
    const uint64_t t0 = (mid << 32) + low, t1 = (__umul64hi(m, kHigh) << 32) + (mid >> 32) + (t0 < low);  // m 2^96 / 2 pi
    const int shift = 32 + 150 - static_cast<int>(e ? e : 1);
    const uint64_t r = shift >= 128 ? 0 : shift >= 64 ? t1 >> (shift - 64) : shift > 0 ? t0 >> shift | t1 << (64 - shift) : shift > -64 ? t0 << -shift : 0;
    return bits >> 31 ? 0 - r : r;
}

enum Kind : int { kQuery, kKey, kValue };

// What a warp knows of its token and its lanes.
template <int kD>
struct Token {
    int64_t place;           // in the cache, -1: none
    bool turns, low;         // this lane's elements are rotated; they are the first of their pairs (half-split)
    int partner;             // the lane that holds the others of their pairs
    uint64_t cos[4], sin[4]; // of this lane's elements, the sine with the sign that its term has
};

// Passes [first, last) of a token's queries, keys or values (n heads from `from` on; a pass is 32 lanes times 8 elements,
// whole heads), kN at a time, side by side: their shuffles and roots take turns. x: the first kN's loads, or null.
template <int kD, bool kE4M3, Kind kKind, int kN>
__device__ __forceinline__ void heads(const AppendArgs& p, const Token<kD>& k, const uint16_t* from, uint16_t* out, const uint16_t* w, int n,
                                      int first, int last, const uint4* x0)
{
    constexpr int kLanes = kD / 8;
    const int lane = threadIdx.x % 32, c0 = lane % kLanes * 8, elements = n * kD;
    const int64_t head_ld = p.c.ld_head;
    uint64_t wf[4];
    if (kKind != kValue && w) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(w + c0));
        const uint64_t off = pair(p.w_offset, p.w_offset), one = pair(1.0f, 1.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) wf[j] = fma2(widen(word(v, j)), one, off);
    }
    auto load = [&](int pass) {
        const int e = pass * 256 + lane * 8;
        return pass < last && e < elements ? *reinterpret_cast<const uint4*>(from + e) : make_uint4(0, 0, 0, 0);
    };
    uint4 next[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) next[i] = x0 ? x0[i] : load(first + i);
    for (int pass = first; pass < last; pass += kN) {
        uint4 x[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            x[i] = next[i];
            next[i] = load(pass + kN + i);
        }
        uint64_t f[kN][4];
        if constexpr (kKind != kValue || kE4M3) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = widen(word(x[i], j));
        }
        if constexpr (kKind != kValue) {
            if (w) {
                float sum[kN];
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    uint64_t s = mul2(f[i][0], f[i][0]);
#pragma unroll
                    for (int j = 1; j < 4; ++j) s = fma2(f[i][j], f[i][j], s);
                    sum[i] = lo_of(s) + hi_of(s);
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < kN; ++i) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], o);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const float r = rsqrtf(sum[i] * (1.0f / kD) + p.eps);
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[i][j] = mul2(mul2(f[i][j], pair(r, r)), wf[j]);
                }
            }
            if (p.rot) {
#pragma unroll
                for (int i = 0; i < kN; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = lo_of(f[i][j]), b = hi_of(f[i][j]);
                        const uint64_t other = p.interleaved ? pair(b, a)
                                                             : pair(__shfl_sync(0xFFFFFFFFu, a, k.partner), __shfl_sync(0xFFFFFFFFu, b, k.partner));
                        const uint64_t turned = fma2(f[i][j], k.cos[j], mul2(other, k.sin[j]));
                        f[i][j] = k.turns ? turned : f[i][j];
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = (pass + i) * 256 + lane * 8, head = e / kD;
            if (pass + i >= last || e >= elements || (kKind != kQuery && k.place < 0)) continue;
            const int64_t at = k.place + head * head_ld + c0;
            if constexpr (kKind != kQuery && kE4M3) {
                const float* sc = kKind == kValue ? p.c.v_scale : p.c.k_scale;
                const float d = sc ? __ldg(sc + head) : 1.0f;
                uint32_t b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = ptx::cvt_e4m3x2(__fdiv_rn(lo_of(f[i][j]), d), __fdiv_rn(hi_of(f[i][j]), d));
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kKind == kValue ? p.c.v : p.c.k) + at) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
            } else {
                uint4 v = x[i];
                if constexpr (kKind != kValue)
                    v = make_uint4(pack_bf16x2(lo_of(f[i][0]), hi_of(f[i][0])), pack_bf16x2(lo_of(f[i][1]), hi_of(f[i][1])),
                                   pack_bf16x2(lo_of(f[i][2]), hi_of(f[i][2])), pack_bf16x2(lo_of(f[i][3]), hi_of(f[i][3])));
                uint16_t* const to = kKind == kQuery ? out + e : static_cast<uint16_t*>(kKind == kValue ? p.c.v : p.c.k) + at;
                *reinterpret_cast<uint4*>(to) = v;
            }
        }
    }
}

template <int kD, bool kE4M3>
__global__ void __launch_bounds__(kWarps * 32) k_cache_append(const __grid_constant__ AppendArgs p, int passes, int chunks)
{
    constexpr int kLanes = kD / 8, kN = 2;
    __shared__ float2 turn_of[kWarps][kD / 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, at = lane % kLanes, c0 = at * 8, half = p.rot / 2;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + warp, t = id / chunks;
    const int chunk = static_cast<int>(id - t * chunks);
    float2* const turn = turn_of[warp];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // the requests' rules, by the first CTA
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < p.r.S; s += kWarps * 32) {
            bool bad;
            load_request(p.r, s, p.T, p.T, bad);
            if (bad) record_status(p.status, kDevBadRequest);
        }
    if (t >= p.T) return;
    // this warp's passes [first, last) of all of the token's: of its queries, then its keys, then its values
    const int nq = p.n_q * kD, nk = p.c.n_kv * kD, q_passes = (nq + 255) / 256, k_passes = (nk + 255) / 256;
    const int first = chunk * passes, last = min(q_passes + 2 * k_passes, first + passes);
    const uint16_t *q = p.q + t * p.ld_q, *k = p.k + t * p.ld_k, *v = p.v + t * p.ld_v;
    uint4 x[kN];  // the first of them, if queries
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int e = (first + i) * 256 + lane * 8;
        x[i] = first + i < min(last, q_passes) && e < nq ? *reinterpret_cast<const uint4*>(q + e) : make_uint4(0, 0, 0, 0);
    }
    uint64_t step[kD / 64];  // turns a position of the frequencies lane, lane + 32, ..
#pragma unroll
    for (int i = 0; i < kD / 64; ++i) step[i] = lane + 32 * i < half ? turns_of(__ldg(p.inv_freq + lane + 32 * i)) : 0;

    const int s = find_request(p.r.seg_offsets, p.r.S, static_cast<int>(t));
    if (s < 0 || s >= p.r.S) return;  // behind the last request
    bool bad;
    const Request r = load_request(p.r, s, p.T, p.T, bad);
    const int pos = r.len - r.n + static_cast<int>(t - r.beg);
    if (r.n == 0 || t < r.beg || t >= r.beg + r.n || pos < 0) return;
    const int page = __ldg(p.r.pages + s * p.r.ld_pages + (pos >> p.c.page_log2));
#pragma unroll
    for (int i = 0; i < kD / 64; ++i)
        if (lane + 32 * i < half) {
            float sn, cs;
            sincospif(static_cast<float>(static_cast<int64_t>(step[i] * static_cast<uint64_t>(pos))) * 0x1p-63f, &sn, &cs);
            turn[lane + 32 * i] = make_float2(cs, sn);
        }
    __syncwarp();
    Token<kD> tok;
    tok.turns = c0 < p.rot;
    tok.low = c0 < half;
    tok.partner = lane - at + (!tok.turns || p.interleaved ? at : tok.low ? at + half / 8 : at - half / 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = tok.turns ? c0 + 2 * j : 0;
        const int f0 = p.interleaved ? c / 2 : c < half ? c : c - half, f1 = p.interleaved ? c / 2 : f0 + 1;
        const float2 a = half ? turn[f0] : make_float2(1.0f, 0.0f), b = half ? turn[f1] : a;
        tok.cos[j] = pair(a.x, b.x);
        tok.sin[j] = p.interleaved ? pair(-a.y, b.y) : tok.low ? pair(-a.y, -b.y) : pair(a.y, b.y);
    }
    tok.place = page * p.c.ld_page + (pos & ((1 << p.c.page_log2) - 1)) * p.c.ld_slot;
    if (page < 0 || page >= p.c.n_pages) {
        tok.place = -1;
        if (lane == 0) record_status(p.status, kDevBadPage);
    }
    heads<kD, kE4M3, kQuery, kN>(p, tok, q, p.q_out + t * p.ld_q_out, p.w_q, p.n_q, first, min(last, q_passes), x);
    // One pass of keys: nothing beside it (12,365 tokens, 2 heads of 64: 19.3 us, 19.9). Not in the code for heads of 256, which
    // have one pass with a single head: it takes registers (16,384 tokens 66.6 us, 60.2).
    if constexpr (kD < 256)
        if (k_passes == 1) {
            heads<kD, kE4M3, kKey, 1>(p, tok, k, nullptr, p.w_k, p.c.n_kv, max(first - q_passes, 0), min(last - q_passes, 1), nullptr);
            heads<kD, kE4M3, kValue, 1>(p, tok, v, nullptr, nullptr, p.c.n_kv, max(first - q_passes - 1, 0), last - q_passes - 1, nullptr);
            return;
        }
    heads<kD, kE4M3, kKey, kN>(p, tok, k, nullptr, p.w_k, p.c.n_kv, max(first - q_passes, 0), min(last - q_passes, k_passes), nullptr);
    heads<kD, kE4M3, kValue, kN>(p, tok, v, nullptr, nullptr, p.c.n_kv, max(first - q_passes - k_passes, 0), last - q_passes - k_passes, nullptr);
}

template <int kD, bool kE4M3>
cudaError_t launch(const AppendArgs& a, int sms, cudaStream_t stream)
{
    const int passes_all = (a.n_q * kD + 255) / 256 + 2 * ((a.c.n_kv * kD + 255) / 256);
    // a warp a token; of few tokens as many warps as 16 an SM are, a pass each at the least
    const int64_t per = static_cast<int64_t>(a.T) * passes_all / (sms * 16LL);
    const int passes = static_cast<int>(per < 1 ? 1 : per > passes_all ? passes_all : per), chunks = (passes_all + passes - 1) / passes;
    const int64_t ctas = (static_cast<int64_t>(a.T) * chunks + kWarps - 1) / kWarps;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(k_cache_append<kD, kE4M3>, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), 0, stream, a, passes, chunks);
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
