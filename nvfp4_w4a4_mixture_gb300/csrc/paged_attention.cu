// paged_attention.cu -- attention of a few new tokens of every request over a paged cache:
//   out = sum_t softmax_t(scale q . k_t) v_t over the tokens that a row sees, in one pass over keys and values
// with the running maximum m and sum l of the softmax: o <- o 2^(m - m') + 2^(s - m') v.
//
// Work: a unit is 64 cached tokens of one key head against up to kRows rows (new tokens x query heads of that key
// head). The units of all requests, in order, are cut into equal runs, one a CTA, so ragged lengths balance by
// themselves. A (request, head) whose units lie in one run is finished there; of the others every run leaves o, m and l
// in the workspace, and a second launch adds them in the order of the runs.
// A CTA of four warps streams K and V through a ring in shared memory (cp.async of 16 bytes a lane, addresses from the
// page table, which is read a unit ahead; a token behind the end is filled with zeros). Of a unit each warp takes 16
// tokens of Q K^T, the warps exchange maxima and weights through shared memory, and each takes a quarter of
// the columns of P V: K and V are read from shared memory once, and the accumulators need no join. mma.sync:
// the products are 4 flops a byte and row, for 16 rows 64 flops a byte, which the memory bounds long before.
// bf16 cache: the weights are two bf16 values (16 bits); E4M3 cache: codes become FP16 (exact), the weights are FP16
// and q is scaled to FP16's range by a power of two a row (exact where q is not 2^-30 of the row's largest).
#include "attention.cuh"

namespace moe {

namespace {

constexpr int kThreads = 128, kTile = 64;
constexpr int kMaxSmem = 227 * 1024, kHalfSmem = 113 * 1024;
constexpr int kMinUnits = 2;  // a run has at least so many units

template <int kD, bool kE4M3, int kWR>
struct Shape {
    static constexpr int kRows = 16 * kWR;
    static constexpr int kRowBytes = kD * (kE4M3 ? 1 : 2);       // of a cached token's head
    static constexpr int kStage = 2 * kTile * kRowBytes;         // K, V
    static constexpr int kQ = kRows * kD * 2;
    static constexpr int kP = kRows * kTile * 2 * (kE4M3 ? 1 : 2);
    static constexpr int kFixed = kQ + kP + kRows * 64 + 256;
    // two CTAs an SM where three stages fit half of its shared memory, else one
    static constexpr int kHalf = (kHalfSmem - kFixed) / kStage;
    static constexpr int kFit = kHalf >= 3 ? kHalf : (kMaxSmem - kFixed) / kStage;
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kSmem = kFixed + kStages * kStage;
    static_assert(kStages >= 2 && kSmem <= kMaxSmem, "shared memory");
};

// ---- the cut of the units into runs
__host__ __device__ __forceinline__ int runs_of(int64_t total, int ctas)
{
    const int64_t n = (total + kMinUnits - 1) / kMinUnits;
    return n < ctas ? static_cast<int>(n) : ctas;
}
struct Cut {
    int64_t q, r;  // runs 0 .. r - 1 have q + 1 units, the others q
    __device__ Cut(int64_t total, int runs) : q(total / runs), r(total % runs) {}
    __device__ int64_t first(int64_t c) const { return c * q + (c < r ? c : r); }
    __device__ int run(int64_t u) const { return static_cast<int>(u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q); }
};

struct Span {
    int beg, n, len, start, tiles, segs;  // rows; tokens; first token seen; units along the tokens; (head, row block) pairs
    __device__ int64_t units() const { return static_cast<int64_t>(tiles) * segs; }
};

template <int kRows>
__device__ __forceinline__ Span span_of(const AttentionArgs& p, int s, bool& bad)
{
    const Request r = load_request(p.r, s, p.T, p.max_new, bad);
    Span a{r.beg, r.n, r.len, 0, 0, 0};
    if (r.n == 0) return a;
    if (p.window > 0) {
        const int64_t first = static_cast<int64_t>(r.len) - r.n - p.window + 1;
        a.start = first > 0 ? static_cast<int>(first) : 0;
    }
    a.tiles = max(1, static_cast<int>((static_cast<int64_t>(r.len) - a.start + kTile - 1) / kTile));  // a request that sees nothing has a unit, too
    a.segs = p.c.n_kv * ((r.n * p.group + kRows - 1) / kRows);
    return a;
}

// A place in the order of units.
template <int kRows>
struct Cursor {
    Span a;
    int s, seg, tile;
    __device__ void at(const AttentionArgs& p, int request, int64_t unit)
    {
        bool bad;
        s = request;
        a = span_of<kRows>(p, s, bad);
        seg = static_cast<int>(unit / a.tiles);
        tile = static_cast<int>(unit - static_cast<int64_t>(seg) * a.tiles);
    }
    // The next unit (there is one).
    __device__ void next(const AttentionArgs& p)
    {
        if (++tile < a.tiles) return;
        tile = 0;
        if (++seg < a.segs) return;
        seg = 0;
        bool bad;
        do a = span_of<kRows>(p, ++s, bad);
        while (a.segs == 0);
    }
};

// ---- warp-level matrix products and their operands
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool kF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (kF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes (the lower 16 bits) as two FP16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v)
{
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}\n" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float f16_to_f32(uint32_t bits16)
{
    float f;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.f32.f16 %0, t;\n\t}\n" : "=f"(f) : "r"(bits16));
    return f;
}
// 2^x, the hardware's (2 units in the last place); 0 for -inf
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 16-byte piece c of row r, so that eight rows' equal pieces lie in different banks
template <int kRowBytes>
__device__ __forceinline__ uint32_t piece(int r, int c)
{
    if constexpr (kRowBytes == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else return r * kRowBytes + ((c ^ (r & 7)) << 4);
}
// the same for E4M3 keys, which are read four pieces of two rows at a time
template <int kRowBytes>
__device__ __forceinline__ uint32_t piece_k8(int r, int c)
{
    if constexpr (kRowBytes == 64) return r * 64 + (c << 4);
    else return r * kRowBytes + ((c ^ ((r & 1) << 2)) << 4);
}

template <int kD, bool kE4M3, int kWR>
__global__ void __launch_bounds__(kThreads) k_paged_attention(const __grid_constant__ AttentionArgs p)
{
    using S = Shape<kD, kE4M3, kWR>;
    constexpr int kRows = S::kRows, kRB = S::kRowBytes, kChunks = kRB / 16, kStages = S::kStages;
    constexpr int kQB = kD * 2;             // bytes of a row of q
    constexpr int kNB = kD / 32;            // 8-column blocks of a warp's quarter of the columns
    constexpr int kKS = kD / 16;            // steps of Q K^T
    constexpr bool kQReg = kWR * kKS <= 8;  // q's fragments stay in registers
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const ring = smem;
    uint8_t* const qs = smem + kStages * S::kStage;
    uint8_t* const ps = qs + S::kQ;         // weights: [kRows][64] 16-bit, bf16: the high parts, then the low ones
    float* const wmax = reinterpret_cast<float*>(ps + S::kP);  // [kRows][4]
    float* const wsum = wmax + kRows * 4;                      // [kRows][4]
    float* const qscale = wsum + kRows * 4;                    // [kRows]
    int64_t* const found = reinterpret_cast<int64_t*>(qscale + kRows);  // 5 sums, then what the search found
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0), lane = tid % 32, g = lane / 4, t4 = lane % 4;
    const uint32_t ring_a = ptx::smem_u32(ring), qs_a = ptx::smem_u32(qs), ps_a = ptx::smem_u32(ps);

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // ---- this CTA's run: the units before each request, a block of requests a thread
    const int block = (p.r.S + kThreads - 1) / kThreads, sb = min(p.r.S, tid * block), se = min(p.r.S, sb + block);
    int64_t mine = 0;
    for (int s = sb; s < se; ++s) {
        bool bad;
        mine += span_of<kRows>(p, s, bad).units();
        if (bad && blockIdx.x == 0) record_status(p.status, kDevBadRequest);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) found[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) before += found[w];
        total += found[w];
    }
    if (blockIdx.x == 0) {  // for the join
        int64_t u = before;
        for (int s = sb; s < se; ++s) {
            bool bad;
            p.prefix[s] = u;
            u += span_of<kRows>(p, s, bad).units();
        }
        if (tid == 0) p.prefix[p.r.S] = total;
    }
    const int runs = runs_of(total, gridDim.x);
    if (static_cast<int>(blockIdx.x) >= runs) return;
    const Cut cut(total, runs);
    const int64_t u0 = cut.first(blockIdx.x), u1 = cut.first(blockIdx.x + 1);
    if (u0 >= before && u0 < before + mine) {
        int64_t u = u0 - before;
        int s = sb;
        for (;; ++s) {
            bool bad;
            const int64_t n = span_of<kRows>(p, s, bad).units();
            if (u < n) break;
            u -= n;
        }
        found[4] = s;
        found[5] = u;
    }
    __syncthreads();
    const int count = static_cast<int>(u1 - u0);
    Cursor<kRows> ld, cu;
    ld.at(p, static_cast<int>(found[4]), found[5]);
    cu = ld;

    // ---- loads: each warp the 16 tokens 16 warp .. + 15 of a unit
    int64_t row_off = -1;  // lanes l and l + 16: the token's offset in the cache, -1: zeros
    int page = 0, row_slot = 0, row_head = 0;
    bool row_in = false;
    int fetched = 0;
    auto fetch = [&]() {  // the page ids of the unit at ld
        if (fetched > 0 && fetched < count) ld.next(p);
        row_in = false;
        if (fetched < count) {
            const int pos = ld.a.start + ld.tile * kTile + warp * 16 + (lane & 15);
            row_in = pos < ld.a.len && pos >= 0;
            if (row_in) page = __ldg(p.r.pages + ld.s * p.r.ld_pages + (pos >> p.c.page_log2));
            row_slot = pos & ((1 << p.c.page_log2) - 1);
            row_head = ld.seg % p.c.n_kv;
        }
        ++fetched;
    };
    int loaded = 0;
    auto issue = [&](int stage) {  // the copies of the unit whose page ids were fetched last
        if (loaded < count) {
            if (row_in && (page < 0 || page >= p.c.n_pages)) {
                row_in = false;
                record_status(p.status, kDevBadPage);
            }
            row_off = row_in ? page * p.c.ld_page + row_slot * p.c.ld_slot + row_head * p.c.ld_head : -1;
            uint8_t* const kd = ring + stage * S::kStage;
            uint8_t* const vd = kd + kTile * kRB;
#pragma unroll
            for (int i = 0; i < kChunks / 2; ++i) {
                const int idx = i * 32 + lane, r = idx / kChunks, c = idx % kChunks, row = warp * 16 + r;
                const int64_t off = __shfl_sync(0xFFFFFFFFu, row_off, r);
                const bool in = off >= 0;
                const int64_t byte = in ? off * (kE4M3 ? 1 : 2) + c * 16 : 0;
                ptx::cp_async_16(kd + (kE4M3 ? piece_k8<kRB>(row, c) : piece<kRB>(row, c)), static_cast<const char*>(p.c.k) + byte, in);
                ptx::cp_async_16(vd + piece<kRB>(row, c), static_cast<const char*>(p.c.v) + byte, in);
            }
        }
        ++loaded;
        ptx::cp_async_commit();
    };
    fetch();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        issue(i);
        fetch();
    }

    float o[kWR][kNB][4], m[kWR][2], l[kWR][2], f[kWR][2];
    int hi[kWR][2], lo[kWR][2];        // the positions that the row sees
    uint32_t qf[kQReg ? kWR : 1][kQReg ? kKS : 1][4];
    int stage = 0;
    bool opens = true;

    for (int j = 0; j < count; ++j) {
        const int h = cu.seg % p.c.n_kv, row0 = cu.seg / p.c.n_kv * kRows;
        const int rows = min(kRows, cu.a.n * p.group - row0);
        if (opens) {
            // ---- the rows' queries
            constexpr int kQC = kD / 8;
#pragma unroll 2
            for (int i = tid; i < kRows * kQC; i += kThreads) {
                const int r = i / kQC, c = i % kQC;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int at = (row0 + r) / p.group, head = h * p.group + (row0 + r) % p.group;
                    v = __ldg(reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(cu.a.beg + at) * p.ld_q + head * kD + c * 8));
                }
                if constexpr (!kE4M3) {
                    *reinterpret_cast<uint4*>(qs + piece<kQB>(r, c)) = v;
                } else {
                    // FP16 with the row's largest in [2^14, 2^15), columns in the order in which the keys' bytes come:
                    // 16 m + k of a block of 64 is element 16 t + 4 m + e, t and e as the fragments have them
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t big = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) big = max(big, max((w[x] << 16) & 0x7FFF0000u, w[x] & 0x7FFF0000u));
#pragma unroll
                    for (int x = kQC / 2; x > 0; x >>= 1) big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, x));
                    const int shift = big ? max(-110, min(100, 14 + 127 - static_cast<int>(big >> 23))) : 0;
                    const float by = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
                    if (c == 0) qscale[r] = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int d = c * 8 + 2 * x, rem = d % 64, k = rem % 4 / 2 * 8 + rem / 16 * 2;
                        const int col = d / 64 * 64 + rem % 16 / 4 * 16 + k;
                        *reinterpret_cast<uint32_t*>(qs + piece<kQB>(r, col / 8) + col % 8 * 2) =
                            pack_f16x2(__uint_as_float(w[x] << 16) * by, __uint_as_float(w[x] & 0xFFFF0000u) * by);
                    }
                }
            }
            __syncthreads();
            if constexpr (kQReg) {
#pragma unroll
                for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
                    for (int ks = 0; ks < kKS; ++ks) ldsm4(qs_a + piece<kQB>(mt * 16 + (lane & 15), 2 * ks + lane / 16), qf[mt][ks]);
            }
            const float sc = p.scale * 1.44269504088896340736f * (kE4M3 && p.c.k_scale ? __ldg(p.c.k_scale + h) : 1.0f);
#pragma unroll
            for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = mt * 16 + g + x * 8;
                    hi[mt][x] = cu.a.len - cu.a.n + (row0 + r) / p.group;
                    lo[mt][x] = p.window > 0 ? static_cast<int>(max(static_cast<int64_t>(0), static_cast<int64_t>(hi[mt][x]) - p.window + 1)) : 0;
                    f[mt][x] = kE4M3 ? sc * qscale[r] : sc;
                    m[mt][x] = -INFINITY;
                    l[mt][x] = 0.0f;
                }
#pragma unroll
            for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[mt][nb][x] = 0.0f;
            opens = false;
        }

        // ---- S = Q K^T of this warp's 16 tokens
        ptx::cp_async_wait<kStages - 2>();
        __syncwarp();
        const uint32_t ks_a = ring_a + stage * S::kStage, vs_a = ks_a + kTile * kRB;
        float sc[kWR][2][4];
#pragma unroll
        for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[mt][nb][x] = 0.0f;
        auto q_frag = [&](int mt, int ks, uint32_t (&a)[4]) {
            if constexpr (kQReg) {
#pragma unroll
                for (int x = 0; x < 4; ++x) a[x] = qf[mt][ks][x];
            } else {
                ldsm4(qs_a + piece<kQB>(mt * 16 + (lane & 15), 2 * ks + lane / 16), a);
            }
        };
        if constexpr (!kE4M3) {
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                uint32_t b[4];
                ldsm4(ks_a + piece<kRB>(warp * 16 + (lane & 7) + (lane >> 4) * 8, 2 * ks + ((lane >> 3) & 1)), b);
#pragma unroll
                for (int mt = 0; mt < kWR; ++mt) {
                    uint32_t a[4];
                    q_frag(mt, ks, a);
                    mma<false>(sc[mt][0], a, b[0], b[1]);
                    mma<false>(sc[mt][1], a, b[2], b[3]);
                }
            }
        } else {
#pragma unroll
            for (int blk = 0; blk < kD / 64; ++blk) {
                uint32_t w[2][4];
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    const uint32_t at = ks_a + piece_k8<kRB>(warp * 16 + nb * 8 + g, 4 * blk + t4);
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[nb][0]), "=r"(w[nb][1]), "=r"(w[nb][2]), "=r"(w[nb][3])
                                 : "r"(at)
                                 : "memory");
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t b[2][2];
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        b[nb][0] = e4m3x2_to_f16x2(w[nb][x] & 0xFFFFu);
                        b[nb][1] = e4m3x2_to_f16x2(w[nb][x] >> 16);
                    }
#pragma unroll
                    for (int mt = 0; mt < kWR; ++mt) {
                        uint32_t a[4];
                        q_frag(mt, 4 * blk + x, a);
                        mma<true>(sc[mt][0], a, b[0][0], b[0][1]);
                        mma<true>(sc[mt][1], a, b[1][0], b[1][1]);
                    }
                }
            }
        }

        // ---- scores in powers of two, masks, maxima
        const int pos0 = cu.a.start + cu.tile * kTile;
        // some row does not see some token (rows further down see later ones)
        const int first_row = cu.a.len - cu.a.n + row0 / p.group, last_row = cu.a.len - cu.a.n + (row0 + rows - 1) / p.group;
        const bool edge = pos0 + kTile - 1 > first_row || (p.window > 0 && static_cast<int64_t>(pos0) + p.window <= last_row);
#pragma unroll
        for (int mt = 0; mt < kWR; ++mt) {
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float v = sc[mt][nb][x] * f[mt][x / 2];
                    if (edge) {
                        const int pos = pos0 + warp * 16 + nb * 8 + 2 * t4 + (x & 1);
                        if (pos > hi[mt][x / 2] || pos < lo[mt][x / 2]) v = -INFINITY;
                    }
                    sc[mt][nb][x] = v;
                }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = fmaxf(fmaxf(sc[mt][0][2 * x], sc[mt][0][2 * x + 1]), fmaxf(sc[mt][1][2 * x], sc[mt][1][2 * x + 1]));
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
                if (t4 == 0) wmax[(mt * 16 + g + x * 8) * 4 + warp] = v;
            }
        }
        __syncthreads();  // the maxima are there, and every warp is done with the unit before

        issue(stage == 0 ? kStages - 1 : stage - 1);
        fetch();

        // ---- weights
        bool moved = false;
        float alpha[kWR][2];
#pragma unroll
        for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4 w = *reinterpret_cast<const float4*>(wmax + (mt * 16 + g + x * 8) * 4);
                const float to = fmaxf(fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)), m[mt][x]);
                moved |= to > m[mt][x];
                const float by = to == -INFINITY ? 0.0f : to;  // a row that has seen nothing yet
                alpha[mt][x] = exp2_fast(m[mt][x] - by);
                m[mt][x] = to;
                float sum = 0.0f;
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    const float u = exp2_fast(sc[mt][nb][2 * x] - by), v = exp2_fast(sc[mt][nb][2 * x + 1] - by);
                    sum += u + v;
                    const uint32_t at = ps_a + piece<128>(mt * 16 + g + x * 8, 2 * warp + nb) + 4 * t4;
                    if constexpr (kE4M3) {
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(pack_f16x2(u, v)) : "memory");
                    } else {
                        const uint32_t high = pack_bf16x2(u, v);
                        const uint32_t low = pack_bf16x2(u - bf16_to_f32(high & 0xFFFFu), v - bf16_to_f32(high >> 16));
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(high) : "memory");
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + kRows * kTile * 2), "r"(low) : "memory");
                    }
                }
                l[mt][x] = l[mt][x] * alpha[mt][x] + sum;
            }
        if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
            for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
                for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[mt][nb][x] *= alpha[mt][x / 2];
        }
        __syncthreads();  // the weights are there

        // ---- O += P V, this warp's quarter of the columns
        if (edge && cu.a.n > 1) {
            // A token that only some rows see may hold infinities or NaN: such values are added row by row
            // and then taken out, for a weight of 0 times them is no 0.
            constexpr int kQuarter = kRB / 4;  // bytes of a token that this warp takes
            uint8_t* const vs = ring + stage * S::kStage + kTile * kRB;
            auto odd = [&](uint32_t w) {
                if constexpr (kE4M3) {
                    bool any = false;
#pragma unroll
                    for (int b = 0; b < 4; ++b) any |= ((w >> (8 * b)) & 0x7Fu) == 0x7Fu;
                    return any;
                } else {
                    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
                }
            };
            for (int tok = 0; tok < kTile; ++tok) {
                uint32_t w = 0;
                if (lane < kQuarter / 4) w = *reinterpret_cast<const uint32_t*>(vs + piece<kRB>(tok, (warp * kQuarter + lane * 4) / 16) + (warp * kQuarter + lane * 4) % 16);
                if (!__any_sync(0xFFFFFFFFu, odd(w))) continue;
                const int pos = pos0 + tok;
#pragma unroll
                for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
                    for (int nb = 0; nb < kNB; ++nb)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if (pos > hi[mt][x / 2] || pos < lo[mt][x / 2]) continue;
                            const uint8_t* pp = ps + piece<128>(mt * 16 + g + x / 2 * 8, tok / 8) + tok % 8 * 2;
                            float wt, val;
                            if constexpr (kE4M3) {
                                const int d = warp * (kD / 4) + nb / 2 * 16 + 4 * t4 + 2 * (x & 1) + nb % 2;
                                wt = f16_to_f32(*reinterpret_cast<const uint16_t*>(pp));
                                val = f16_to_f32(e4m3x2_to_f16x2(vs[piece<kRB>(tok, d / 16) + d % 16]) & 0xFFFFu);
                            } else {
                                const int d = warp * (kD / 4) + nb * 8 + 2 * t4 + (x & 1);
                                wt = bf16_to_f32(*reinterpret_cast<const uint16_t*>(pp)) +
                                     bf16_to_f32(*reinterpret_cast<const uint16_t*>(pp + kRows * kTile * 2));
                                val = bf16_to_f32(*reinterpret_cast<const uint16_t*>(vs + piece<kRB>(tok, d / 8) + d % 8 * 2));
                            }
                            o[mt][nb][x] += wt * val;
                        }
                __syncwarp();
                if (lane < kQuarter / 4) *reinterpret_cast<uint32_t*>(vs + piece<kRB>(tok, (warp * kQuarter + lane * 4) / 16) + (warp * kQuarter + lane * 4) % 16) = 0;
                __syncwarp();
            }
        }
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
            uint32_t a[kWR][4], al[kE4M3 ? 1 : kWR][4];
#pragma unroll
            for (int mt = 0; mt < kWR; ++mt) {
                const uint32_t at = ps_a + piece<128>(mt * 16 + (lane & 15), 2 * kk + lane / 16);
                ldsm4(at, a[mt]);
                if constexpr (!kE4M3) ldsm4(at + kRows * kTile * 2, al[mt]);
            }
            const int tok = kk * 16 + (lane & 15);  // lanes 16 .. 31: the next piece of columns
            if constexpr (!kE4M3) {
#pragma unroll
                for (int nb = 0; nb < kNB; nb += 2) {
                    uint32_t b[4];
                    ldsm4t(vs_a + piece<kRB>(tok, warp * (kD / 32) + nb + (lane >> 4)), b);
#pragma unroll
                    for (int mt = 0; mt < kWR; ++mt) {
                        mma<false>(o[mt][nb], a[mt], b[0], b[1]);
                        mma<false>(o[mt][nb + 1], a[mt], b[2], b[3]);
                        mma<false>(o[mt][nb], al[mt], b[0], b[1]);
                        mma<false>(o[mt][nb + 1], al[mt], b[2], b[3]);
                    }
                }
            } else {
                // a piece is 16 columns: the transposed load gives bytes of two columns of two tokens
#pragma unroll
                for (int ch = 0; ch < (kNB + 3) / 4; ++ch) {
                    // two pieces of columns; a quarter of a single one (D = 64) loads it twice
                    const int c = warp * (kD / 64) + (kNB >= 4 ? 2 * ch + (lane >> 4) : 0);
                    uint32_t b[4];
                    ldsm4t(vs_a + piece<kRB>(tok, c), b);
#pragma unroll
                    for (int half = 0; half < (kNB >= 4 ? 2 : 1); ++half) {
                        const uint32_t u = __byte_perm(b[2 * half], 0, 0x3120), v = __byte_perm(b[2 * half + 1], 0, 0x3120);
                        const uint32_t b00 = e4m3x2_to_f16x2(u & 0xFFFFu), b01 = e4m3x2_to_f16x2(v & 0xFFFFu);
                        const uint32_t b10 = e4m3x2_to_f16x2(u >> 16), b11 = e4m3x2_to_f16x2(v >> 16);
#pragma unroll
                        for (int mt = 0; mt < kWR; ++mt) {
                            mma<true>(o[mt][4 * ch + 2 * half], a[mt], b00, b01);
                            mma<true>(o[mt][4 * ch + 2 * half + 1], a[mt], b10, b11);
                        }
                    }
                }
            }
        }
        if (++stage == kStages) stage = 0;

        // ---- the end of a (request, head): finished here, or a part of it
        const bool last = j == count - 1, closes = cu.tile == cu.a.tiles - 1;
        if (last || closes) {
#pragma unroll
            for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = l[mt][x];
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
                    v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
                    if (t4 == 0) wsum[(mt * 16 + g + x * 8) * 4 + warp] = v;
                }
            __syncthreads();
            const bool whole = closes && cu.tile <= j;  // its first unit is in this run as well
            // a part: slot 0 where the (request, head) holds the run's first unit, else 1
            const int64_t slot = blockIdx.x * 2 + (cu.tile >= j ? 0 : 1);
#pragma unroll
            for (int mt = 0; mt < kWR; ++mt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = mt * 16 + g + x * 8;
                    const float4 w = *reinterpret_cast<const float4*>(wsum + r * 4);
                    const float sum = (w.x + w.y) + (w.z + w.w);
                    if (r >= rows) continue;
                    if (whole) {
                        const int at = (row0 + r) / p.group, head = h * p.group + (row0 + r) % p.group;
                        const int64_t t = cu.a.beg + at;
                        float by = sum == 0.0f ? 0.0f : 1.0f / sum;
                        if (kE4M3 && p.c.v_scale) by *= __ldg(p.c.v_scale + h);
                        uint16_t* const to = p.out + t * p.ld_out + head * kD;
#pragma unroll
                        for (int nb = 0; nb < kNB; ++nb) {
                            const float u = o[mt][nb][2 * x] * by, v = o[mt][nb][2 * x + 1] * by;
                            if constexpr (!kE4M3) {
                                *reinterpret_cast<uint32_t*>(to + warp * (kD / 4) + nb * 8 + 2 * t4) = pack_bf16x2(u, v);
                            } else if (nb % 2 == 0) {
                                const float u1 = o[mt][nb + 1][2 * x] * by, v1 = o[mt][nb + 1][2 * x + 1] * by;
                                *reinterpret_cast<uint2*>(to + warp * (kD / 4) + nb / 2 * 16 + 4 * t4) = make_uint2(pack_bf16x2(u, u1), pack_bf16x2(v, v1));
                            }
                        }
                        if (p.lse && warp == 0 && t4 == 0)
                            p.lse[t * p.n_q + head] = sum == 0.0f ? -INFINITY : (m[mt][x] + log2f(sum)) * 0.69314718055994530942f;
                    } else {
                        float* const to = p.part + (slot * kRows + r) * kD;
#pragma unroll
                        for (int nb = 0; nb < kNB; ++nb) {
                            const float u = o[mt][nb][2 * x], v = o[mt][nb][2 * x + 1];
                            if constexpr (!kE4M3) {
                                *reinterpret_cast<float2*>(to + warp * (kD / 4) + nb * 8 + 2 * t4) = make_float2(u, v);
                            } else if (nb % 2 == 0) {
                                const float u1 = o[mt][nb + 1][2 * x], v1 = o[mt][nb + 1][2 * x + 1];
                                *reinterpret_cast<float4*>(to + warp * (kD / 4) + nb / 2 * 16 + 4 * t4) = make_float4(u, u1, v, v1);
                            }
                        }
                        if (warp == 0 && t4 == 0) *reinterpret_cast<float2*>(p.part_ml + (slot * kRows + r) * 2) = make_float2(m[mt][x], sum);
                    }
                }
            opens = true;
        }
        if (!last) cu.next(p);
    }
    ptx::cp_async_wait<0>();
}

// ---- the join: a row's parts, in the order of the runs. Few parts: a warp a row; many: the CTA's eight warps.
constexpr int kJoinWarps = 8;

template <int kD, bool kE4M3, int kWR>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attention_join(const __grid_constant__ AttentionArgs p, int ctas, int segs_most, int rows_per_cta)
{
    constexpr int kRows = 16 * kWR, kV = kD / 32;  // columns a lane: lane * kV ..
    __shared__ float sm_o[kJoinWarps][kD], sm_ml[kJoinWarps][2];
    const int s = blockIdx.x / segs_most, seg = blockIdx.x % segs_most, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t first = p.prefix[s], units = p.prefix[s + 1] - first, total = p.prefix[p.r.S];
    if (units == 0) return;
    bool bad;
    const Span a = span_of<kRows>(p, s, bad);
    if (seg >= a.segs) return;
    const Cut cut(total, runs_of(total, ctas));
    const int64_t u0 = first + static_cast<int64_t>(seg) * a.tiles, u1 = u0 + a.tiles;
    const int c0 = cut.run(u0), c1 = cut.run(u1 - 1);
    if (c0 == c1) return;  // finished by its run
    const int h = seg % p.c.n_kv, row0 = seg / p.c.n_kv * kRows, rows = min(kRows, a.n * p.group - row0);
    const bool alone = c1 - c0 < 16;
    const int r0 = blockIdx.y * rows_per_cta, r1 = min(rows, r0 + rows_per_cta);
    const bool from_start = cut.first(c0) == u0;

    for (int r = r0 + (alone ? warp : 0); r < r1; r += alone ? kJoinWarps : 1) {
        // this warp's parts: all of them, or every eighth run of 8
        float mx = -INFINITY, sum = 0.0f, o[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) o[i] = 0.0f;
        const int n = c1 - c0 + 1, per = (n + kJoinWarps - 1) / kJoinWarps;
        const int b = alone ? 0 : min(n, warp * per), e = alone ? n : min(n, b + per);
        for (int i0 = b; i0 < e; i0 += 32) {
            const int i = i0 + lane;
            float2 ml = make_float2(-INFINITY, 0.0f);
            auto slot_of = [&](int x) { return static_cast<int64_t>(c0 + x) * 2 + (x == 0 && !from_start ? 1 : 0); };
            if (i < e) ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (slot_of(i) * kRows + r) * 2));
            float top = ml.x;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            const float to = fmaxf(mx, top), by = to == -INFINITY ? 0.0f : to;
            const float keep = exp2_fast(mx - by), w = exp2_fast(ml.x - by);
            mx = to;
            float part = w * ml.y;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, x);
            sum = sum * keep + part;
#pragma unroll
            for (int x = 0; x < kV; ++x) o[x] *= keep;
            const int in = min(32, e - i0);
#pragma unroll 8
            for (int x = 0; x < in; ++x) {
                const float wx = __shfl_sync(0xFFFFFFFFu, w, x);
                const float* from = p.part + (slot_of(i0 + x) * kRows + r) * kD + lane * kV;
                if constexpr (kV == 2) {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(from));
                    o[0] += wx * v.x;
                    o[1] += wx * v.y;
                } else {
#pragma unroll
                    for (int y = 0; y < kV; y += 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(from + y));
                        o[y] += wx * v.x;
                        o[y + 1] += wx * v.y;
                        o[y + 2] += wx * v.z;
                        o[y + 3] += wx * v.w;
                    }
                }
            }
        }
        if (!alone) {
#pragma unroll
            for (int x = 0; x < kV; ++x) sm_o[warp][lane * kV + x] = o[x];
            if (lane == 0) {
                sm_ml[warp][0] = mx;
                sm_ml[warp][1] = sum;
            }
            __syncthreads();
            if (warp == 0) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sm_ml[w][0]);
                const float by = top == -INFINITY ? 0.0f : top;
                sum = 0.0f;
#pragma unroll
                for (int x = 0; x < kV; ++x) o[x] = 0.0f;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) {
                    const float f = exp2_fast(sm_ml[w][0] - by);
                    sum += f * sm_ml[w][1];
#pragma unroll
                    for (int x = 0; x < kV; ++x) o[x] += f * sm_o[w][lane * kV + x];
                }
                mx = top;
            }
        }
        if (alone || warp == 0) {
            const int at = (row0 + r) / p.group, head = h * p.group + (row0 + r) % p.group;
            const int64_t t = a.beg + at;
            float by = sum == 0.0f ? 0.0f : 1.0f / sum;
            if (kE4M3 && p.c.v_scale) by *= __ldg(p.c.v_scale + h);
            uint16_t* const to = p.out + t * p.ld_out + head * kD + lane * kV;
#pragma unroll
            for (int x = 0; x < kV; x += 2) *reinterpret_cast<uint32_t*>(to + x) = pack_bf16x2(o[x] * by, o[x + 1] * by);
            if (p.lse && lane == 0) p.lse[t * p.n_q + head] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994530942f;
        }
        if (!alone) __syncthreads();
    }
}

// the 16-row tiles of a CTA: what max_new tokens of a key head's queries need, at most four
int row_tiles(int group, int max_new)
{
    const int rows = group * max_new;
    return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

// CTAs of the main launch; two an SM at most leave partial sums
int ctas_of(int sms, int per_sm) { return sms * per_sm; }

template <int kD, bool kE4M3, int kWR>
cudaError_t launch(const AttentionArgs& a, int sms, cudaStream_t stream)
{
    using S = Shape<kD, kE4M3, kWR>;
    static bool set = false;
    if (!set) {
        cudaError_t e = cudaFuncSetAttribute(k_paged_attention<kD, kE4M3, kWR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        set = true;
    }
    const int ctas = ctas_of(sms, S::kSmem <= kHalfSmem ? 2 : 1);
    cudaError_t e = launch_pdl(k_paged_attention<kD, kE4M3, kWR>, dim3(ctas), dim3(kThreads), S::kSmem, stream, a);
    if (e != cudaSuccess) return e;
    // few rows: one a CTA of the join, else eight
    const int segs = a.c.n_kv * ((a.max_new * a.group + S::kRows - 1) / S::kRows);
    const int per = static_cast<int64_t>(a.T) * a.n_q <= 2048 ? 1 : 8;
    return launch_pdl(k_attention_join<kD, kE4M3, kWR>, dim3(static_cast<unsigned>(a.r.S) * segs, (S::kRows + per - 1) / per),
                      dim3(kJoinWarps * 32), 0, stream, a, ctas, segs, per);
}

template <int kD, bool kE4M3>
cudaError_t launch_rows(const AttentionArgs& a, int sms, cudaStream_t stream)
{
    switch (row_tiles(a.group, a.max_new)) {
    case 1: return launch<kD, kE4M3, 1>(a, sms, stream);
    case 2: return launch<kD, kE4M3, 2>(a, sms, stream);
    default: return launch<kD, kE4M3, 4>(a, sms, stream);
    }
}

template <bool kE4M3>
cudaError_t launch_d(const AttentionArgs& a, int sms, cudaStream_t stream)
{
    switch (a.c.D) {
    case 64: return launch_rows<64, kE4M3>(a, sms, stream);
    case 128: return launch_rows<128, kE4M3>(a, sms, stream);
    case 256: return launch_rows<256, kE4M3>(a, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// header, prefix, maxima and sums, partial outputs: two slots a CTA
size_t ml_at(int S) { return sizeof(WsHeader) + up256((static_cast<size_t>(S) + 1) * 8); }
size_t part_at(int S, int rows, int sms) { return ml_at(S) + up256(static_cast<size_t>(ctas_of(sms, 2)) * 2 * rows * 8); }

}  // namespace

size_t attention_workspace_bytes(int S, int n_q, int n_kv, int D, int max_new, int sms)
{
    const int rows = 16 * row_tiles(n_q / n_kv, max_new);
    return part_at(S, rows, sms) + static_cast<size_t>(ctas_of(sms, 2)) * 2 * rows * D * 4;
}

cudaError_t launch_paged_attention(AttentionArgs a, void* ws, int sms, cudaStream_t stream)
{
    char* const base = static_cast<char*>(ws);
    const int rows = 16 * row_tiles(a.group, a.max_new);
    a.prefix = reinterpret_cast<int64_t*>(base + sizeof(WsHeader));
    a.part_ml = reinterpret_cast<float*>(base + ml_at(a.r.S));
    a.part = reinterpret_cast<float*>(base + part_at(a.r.S, rows, sms));
    return a.c.e4m3 ? launch_d<true>(a, sms, stream) : launch_d<false>(a, sms, stream);
}

}  // namespace moe
