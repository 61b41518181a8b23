// paged_attention.cuh -- attention of a few new tokens of every request over a paged cache:
//   out = sum_t softmax_t(scale q . k_t) v_t over the tokens that a row sees, in one pass over keys and values
// with the running maximum m and sum l of the softmax: o <- o 2^(m - m') + 2^(s - m') v.
//
// Work: a unit is 64 cached tokens (128 where they have 128 bytes or less) of one key head against up to kRows rows (new
// tokens x query heads of that key head). The units of all requests, in order, are cut into runs of equal cost, one a
// CTA, so ragged lengths balance by themselves. A (request, head) whose units lie in one run is finished there; of the others
// every run leaves o, m and l in the workspace, and a second launch adds them in the order of the runs.
// A CTA streams K and V through a ring in shared memory: two warps load (cp.async of 16 bytes a lane, addresses from
// the page table, which is read a unit ahead; a token behind the end is filled with zeros). The rows' eights are dealt to
// one to four groups of four warps. Of a unit each warp of a group takes a quarter of the tokens for K Q^T, the four exchange
// maxima and weights through shared memory, and each takes a quarter of the columns of V^T P^T, so the accumulators need no
// join.
// mma.sync with the tokens (and V's columns) on its M side: rows are padded to eight, not sixteen. A token's keys and values
// are 4 D bytes in bf16 (2 D in 8 bits) and take 6 D flops a row, the weights' two parts counted: 12 flops a byte for 8 rows
// (24), 48 for 32 (96), at the memory's rate 80 to 640 TFLOP/s. More than 64 rows of a key head read K and V again for every 64
// (16 requests of 16 tokens over to 4,000, 16 heads on 2 of 256: 69 us, their bytes in 11): decode steps and short windows are
// what this is for.
// Weights in the second product: of a bf16 cache two bf16 values (16 bits; one would add an error of the size of the output's
// own rounding, three took 39.4 us for 36.2 in 200 windows of 1,024 and 133 for 116 with 128 rows a key head, for bits that
// are 2^-8 of the output's rounding); of an E4M3 cache, whose codes become FP16 exactly, two FP16 values (22 bits) in parts of
// 2^-15 of the largest. (One, 11 bits, is off by an eighth of the output's rounding: 1 request over 300,001 59.5 us either
// way, 200 over to 2,000, 14 heads on 2 of 64, 22.0 and 20.8, 100 of four tokens over to 2,000, 32 on 4 of 128, 64.7 and 60.4.)
// q of an E4M3 cache is scaled to FP16's range by a power of two a row (exact where q is not 2^-30 of the row's largest).
// Measured: 64 requests of ragged lengths to 8,192, 32 heads on 8 of 128: 168 us, 6.2 TB/s (93 % of what a copy
// reaches); one request over 300,001 tokens in 8 bits, 16 heads on 2 of 256: 58 us, 5.3 TB/s, 10 us of it the two launches,
// the first loads and the join; 200 verify windows of one to three tokens, 14 heads on 2 of 64, window 1,024: 34 us, bound
// by its groups' chains, two barriers and two ways through shared memory a unit (49 % of the issue slots and 15 % of the
// tensor pipe are in use); 4 tokens over 4,100, 16 heads on 2 of 256: 12 us, one unit's chain and the join's.
#pragma once
#include <climits>

#include "attention.cuh"
#include "ptx_cluster.cuh"

namespace moe {

namespace attention {

constexpr int kWarps = 4, kGroup = 32 * kWarps;  // a group of warps that computes
// Warps that load. (Four took issue slots: 200 windows of 1,024 61 us against 54.)
constexpr int kLoaders = 2;
// A unit costs so much besides the groups that have rows in it. (2, 4, 5, 7 and 100, where the rows hardly count: 200
// windows of 1,024 35.9, 35.7, 36.0, 36.8, 38.1 us, 200 requests of one to three tokens over to 4,096 58.1, 55.4, 56.3, 56.2,
// 61.1.)
constexpr int kUnit = 4;
// What the begin and the end of a (request, head) cost, in units: queries, sums, output. (0, 1, 2, 4 of them: 200 windows of
// 1,024 49.7, 42.8, 42.6, 43.6 us, 200 requests to 500 with heads of 128 40.8, 34.8, 34.3, 34.8.)
constexpr int kExtra = 2;

// Tokens of a unit: 16 a warp, or of short rows 32, for what a unit costs besides its products is then for twice as many.
// (64 and 128 of them, 200 requests, 14 heads on 2 of 64: windows of 1,024 39.8 and 37.7 us, three new tokens over to 4,096
// 68.9 and 60.2, one over to 2,000 in 8 bits 23.1 and 21.0; against it, one over to 1,024 19.8 and 20.4.)
template <int kD, bool kE4M3>
constexpr int tile_of() { return kD * (kE4M3 ? 1 : 2) <= 128 ? 128 : 64; }

// kRG: groups, kNR: a group's rows in eights
template <int kD, bool kE4M3, int kRG, int kNR>
struct Shape {
    static constexpr int kGroups = kRG, kThreads = kRG * kGroup + kLoaders * 32;
    static constexpr int kRows = 8 * kRG * kNR;
    static constexpr int kRowBytes = kD * (kE4M3 ? 1 : 2);       // of a cached token's head
    static constexpr int kTile = tile_of<kD, kE4M3>();
    static constexpr int kStage = 2 * kTile * kRowBytes;         // K, V
    static constexpr int kQ = kRows * kD * 2;
    static constexpr int kParts = 2;                             // values that hold a weight
    static constexpr int kP = kRows * kTile * 2 * kParts;
    static constexpr int kFixed = kQ + kP + kRows * (2 * kWarps * 4 + 8) + 512;
    // As many CTAs an SM as hold three stages each, and as the registers of so many rows allow: one to three. Two of two
    // stages are better than one, too (100 requests of 4 new tokens over to 2,000, 32 heads on 4 of 128: 67 us against 77),
    // but of heads of 256, whose sums two CTAs' registers do not hold (60 such requests, 16 heads on 2, 8 bits: 39.5, 35.2).
    static constexpr int kByRegs = kRG == 4 ? 1 : kRG >= 2 ? 2 : 3;
    // (a multiprocessor's 228 KB less 1 KB a CTA, and 10 KB in which the join's CTAs can wait)
    static constexpr int most(int ctas) { return (218 / ctas - 1) * 1024; }
    static constexpr int by_smem(int ctas) { return ctas == 1 || (most(ctas) - kFixed) / kStage >= (ctas == 2 && kD <= 128 ? 2 : 3) ? ctas : by_smem(ctas - 1); }
    static constexpr int kCtas = by_smem(kByRegs);
    static constexpr int kFit = (most(kCtas) - kFixed) / kStage;
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kSmem = kFixed + kStages * kStage;
    static_assert(kStages >= 2 && kSmem <= most(kCtas), "shared memory");
};

// ---- the cut into runs of equal cost. A (request, head) of n units that cost w each costs (kExtra + n) w, its unit i lying
// at offset (kExtra + i) w: a border inside a unit is one before it, a border inside the extra part one before the first
// unit. No run costs less than a unit, so there is a border in each unit at the most.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)  // of numbers that mostly fit 32 bits
{
    return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}
struct Cut {
    int64_t q, r;  // runs 0 .. r - 1 have q + 1 units, the others q
    __device__ int64_t first(int64_t c) const { return c * q + (c < r ? c : r); }
    __device__ int run(int64_t u) const { return static_cast<int>(u < r * (q + 1) ? quotient(u, q + 1) : r + quotient(u - r * (q + 1), q)); }
};

// The token of a row of a key head's queries (less than 1,088 of them): row / group, by a multiplication.
__device__ __forceinline__ int token_of(const AttentionArgs& p, int row) { return static_cast<int>(static_cast<unsigned>(row) * p.group_mul >> 16); }

struct Span {
    int beg, n, len, start, tiles, segs, w;  // rows; tokens; first token seen; units along the tokens; (head, row block) pairs
    __device__ int64_t each() const { return static_cast<int64_t>(tiles + kExtra) * w; }
    __device__ int64_t cost() const { return tiles ? each() * segs : 0; }
};

template <class S>
__device__ __forceinline__ Span span_of(const AttentionArgs& p, int s, bool& bad)
{
    const Request r = load_request(p.r, s, p.T, p.max_new, bad);
    Span a{r.beg, r.n, r.len, 0, 0, 0, 0};
    if (r.n == 0) return a;
    if (p.window > 0) {
        const int64_t first = static_cast<int64_t>(r.len) - r.n - p.window + 1;
        a.start = first > 0 ? static_cast<int>(first) : 0;
    }
    // (a request that sees nothing has a unit, too)
    a.tiles = max(1, static_cast<int>((static_cast<int64_t>(r.len) - a.start + S::kTile - 1) / S::kTile));
    a.segs = p.c.n_kv * ((r.n * p.group + S::kRows - 1) / S::kRows);
    a.w = S::kGroups == 1 ? 1 : kUnit + min(S::kGroups, (r.n * p.group + 7) / 8);
    return a;
}

// A place in the order of units.
template <class S>
struct Cursor {
    Span a;
    int s, seg, tile;
    // The next unit (there is one).
    __device__ void next(const AttentionArgs& p)
    {
        if (++tile < a.tiles) return;
        tile = 0;
        if (++seg < a.segs) return;
        seg = 0;
        bool bad;
        do a = span_of<S>(p, ++s, bad);
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
// Two 8 x 8 blocks of 16-bit values, stored transposed: lanes 0 .. 7 and 8 .. 15 give the rows' addresses.
__device__ __forceinline__ void stsm2t(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
template <bool kF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (kF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four E4M3 codes as FP16 values, exactly: the lower two and the upper two.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
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

// The elements of a word (four bytes or two halves) that are no finite numbers: their top bits.
template <bool kE4M3>
__device__ __forceinline__ uint32_t odd_mask(uint32_t w)
{
    if constexpr (kE4M3) return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // 0x7F: NaN
    else return (((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u);                // an exponent of all ones
}

template <int kD, bool kE4M3, int kRG, int kNR>
__global__ void __launch_bounds__(Shape<kD, kE4M3, kRG, kNR>::kThreads, Shape<kD, kE4M3, kRG, kNR>::kCtas) k_paged_attention(const __grid_constant__ AttentionArgs p)
{
    using S = Shape<kD, kE4M3, kRG, kNR>;
    constexpr int kThreads = S::kThreads, kCompute = kRG * kGroup;
    constexpr int kRows = S::kRows, kTile = S::kTile, kRB = S::kRowBytes, kChunks = kRB / 16, kStages = S::kStages;
    constexpr int kMQ = kTile / 64, kLoad = kTile / kLoaders;  // a warp's tokens in Q K^T in sixteens, in loading
    constexpr int kPB = kTile * 2;          // bytes of a row of weights
    constexpr int kQB = kD * 2;             // bytes of a row of q
    constexpr int kMT = kD / 64;            // 16-column tiles of a warp's quarter of the columns
    constexpr int kKS = kD / 16;            // steps of Q K^T
    constexpr bool kQReg = kNR * kKS <= 8;  // q's fragments stay in registers
    // m is so far below the largest score: FP16 weights are 2^15 at the most, and both parts together within 2^-22 of a weight
    // or 2^-25 (2^-40 of the largest); with 1 at the most, all that lies 2^-25 below the largest would be lost.
    constexpr float kLift = kE4M3 ? 15.0f : 0.0f;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const ring = smem;
    uint8_t* const qs = smem + kStages * S::kStage;
    uint8_t* const ps = qs + S::kQ;         // weights: [kRows][kTile] 16-bit, the high parts, then the low ones
    float* const wmax = reinterpret_cast<float*>(ps + S::kP);  // [kRows][kWarps]
    float* const wsum = wmax + kRows * kWarps;                 // [kRows][kWarps]
    float* const qscale = wsum + kRows * kWarps;               // [kRows] (E4M3) what the row of q was divided by
    int* const row_pos = reinterpret_cast<int*>(qscale + kRows);  // [kRows] the row's position
    int64_t* const found = reinterpret_cast<int64_t*>(row_pos + kRows);  // a sum a warp, then what the search found
    Cursor<S>* const start = reinterpret_cast<Cursor<S>*>(found + 20);
    uint64_t* const full = reinterpret_cast<uint64_t*>(found + 30);  // [kStages]
    uint64_t* const empty = full + kStages;                            // [kStages]
    uint64_t* const never = empty + kStages;
    int* const abort = reinterpret_cast<int*>(never + 1);
    int* const costs = abort + 1;  // a number a warp
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0), lane = tid % 32, g = lane / 4, t4 = lane % 4;
    const uint32_t ring_a = ptx::smem_u32(ring), qs_a = ptx::smem_u32(qs), ps_a = ptx::smem_u32(ps);

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(full + s, kLoaders * 32);  // the loading lanes
            ptx::mbar_init(empty + s, kRG * kWarps);
        }
        ptx::mbar_init(never, 1);
        *abort = 0;
        ptx::fence_mbar_init();
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    // a test makes the first wait run out: then it is for a barrier that nobody arrives at
    const bool stuck = *reinterpret_cast<const volatile int*>(&p.hooks->test_ready_extra) > 0;

    // ---- this CTA's run: the units before each request, a block of requests a thread
    const int block = (p.r.S + kThreads - 1) / kThreads, sb = min(p.r.S, tid * block), se = min(p.r.S, sb + block);
    int64_t mine = 0;
    int most = 1;  // what a unit costs at the most
    for (int s = sb; s < se; ++s) {
        bool bad;
        const Span a = span_of<S>(p, s, bad);
        mine += a.cost();
        if constexpr (kRG > 1) most = max(most, a.w);
        if (bad && blockIdx.x == 0) record_status(p.status, kDevBadRequest);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if constexpr (kRG > 1) most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 31) {
        found[warp] = incl;
        costs[warp] = most;
    }
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += found[w];
        total += found[w];
        if constexpr (kRG > 1) most = max(most, costs[w]);
    }
    const int runs = static_cast<int>(min(static_cast<int64_t>(gridDim.x), quotient(total, most)));
    Cut cut{0, 0};
    if (runs) {
        cut.q = quotient(total, runs);
        cut.r = total - cut.q * runs;
    }
    if (blockIdx.x == 0) {  // for the join
        int64_t u = before;
        for (int s = sb; s < se; ++s) {
            bool bad;
            p.prefix[s] = u;
            u += span_of<S>(p, s, bad).cost();
        }
        if (tid == 0) {
            p.prefix[p.r.S] = total;
            p.prefix[p.r.S + 1] = cut.q;
            p.prefix[p.r.S + 2] = cut.r;
        }
    }
    if (static_cast<int>(blockIdx.x) >= runs) return;
    // its first unit, and the place of both borders in the order of units
    const int64_t border[2] = {cut.first(blockIdx.x), cut.first(blockIdx.x + 1)};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (border[e] < before || border[e] >= before + mine) continue;
        int64_t u = border[e] - before;
        Cursor<S> c;
        for (c.s = sb;; ++c.s) {
            bool bad;
            c.a = span_of<S>(p, c.s, bad);
            if (u < c.a.cost()) break;
            u -= c.a.cost();
        }
        c.seg = static_cast<int>(quotient(u, c.a.each()));
        u -= c.seg * c.a.each();
        c.tile = max(0, static_cast<int>(kRG > 1 ? quotient(u, c.a.w) : u) - kExtra);
        start[e] = c;
    }
    __syncthreads();
    Cursor<S> cu = start[0];
    // the units between the borders
    int count;
    {
        const bool to_end = border[1] == total;
        const Cursor<S> end = start[1];
        const int last_s = to_end ? p.r.S : end.s;
        int64_t n = -(static_cast<int64_t>(cu.seg) * cu.a.tiles + cu.tile) + (to_end ? 0 : static_cast<int64_t>(end.seg) * end.a.tiles + end.tile);
        for (int s = cu.s; s < last_s; ++s) {
            bool bad;
            const Span a = s == cu.s ? cu.a : span_of<S>(p, s, bad);
            n += static_cast<int64_t>(a.tiles) * a.segs;
        }
        count = static_cast<int>(n);
    }
    // A bounded wait (a waiting warp takes no issue slots). After one that ran out there are no more: the rest runs on
    // whatever is there, to its end.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!ptx::mbar_try_wait(bar, parity) && *reinterpret_cast<volatile int*>(abort) == 0 && !ptx::mbar_wait(bar, parity)) {
            *reinterpret_cast<volatile int*>(abort) = 1;
            record_status(p.status, kDevTimeoutAttention);
        }
        __syncwarp();  // the warp's matrix products take all of its lanes
    };

    if (warp >= kRG * kWarps) {
        // ---- loads: a warp kLoad tokens of a unit, four lanes a token; page ids come a unit ahead
        const int lw = warp - kRG * kWarps;
        const int64_t v_from_k = static_cast<const char*>(p.c.v) - static_cast<const char*>(p.c.k);
        const uint32_t k_even = lw * kLoad * kRB + (kE4M3 ? piece_k8<kRB>(g, t4) : piece<kRB>(g, t4)), k_odd = k_even ^ 64;
        const uint32_t v_even = (kTile + lw * kLoad) * kRB + piece<kRB>(g, t4), v_odd = v_even ^ 64;
        const int mask = (1 << p.c.page_log2) - 1;
        int page[kLoad / 32];  // of the tokens lane, lane + 32
        unsigned pos = 0;      // the first one's position
        bool first = true;
        int64_t head_off = 0;
        auto fetch = [&]() {
            const int pos0 = cu.a.start + cu.tile * kTile, left = cu.a.len - pos0;  // (the unit's end may pass 2^31)
            pos = static_cast<unsigned>(pos0) + lw * kLoad + lane;
            if (first || cu.tile == 0) head_off = (cu.seg % p.c.n_kv) * p.c.ld_head;
            first = false;
#pragma unroll
            for (int x = 0; x < kLoad / 32; ++x)  // INT_MIN: no token
                page[x] = lw * kLoad + lane + x * 32 < left ? __ldg(p.r.pages + cu.s * p.r.ld_pages + ((pos + x * 32) >> p.c.page_log2)) : INT_MIN;
        };
        fetch();
        int s = 0;
        uint32_t ph = 1;
        for (int j = 0; j < count; ++j) {
            int64_t mine[kLoad / 32];
#pragma unroll
            for (int x = 0; x < kLoad / 32; ++x) {
                mine[x] = -1;
                if (static_cast<unsigned>(page[x]) < static_cast<unsigned>(p.c.n_pages))
                    mine[x] = (page[x] * p.c.ld_page + static_cast<int>((pos + x * 32) & mask) * p.c.ld_slot + head_off) * (kE4M3 ? 1 : 2);
                else if (page[x] != INT_MIN)
                    record_status(p.status, kDevBadPage);
            }
            if (j + 1 < count) {
                cu.next(p);
                fetch();
            }
            wait(empty + s, ph);
            uint8_t* const to = ring + s * S::kStage;
#pragma unroll
            for (int b = 0; b < kLoad / 8; ++b) {
                const int64_t off = __shfl_sync(0xFFFFFFFFu, mine[b / 4], b % 4 * 8 + g);
                const bool there = off >= 0;
                const char* const k = static_cast<const char*>(p.c.k) + (there ? off + t4 * 16 : 0);
                const char* const v = k + v_from_k;
#pragma unroll
                for (int i = 0; i < kChunks / 4; ++i) {
                    ptx::cp_async_16(to + b * 8 * kRB + (i & 1 ? k_odd : k_even) + i / 2 * 128, k + i * 64, there);
                    ptx::cp_async_16(to + b * 8 * kRB + (i & 1 ? v_odd : v_even) + i / 2 * 128, v + i * 64, there);
                }
            }
            ptx::cp_async_arrive_noinc(full + s);
            if (++s == kStages) { s = 0; ph ^= 1; }
        }
        ptx::cp_async_commit();
        ptx::cp_async_wait<0>();
        return;
    }

    if (stuck && !ptx::mbar_wait_us(never, 0, p.hooks->test_wait_us)) {
        *reinterpret_cast<volatile int*>(abort) = 1;
        record_status(p.status, kDevTimeoutAttention);
    }

    // group rg, its warp gw, thread gt; its rows are the eights rg, rg + kRG, ..
    const int rg = warp / kWarps, gw = warp % kWarps, gt = tid % kGroup;
    auto base_of = [&](int nr) { return (nr * kRG + rg) * 8; };
    auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + rg), "n"(kGroup) : "memory"); };  // of the group
    auto sync_all = [] { asm volatile("bar.sync 8, %0;" ::"n"(kCompute) : "memory"); };           // of all groups
    auto any_of = [](bool v) {
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.u32 q, %1, 0;\n\t"
            "bar.red.or.pred p, 8, %2, q;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(r)
            : "r"(static_cast<uint32_t>(v)), "n"(kCompute)
            : "memory");
        return r != 0;
    };

    // This lane's addresses in a stage, in q and in the weights. A step along a row is an exclusive or: pieces are swapped
    // within 128 bytes, and what a step adds are bits that the first piece's number does not have.
    const uint32_t k_lane = ring_a + (kE4M3 ? piece_k8<kRB>(gw * 16 + g, t4) : piece<kRB>(gw * 16 + (lane & 15), lane >> 4));
    const uint32_t v_lane = ring_a + kTile * kRB + (kE4M3 ? piece<kRB>(lane, gw * (kD / 64)) : piece<kRB>((lane & 7) + (lane >> 4) * 8, gw * (kD / 32) + ((lane >> 3) & 1)));
    const uint32_t q_lane = qs_a + piece<kQB>(lane & 7, lane >> 3), p_lane = ps_a + piece<kPB>(lane & 7, lane >> 3);
    const uint32_t p_mine = ps_a + piece<kPB>(lane & 7, 2 * gw + ((lane >> 3) & 1));

    float o[kMT][kNR][4], m[kNR][2], l[kNR][2];  // rows 8 nr + 2 t4, + 1; columns of v by g
    uint32_t qf[kQReg ? kNR : 1][kQReg ? kKS : 1][2];
    uint32_t stage_off = 0;
    int stage = 0;
    uint32_t phase = 0;
    bool opens = true;
    int h = 0, row0 = 0, rows = 0, live = 0, first_row = 0, before_window = -1;
    float factor = 0.0f;
    bool active = false;  // this group has rows

    for (int j = 0; j < count; ++j) {
        if (opens) {
            // ---- the rows' queries
            h = cu.seg % p.c.n_kv;
            row0 = cu.seg / p.c.n_kv * kRows;
            rows = min(kRows, cu.a.n * p.group - row0);
            live = (rows + 7) / 8;
            first_row = cu.a.len - cu.a.n + token_of(p, row0);
            // the last token that the last row does not see (rows further down see later ones)
            before_window = p.window > 0 ? static_cast<int>(max(static_cast<int64_t>(-1), static_cast<int64_t>(cu.a.len) - cu.a.n + token_of(p, row0 + rows - 1) - p.window)) : -1;
            factor = p.scale * 1.44269504088896340736f * (kE4M3 && p.c.k_scale ? __ldg(p.c.k_scale + h) : 1.0f);
            active = rg < live;
            constexpr int kQC = kD / 8;
#pragma unroll 4
            for (int i = gt; i < 8 * kNR * kQC; i += kGroup) {
                const int r = base_of(i / kQC / 8) + i / kQC % 8, c = i % kQC, at = token_of(p, row0 + r);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows) v = __ldg(reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(cu.a.beg + at) * p.ld_q + (h * p.group + (row0 + r) - at * p.group) * kD + c * 8));
                if (c == 0) row_pos[r] = cu.a.len - cu.a.n + at;
                if constexpr (!kE4M3) {
                    *reinterpret_cast<uint4*>(qs + piece<kQB>(r, c)) = v;
                } else {
                    // FP16 with the row's largest in [2^14, 2^15), columns in the order in which the keys' bytes come:
                    // column 16 x + k of a block of 64 is element 16 t + 4 x + e, t and e as the fragments have them
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t big = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) big = max(big, max((w[x] << 16) & 0x7FFF0000u, w[x] & 0x7FFF0000u));
#pragma unroll
                    for (int x = kQC / 2; x > 0; x >>= 1) big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, x));
                    const int shift = big ? min(100, 14 + 127 - static_cast<int>(big >> 23)) : 0;  // -114 (infinities) at the least
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
            sync();  // (of a group without rows, too)
            if constexpr (kQReg) {
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                    for (int ks = 0; ks < kKS; ks += 2) {
                        uint32_t b[4];
                        ldsm4((q_lane ^ (ks * 32)) + base_of(nr) * kQB, b);
                        qf[nr][ks][0] = b[0];
                        qf[nr][ks][1] = b[1];
                        qf[nr][ks + 1][0] = b[2];
                        qf[nr][ks + 1][1] = b[3];
                    }
            }
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr) {
                m[nr][0] = m[nr][1] = -INFINITY;
                l[nr][0] = l[nr][1] = 0.0f;
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[mt][nr][x] = 0.0f;
            }
            opens = false;
        }

        wait(full + stage, phase);
        const uint32_t k_at = k_lane + stage_off, v_at = v_lane + stage_off;
        const int pos0 = cu.a.start + cu.tile * kTile;
        const bool edge = pos0 > first_row - (kTile - 1) || pos0 <= before_window;  // some row does not see some token
        // whether the row at a position sees the unit's token x
        auto sees = [&](int at, int x) { return x <= at - pos0 && (p.window <= 0 || static_cast<int64_t>(x) + p.window > at - pos0); };
        if (active) {
            // ---- S^T = K Q^T of this warp's tokens (16 from 16 gw on, and 64 further), each in two chains of sums
            float sc[kNR][kMQ][4], sc2[kNR][kMQ][4];
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                for (int y = 0; y < kMQ; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[nr][y][x] = sc2[nr][y][x] = 0.0f;
            // q's fragments of steps ks and ks + 1
            auto q_frag = [&](int nr, int ks, uint32_t (&b)[4]) {
                if constexpr (kQReg) {
                    b[0] = qf[nr][ks][0];
                    b[1] = qf[nr][ks][1];
                    b[2] = qf[nr][ks + 1][0];
                    b[3] = qf[nr][ks + 1][1];
                } else {
                    ldsm4((q_lane ^ (ks * 32)) + base_of(nr) * kQB, b);
                }
            };
            if constexpr (!kE4M3) {
#pragma unroll
                for (int ks = 0; ks < kKS; ks += 2) {
                    uint32_t a[kMQ][4], a2[kMQ][4];
#pragma unroll
                    for (int y = 0; y < kMQ; ++y) {
                        ldsm4((k_at ^ (ks * 32)) + y * 64 * kRB, a[y]);
                        ldsm4((k_at ^ (ks * 32 + 32)) + y * 64 * kRB, a2[y]);
                    }
#pragma unroll
                    for (int nr = 0; nr < kNR; ++nr) {
                        uint32_t b[4];
                        q_frag(nr, ks, b);
#pragma unroll
                        for (int y = 0; y < kMQ; ++y) {
                            mma<false>(sc[nr][y], a[y][0], a[y][1], a[y][2], a[y][3], b[0], b[1]);
                            mma<false>(sc2[nr][y], a2[y][0], a2[y][1], a2[y][2], a2[y][3], b[2], b[3]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int blk = 0; blk < kD / 64; ++blk)
#pragma unroll
                    for (int y = 0; y < kMQ; ++y) {
                        uint32_t w[2][4];
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(w[z][0]), "=r"(w[z][1]), "=r"(w[z][2]), "=r"(w[z][3])
                                         : "r"((k_at ^ (blk * 64)) + (y * 64 + z * 8) * kRB)
                                         : "memory");
#pragma unroll
                        for (int x = 0; x < 4; x += 2) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int z = 0; z < 2; ++z) e4m3x4_to_f16(w[z][x + u], a[u][z], a[u][2 + z]);
#pragma unroll
                            for (int nr = 0; nr < kNR; ++nr) {
                                uint32_t b[4];
                                q_frag(nr, 4 * blk + x, b);
                                mma<true>(sc[nr][y], a[0][0], a[0][1], a[0][2], a[0][3], b[0], b[1]);
                                mma<true>(sc2[nr][y], a[1][0], a[1][1], a[1][2], a[1][3], b[2], b[3]);
                            }
                        }
                    }
            }

            // ---- scores in powers of two, masks, maxima
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr) {
                const float2 by = kE4M3 ? *reinterpret_cast<const float2*>(qscale + base_of(nr) + 2 * t4) : make_float2(1.0f, 1.0f);
#pragma unroll
                for (int y = 0; y < kMQ; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[nr][y][x] = (sc[nr][y][x] + sc2[nr][y][x]) * (kE4M3 ? factor * (x & 1 ? by.y : by.x) : factor);
                if (edge) {
                    const int2 at = *reinterpret_cast<const int2*>(row_pos + base_of(nr) + 2 * t4);
#pragma unroll
                    for (int y = 0; y < kMQ; ++y)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (!sees(x & 1 ? at.y : at.x, y * 64 + gw * 16 + g + x / 2 * 8)) sc[nr][y][x] = -INFINITY;
                }
                float u = fmaxf(sc[nr][0][0], sc[nr][0][2]), v = fmaxf(sc[nr][0][1], sc[nr][0][3]);
#pragma unroll
                for (int y = 1; y < kMQ; ++y) {
                    u = fmaxf(u, fmaxf(sc[nr][y][0], sc[nr][y][2]));
                    v = fmaxf(v, fmaxf(sc[nr][y][1], sc[nr][y][3]));
                }
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    u = fmaxf(u, __shfl_xor_sync(0xFFFFFFFFu, u, x));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, x));
                }
                if (g == 0) {
                    wmax[(base_of(nr) + 2 * t4) * kWarps + gw] = u;
                    wmax[(base_of(nr) + 2 * t4 + 1) * kWarps + gw] = v;
                }
            }
            sync();  // the maxima are there, and every warp is done with the weights of the unit before

            // ---- weights
            bool moved = false;
            float alpha[kNR][2];
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr) {
                float by[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float4 w = *reinterpret_cast<const float4*>(wmax + (base_of(nr) + 2 * t4 + x) * kWarps);
                    const float to = fmaxf(fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)) - kLift, m[nr][x]);
                    moved |= to > m[nr][x];
                    by[x] = to == -INFINITY ? 0.0f : to;  // a row that has seen nothing yet
                    alpha[nr][x] = exp2_fast(m[nr][x] - by[x]);
                    m[nr][x] = to;
                    l[nr][x] *= alpha[nr][x];
                }
#pragma unroll
                for (int y = 0; y < kMQ; ++y) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[nr][y][x] = exp2_fast(sc[nr][y][x] - by[x & 1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) l[nr][x] += sc[nr][y][x] + sc[nr][y][x + 2];
                    // rows of kTile tokens: these 16 are two pieces
                    const uint32_t at = (p_mine ^ (y * 128)) + base_of(nr) * kPB;
                    if constexpr (kE4M3) {
                        uint32_t high[2], low[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            high[x] = pack_f16x2(sc[nr][y][2 * x], sc[nr][y][2 * x + 1]);
                            low[x] = pack_f16x2(sc[nr][y][2 * x] - f16_to_f32(high[x] & 0xFFFFu), sc[nr][y][2 * x + 1] - f16_to_f32(high[x] >> 16));
                        }
                        stsm2t(at, high[0], high[1]);
                        stsm2t(at + kRows * kPB, low[0], low[1]);
                    } else {
                        // The high parts are cut, the low ones what is left, never 0: both are positive, so an infinite value
                        // times them is one infinity (rounded high parts leave some low ones negative: infinities of both
                        // signs, a NaN). 8 bits and 8 more of less than 2^-7: within 2^-16.
                        uint32_t high[2], low[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t w0 = __float_as_uint(sc[nr][y][2 * x]) | 1u, w1 = __float_as_uint(sc[nr][y][2 * x + 1]) | 1u;
                            high[x] = __byte_perm(w0, w1, 0x7632);
                            low[x] = pack_bf16x2(__uint_as_float(w0) - __uint_as_float(w0 & 0xFFFF0000u), __uint_as_float(w1) - __uint_as_float(w1 & 0xFFFF0000u));
                        }
                        stsm2t(at, high[0], high[1]);
                        stsm2t(at + kRows * kPB, low[0], low[1]);
                    }
                }
            }
            if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[mt][nr][x] *= alpha[nr][x & 1];
            }
        }

        // an accumulator's column of v: x / 2 is the lower or upper eight of a tile (E4M3: the even or odd columns)
        auto column = [&](int mt, int x) {
            return gw * (kD / 4) + mt * 16 + (kE4M3 ? 2 * g + x / 2 : g + x / 2 * 8);
        };
        if (edge && cu.a.n > 1) {
            // A token that only some rows see may hold infinities or NaN, and a weight of 0 times them is no 0: such
            // elements are added by the rows that see them, one by one, and taken out of the unit.
            uint8_t* const vs = ring + stage_off + kTile * kRB;
            bool odd = false;
            for (int i = tid; i < kTile * kRB / 16; i += kCompute) {
                const uint4 w = *reinterpret_cast<const uint4*>(vs + i * 16);
                odd |= (odd_mask<kE4M3>(w.x) | odd_mask<kE4M3>(w.y) | odd_mask<kE4M3>(w.z) | odd_mask<kE4M3>(w.w)) != 0;
            }
            if (any_of(odd)) {  // (the weights are there)
#pragma unroll 1
                for (int tok = 0; tok < (active ? kTile : 0); ++tok) {
#pragma unroll
                    for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int r = base_of(nr) + 2 * t4 + y;
                            if (!sees(row_pos[r], tok)) continue;
                            const uint8_t* pp = ps + piece<kPB>(r, tok / 8) + tok % 8 * 2;
                            float wt;
                            if constexpr (kE4M3) wt = f16_to_f32(*reinterpret_cast<const uint16_t*>(pp)) + f16_to_f32(*reinterpret_cast<const uint16_t*>(pp + kRows * kPB));
                            else wt = bf16_to_f32(*reinterpret_cast<const uint16_t*>(pp)) + bf16_to_f32(*reinterpret_cast<const uint16_t*>(pp + kRows * kPB));
#pragma unroll
                            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                                for (int x = y; x < 4; x += 2) {
                                    const int d = column(mt, x);
                                    if constexpr (kE4M3) {
                                        const uint32_t b = vs[piece<kRB>(tok, d / 16) + d % 16];
                                        if ((b & 0x7Fu) == 0x7Fu) o[mt][nr][x] += wt * NAN;
                                    } else {
                                        const uint32_t b = *reinterpret_cast<const uint16_t*>(vs + piece<kRB>(tok, d / 8) + d % 8 * 2);
                                        if ((b & 0x7F80u) == 0x7F80u) o[mt][nr][x] += wt * bf16_to_f32(b);
                                    }
                                }
                        }
                }
                sync_all();
                for (int i = tid; i < kTile * kRB / 4; i += kCompute) {
                    uint32_t* const w = reinterpret_cast<uint32_t*>(vs) + i;
                    const uint32_t odds = odd_mask<kE4M3>(*w);
                    // the elements of the marked top bits, as whole bytes or halves
                    if (odds) *w &= ~(kE4M3 ? (odds >> 7) * 0xFFu : (odds >> 15) * 0xFFFFu);
                }
                sync_all();
            }
        } else if (active) {
            sync();  // the weights are there
        }

        if (active) {
            // ---- O^T += V^T P^T, this warp's quarter of the columns, 32 tokens at a time
#pragma unroll 1
            for (int kk = 0; kk < kTile / 16; kk += 2) {
                uint32_t b[S::kParts][kNR][4];
#pragma unroll
                for (int nr = 0; nr < kNR; ++nr) {
                    const uint32_t at = (p_lane ^ (kk * 32)) + base_of(nr) * kPB;
#pragma unroll
                    for (int z = 0; z < S::kParts; ++z) ldsm4(at + z * kRows * kPB, b[z][nr]);
                }
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                    uint32_t a[2][4];  // of both steps
                    if constexpr (!kE4M3) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) ldsm4t((v_at ^ (mt * 32)) + (kk + x) * 16 * kRB, a[x]);
                    } else {
                        // a piece is 16 columns: the transposed load gives the bytes of two columns of two tokens
                        uint32_t w[4];
                        ldsm4t((v_at ^ (mt * 16)) + kk * 16 * kRB, w);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            e4m3x4_to_f16(__byte_perm(w[x], 0, 0x3120), a[x / 2][x % 2 * 2], a[x / 2][x % 2 * 2 + 1]);
                    }
#pragma unroll
                    for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int z = 0; z < S::kParts; ++z) mma<kE4M3>(o[mt][nr], a[x][0], a[x][1], a[x][2], a[x][3], b[z][nr][2 * x], b[z][nr][2 * x + 1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty + stage);
        stage_off += S::kStage;
        if (++stage == kStages) {
            stage = 0;
            stage_off = 0;
            phase ^= 1;
        }

        // ---- the end of a (request, head): finished here, or a part of it
        const bool last = j == count - 1, closes = cu.tile == cu.a.tiles - 1;
        if ((last || closes) && active) {
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = l[nr][x];
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, y);
                    if (g == 0) wsum[(base_of(nr) + 2 * t4 + x) * kWarps + gw] = v;
                }
            sync();
            const bool whole = closes && cu.tile <= j;  // its first unit is in this run as well
            // a part: slot 0 where the (request, head) holds the run's first unit, else 1
            const int64_t part = blockIdx.x * 2 + (cu.tile >= j ? 0 : 1);
#pragma unroll
            for (int nr = 0; nr < kNR; ++nr)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = base_of(nr) + 2 * t4 + x;
                    const float4 w = *reinterpret_cast<const float4*>(wsum + r * kWarps);
                    const float sum = (w.x + w.y) + (w.z + w.w);
                    if (r >= rows) continue;
                    if (whole) {
                        const int at = token_of(p, row0 + r), head = h * p.group + (row0 + r) - at * p.group;
                        const int64_t t = cu.a.beg + at;
                        float by = sum == 0.0f ? 0.0f : 1.0f / sum;
                        if (kE4M3 && p.c.v_scale) by *= __ldg(p.c.v_scale + h);
                        uint16_t* const to = p.out + t * p.ld_out + head * kD;
                        if (p.lse && gw == 0 && g == 0)
                            p.lse[t * p.n_q + head] = sum == 0.0f ? -INFINITY : (m[nr][x] + log2f(sum)) * 0.69314718055994530942f;
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt) {
                            const uint32_t b = pack_bf16x2(o[mt][nr][x] * by, o[mt][nr][x + 2] * by);
                            if constexpr (kE4M3) {
                                *reinterpret_cast<uint32_t*>(to + column(mt, 0)) = b;
                            } else {
                                to[column(mt, 0)] = static_cast<uint16_t>(b);
                                to[column(mt, 2)] = static_cast<uint16_t>(b >> 16);
                            }
                        }
                    } else {
                        float* const to = p.part + (part * kRows + r) * kD;
                        if (gw == 0 && g == 0) *reinterpret_cast<float2*>(p.part_ml + (part * kRows + r) * 2) = make_float2(m[nr][x], sum);
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt) {
                            if constexpr (kE4M3) {
                                *reinterpret_cast<float2*>(to + column(mt, 0)) = make_float2(o[mt][nr][x], o[mt][nr][x + 2]);
                            } else {
                                to[column(mt, 0)] = o[mt][nr][x];
                                to[column(mt, 2)] = o[mt][nr][x + 2];
                            }
                        }
                    }
                }
        }
        opens = closes;
        if (!last) cu.next(p);
    }
}

// ---- the join: a row's parts, in the order of the runs. Few rows: 64 columns a CTA, the parts over its eight warps, each with
// all of its loads in flight; many rows: a warp a row.
constexpr int kJoinWarps = 8;

template <int kD, bool kE4M3, int kRG, int kNR, bool kFew>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attention_join(const __grid_constant__ AttentionArgs p)
{
    using S = Shape<kD, kE4M3, kRG, kNR>;
    constexpr int kRows = S::kRows, kCols = kFew ? 64 : kD, kV = kCols / 32;  // columns a CTA, a lane: col0 + lane * kV ..
    constexpr int kFlight = kFew ? 20 : 8;                                    // parts whose loads are in flight
    __shared__ float sm_o[kFew ? kJoinWarps : 1][kCols], sm_ml[kJoinWarps][2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = kFew ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) * kJoinWarps + warp, col0 = kFew ? blockIdx.y * 64 : 0;
    // (the tables were there before the main launch began)
    const int t = row / p.n_q, head = row - t * p.n_q, s = t < p.T ? find_request(p.r.seg_offsets, p.r.S, t) : -1;
    Span a{};
    bool bad = true;
    if (s >= 0 && s < p.r.S) a = span_of<S>(p, s, bad);
    const bool mine = a.segs != 0 && t >= a.beg && t < a.beg + a.n;
    const int h = head / p.group, in_seg = (t - a.beg) * p.group + head % p.group, r = in_seg % kRows;
    const int seg = in_seg / kRows * p.c.n_kv + h;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (!mine) return;  // the same in all warps of a row
    const int64_t u0 = p.prefix[s] + seg * a.each() + kExtra * a.w, last = u0 + static_cast<int64_t>(a.tiles) * a.w - 1;  // of its units
    const Cut cut{p.prefix[p.r.S + 1], p.prefix[p.r.S + 2]};
    const int c0 = cut.run(u0 + a.w - 1), n = cut.run(last) - c0 + 1;
    if (n == 1) return;  // finished by its run
    const bool from_start = cut.first(c0) >= u0 - kExtra * a.w;
    auto slot_of = [&](int x) { return static_cast<int64_t>(c0 + x) * 2 + (x == 0 && !from_start ? 1 : 0); };

    float mx = -INFINITY, sum = 0.0f, o[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) o[i] = 0.0f;
    const int per = (n + kJoinWarps - 1) / kJoinWarps;
    const int b = kFew ? min(n, warp * per) : 0, e = kFew ? min(n, b + per) : n;
    for (int i0 = b; i0 < e; i0 += 32) {
        const int i = i0 + lane;
        float2 ml = make_float2(-INFINITY, 0.0f);
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
        for (int x0 = 0; x0 < in; x0 += kFlight) {
            float v[kFlight][kV];
#pragma unroll
            for (int x = 0; x < kFlight; ++x) {
                const float* from = p.part + (slot_of(i0 + x0 + x) * kRows + r) * kD + col0 + lane * kV;
#pragma unroll
                for (int y = 0; y < kV; ++y) v[x][y] = 0.0f;
                if (x0 + x < in) {
                    if constexpr (kV == 2) {
                        *reinterpret_cast<float2*>(v[x]) = __ldcg(reinterpret_cast<const float2*>(from));
                    } else {
#pragma unroll
                        for (int y = 0; y < kV; y += 4) *reinterpret_cast<float4*>(v[x] + y) = __ldcg(reinterpret_cast<const float4*>(from + y));
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < kFlight; ++x) {
                const float wx = __shfl_sync(0xFFFFFFFFu, w, (x0 + x) & 31);  // (past the last part: times zeros)
#pragma unroll
                for (int y = 0; y < kV; ++y) o[y] += wx * v[x][y];
            }
        }
    }
    if constexpr (kFew) {
#pragma unroll
        for (int x = 0; x < kV; ++x) sm_o[warp][lane * kV + x] = o[x];
        if (lane == 0) {
            sm_ml[warp][0] = mx;
            sm_ml[warp][1] = sum;
        }
        __syncthreads();
        if (warp) return;
        mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, sm_ml[w][0]);
        const float by = mx == -INFINITY ? 0.0f : mx;
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
    }
    float by = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (kE4M3 && p.c.v_scale) by *= __ldg(p.c.v_scale + h);
    uint16_t* const to = p.out + static_cast<int64_t>(t) * p.ld_out + head * kD + col0 + lane * kV;
#pragma unroll
    for (int x = 0; x < kV; x += 2) *reinterpret_cast<uint32_t*>(to + x) = pack_bf16x2(o[x] * by, o[x + 1] * by);
    if (p.lse && lane == 0 && col0 == 0) p.lse[row] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994530942f;
}

template <int kD, bool kE4M3, int kRG, int kNR>
cudaError_t launch(const AttentionArgs& a, int sms, cudaStream_t stream)
{
    using S = Shape<kD, kE4M3, kRG, kNR>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(smem_set, reinterpret_cast<const void*>(k_paged_attention<kD, kE4M3, kRG, kNR>), S::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = sms * S::kCtas;
    e = launch_pdl(k_paged_attention<kD, kE4M3, kRG, kNR>, dim3(ctas), dim3(S::kThreads), S::kSmem, stream, a);
    if (e != cudaSuccess) return e;
    const int64_t n = static_cast<int64_t>(a.T) * a.n_q;
    if (n <= 512)
        return launch_pdl(k_attention_join<kD, kE4M3, kRG, kNR, true>, dim3(static_cast<unsigned>(n), kD / 64), dim3(kJoinWarps * 32), 0, stream, a);
    return launch_pdl(k_attention_join<kD, kE4M3, kRG, kNR, false>, dim3(static_cast<unsigned>((n + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32),
                      0, stream, a);
}

template <int kD, bool kE4M3>
cudaError_t launch_head_size(const AttentionArgs& a, int sms, cudaStream_t stream)
{
    switch (row_eights(a.group, a.max_new)) {
    case 1: return launch<kD, kE4M3, 1, 1>(a, sms, stream);
    case 2: return launch<kD, kE4M3, 2, 1>(a, sms, stream);
    // (One group reads K and V once for the three eights, three hide one another's waits: 100 requests over to 2,000, 32
    // heads on 4 of 128, 59.5 and 66.0 us; 60, 16 on 2 of 256, 45.2 and 44.2; 200 over to 4,096, 14 on 2 of 64,
    // 58.8 and 55.4.)
    case 3: return launch<kD, kE4M3, kD == 128 && !kE4M3 ? 1 : 3, kD == 128 && !kE4M3 ? 3 : 1>(a, sms, stream);
    case 4: return launch<kD, kE4M3, 2, 2>(a, sms, stream);
    default: return launch<kD, kE4M3, 4, 2>(a, sms, stream);
    }
}

}  // namespace attention
}  // namespace moe
