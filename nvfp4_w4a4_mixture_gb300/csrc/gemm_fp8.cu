// gemm_fp8.cu -- FP8 matrix product with a scale for each block of 128:
//   out[t][n] = sum_b sa[t][b] sb[n / 128][b] sum_{k in b} a[t][k] b[n][k]
// tcgen05.mma kind::f8f6f4 sums a block's 128 products in tensor memory (four MMAs of K = 32); the scales are FP32 and
// differ from block to block, so a block's sum leaves tensor memory and is scaled and added in registers, while the next
// block's MMAs run into another buffer. Two kernels, by the number of tiles:
//   k_gemm_fp8       128 tokens x 256 outputs a tile: a lane is a token, its scale one number a block. CTAs stay and
//                    walk the tiles; two groups of four warps take 128 outputs each, and their rows go out by bulk copies.
//   k_gemm_fp8_few   128 outputs x 16, 32 or 64 tokens a tile (weights on the MMA's M side): few tokens then read each
//                    weight once without padding; a cluster of CTAs shares a tile's blocks along K and adds the parts
//                    through distributed shared memory, in the order of their ranks.
// TMA fills the ragged ends of K, T and N with zeros.
// Measured: 16,384 x 4,096 x 2,048 104 us, 2.6 PFLOP/s (70 % of twice the rate of bf16 matrix products), in bursts of some 20
// calls; in hundreds on end, where the power limit holds the clock at 1.7 GHz instead of 2.07, 115 to 117 us (2.4, 69 % of
// twice what bf16 sustains there). The variants that follow are bursts, too. Without the sums in registers it took 95 us, with
// the loads from tensor memory alone 93: the rest is the MMAs (512 cycles a block at their nominal rate, some 850 here) and
// the sums' turn between them. Two values an instruction (fma.rn.f32x2: 123 us) and
// registers moved to the summing warps for two loads of 32 columns in flight (107) were slower. Pairs of multiprocessors on
// one tile (cta_group::2, 256 x 256, half of A and of B each) took 104 to 106, too, with eight or sixteen summing warps and
// two or four buffers: without the loads 98 to 101, without the sums 86, with neither 78, so the sums are what is left, while
// fewer tokens took longer (256: 9.7 to 10.4 us, 9.1 here). 4 x 5,120 x 2,048 5.1 us
// (its weights in 1.6).
#include "attention.cuh"
#include "ptx_cluster.cuh"

namespace moe {

namespace {

constexpr int kSmemMax = 227 * 1024;

// D(tmem, f32) (+)= A(smem, e4m3) * B(smem, e4m3)^T, K = 32
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor, kind::f8f6f4: D f32 [4,6) = 1, A and B E4M3 (format 0), both K-major, N >> 3 at [17,23), M >> 4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A test makes the first wait run out: then it is for a barrier that nobody arrives at. With kOneWarp one summing warp of
// k_gemm_fp8_few gives up instead, and the others go on.
constexpr int kOneWarp = 2;
__device__ __forceinline__ int test_hook(const GemmFp8Args& p) { return *reinterpret_cast<const volatile int*>(&p.hooks->test_ready_extra); }

// ------------------------------------------------------------------------------------------------
// many tokens
// ------------------------------------------------------------------------------------------------
constexpr int kBigM = 128, kBigN = 256, kBigStages = 4, kBigThreads = 320, kEpiWarps = 8, kFirstEpi = 2;
constexpr int kBigA = kBigM * 128, kBigStage = kBigA + kBigN * 128;
constexpr int kOutBox = 32 * 128;  // a warp's piece of the output: 32 rows of 128 bytes

struct BigTail {
    uint64_t full[kBigStages], empty[kBigStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
};
constexpr size_t kBigSmem = 1024 + static_cast<size_t>(kBigStages) * kBigStage + kEpiWarps * kOutBox + sizeof(BigTail);
static_assert(kBigSmem <= kSmemMax, "shared memory");

template <bool kF32>
__global__ void __launch_bounds__(kBigThreads, 1)
    k_gemm_fp8(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_out,
               const __grid_constant__ GemmFp8Args p, int n_tiles_n, int n_tiles)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* obuf = smem + kBigStages * kBigStage;  // [epilogue warp]
    BigTail& st = *reinterpret_cast<BigTail*>(obuf + kEpiWarps * kOutBox);
    const int tid = threadIdx.x, warp = __reduce_max_sync(0xFFFFFFFFu, tid / 32), lane = tid % 32;
    const int nk = (p.K + 127) / 128;
    if (tid == 0) {
        for (int s = 0; s < kBigStages; ++s) {
            ptx::mbar_init(&st.full[s], 1);
            ptx::mbar_init(&st.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&st.acc_full[b], 1);
            ptx::mbar_init(&st.acc_empty[b], kEpiWarps);
        }
        ptx::mbar_init(&st.drain, 1);
        st.abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map_a);
        ptx::prefetch_tmap(&map_b);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&st.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::griddep_launch_dependents();  // not before the tensor memory is allocated: the next launch's CTAs take some, too
    ptx::tc_fence_after();
    const uint32_t tmem = st.tmem;
    auto fail = [&]() {
        if (atomicExch(&st.abort, 1) == 0) record_status(p.status, kDevTimeoutGemmFp8);
    };
    auto all = [&](bool got) { return __all_sync(0xFFFFFFFFu, got) != 0; };

    if (warp == 0) {
        const bool leader = ptx::elect_one();
        int s = 0;
        uint32_t ph = 0, fills = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < n_tiles; tile += gridDim.x) {
            const int tm = tile / n_tiles_n, tn = tile % n_tiles_n;
            for (int kb = 0; kb < nk; ++kb) {
                ok = all(ptx::mbar_wait_near(&st.empty[s], ph ^ 1));
                if (!ok) break;
                uint8_t* b = smem + s * kBigStage;
                if (leader) {
                    ptx::mbar_arrive_expect_tx(&st.full[s], kBigStage);
                    ptx::tma_load_3d(b, &map_a, &st.full[s], kb * 128, tm * kBigM, 0);
                    ptx::tma_load_3d(b + kBigA, &map_b, &st.full[s], kb * 128, tn * kBigN, 0);
                }
                ++fills;
                if (++s == kBigStages) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) fail();
        if (leader && !ptx::ring_drain(st.full, kBigStages, fills)) fail();
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_e4m3(kBigM, kBigN);
        const uint64_t da = ptx::sdesc_sw128(ptx::smem_u32(smem)), db = ptx::sdesc_sw128(ptx::smem_u32(smem + kBigA));
        const bool leader = ptx::elect_one();
        int s = 0;
        uint32_t ph = 0, it = 0;
        bool ok = test_hook(p) <= 0 || all(ptx::mbar_wait_us(&st.drain, 0, p.hooks->test_wait_us));
        for (int tile = blockIdx.x; ok && tile < n_tiles; tile += gridDim.x)
            for (int kb = 0; ok && kb < nk; ++kb, ++it) {
                const uint32_t buf = it & 1;
                ok = all(ptx::mbar_wait_near(&st.full[s], ph)) && all(ptx::mbar_wait_near(&st.acc_empty[buf], ((it >> 1) & 1) ^ 1));
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t so = static_cast<uint64_t>(s) * (kBigStage >> 4);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_e4m3(tmem + buf * kBigN, da + so + kk * 2, db + so + kk * 2, idesc, kk > 0);
                    ptx::tc_commit(&st.empty[s]);
                    ptx::tc_commit(&st.acc_full[buf]);
                }
                if (++s == kBigStages) { s = 0; ph ^= 1; }
            }
        if (!ok) {
            fail();
            if (leader) ptx::tc_commit(&st.drain);  // what was issued ends before the tensor memory goes
            ptx::mbar_wait(&st.drain, 0);
        }
    } else {
        const int ew = warp - kFirstEpi, grp = ew / 4, q = warp & 3;
        const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16) + grp * 128;
        uint32_t it = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < n_tiles; tile += gridDim.x) {
            const int tm = tile / n_tiles_n, tn = tile % n_tiles_n;
            const int row = tm * kBigM + q * 32 + lane, col = tn * kBigN + grp * 128;
            const float* sa = p.a_scale + static_cast<int64_t>(min(row, p.T - 1)) * nk;
            const float* sb = p.b_scale + static_cast<int64_t>(min(col, p.N - 1) / 128) * nk;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
            // the scales come a block ahead
            float fa = __ldg(sa), fb = __ldg(sb);
            for (int kb = 0; kb < nk; ++kb, ++it) {
                const uint32_t buf = it & 1;
                const float f = fa * fb;
                if (kb + 1 < nk) {
                    fa = __ldg(sa + kb + 1);
                    fb = __ldg(sb + kb + 1);
                }
                ok = all(ptx::mbar_wait_near(&st.acc_full[buf], (it >> 1) & 1));
                if (!ok) break;
                ptx::tc_fence_after();
                // 16 columns at a time, the next ones' load in flight while some are scaled and added
                uint32_t v[2][16];
                ptx::tmem_ld16(tq + buf * kBigN, v[0]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[c & 1][i]));  // no use of them is moved before the wait
                    if (c < 7) {
                        ptx::tmem_ld16(tq + buf * kBigN + (c + 1) * 16, v[(c + 1) & 1]);
                    } else {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&st.acc_empty[buf]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c * 16 + i] = fmaf(__uint_as_float(v[c & 1][i]), f, acc[c * 16 + i]);
                }
            }
            if (!ok) break;
            // the rows go out in pieces of 128 bytes, by way of shared memory: one copy of 32 of them, which clips at T and N
            constexpr int kCols = kF32 ? 32 : 64;  // of a piece
            const uint32_t ob = ptx::smem_u32(obuf + ew * kOutBox);
#pragma unroll
            for (int h = 0; h < 128 / kCols; ++h) {
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the copy before has read the buffer
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 w;
                    if constexpr (kF32) {
                        const float* a = acc + h * 32 + 4 * i;
                        w = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3]));
                    } else {
                        const float* a = acc + h * 64 + 8 * i;
                        w = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
                    }
                    ptx::shared_store16(ob + lane * 128 + ((i ^ (lane & 7)) << 4), w);  // as the 128-byte swizzle has it
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && col + h * kCols < p.N && tm * kBigM + q * 32 < p.T) {
                    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                                 ::"l"(reinterpret_cast<uint64_t>(&map_out)), "r"(col + h * kCols), "r"(tm * kBigM + q * 32), "r"(ob)
                                 : "memory");
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!ok) fail();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------------------
// few tokens
// ------------------------------------------------------------------------------------------------
constexpr int kFewM = 128, kFewThreads = 192, kFewBufs = 4, kChunk = 8;  // kChunk: blocks whose token scales are staged together

template <int kN>
struct Few {
    static constexpr int kA = kFewM * 128, kStage = kA + kN * 128;
    static constexpr int kPart = kN * kFewM * 4;      // the parts of this CTA's share of the tokens
    static constexpr int kScales = 2 * kChunk * kN * 4;
    static constexpr int kStages = kN == 64 ? 3 : kN == 32 ? 4 : 5;  // two CTAs an SM
    static constexpr uint32_t kCols = kFewBufs * kN;
};
template <int kStages>
struct FewTail {
    uint64_t full[kStages], empty[kStages], acc_full[kFewBufs], acc_empty[kFewBufs], drain;
    uint32_t tmem;
    int abort;
};
template <int kN>
constexpr size_t few_smem()
{
    using S = Few<kN>;
    constexpr size_t n = 1024 + static_cast<size_t>(S::kStages) * S::kStage + S::kPart + S::kScales + sizeof(FewTail<S::kStages>);
    static_assert(n <= kSmemMax, "shared memory");
    return n;
}

template <int kN, bool kF32>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_gemm_fp8_few(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const __grid_constant__ GemmFp8Args p,
                   int n_tiles_t)
{
    using S = Few<kN>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* const part = reinterpret_cast<float*>(smem + kStages * S::kStage);  // [rank][token of the share][128]
    float* const scales = part + S::kPart / 4;                                 // [2][kChunk][kN]
    FewTail<kStages>& st = *reinterpret_cast<FewTail<kStages>*>(scales + S::kScales / 4);
    const int tid = threadIdx.x, warp = __reduce_max_sync(0xFFFFFFFFu, tid / 32), lane = tid % 32;
    const int cs = static_cast<int>(ptx::cluster_size()), rank = static_cast<int>(ptx::cluster_rank());
    const int tile = blockIdx.x / cs, tt = tile % n_tiles_t, tn = tile / n_tiles_t;
    const int nk = (p.K + 127) / 128, k0 = static_cast<int>(static_cast<int64_t>(nk) * rank / cs), k1 = static_cast<int>(static_cast<int64_t>(nk) * (rank + 1) / cs);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&st.full[s], 1);
            ptx::mbar_init(&st.empty[s], 1);
        }
        for (int b = 0; b < kFewBufs; ++b) {
            ptx::mbar_init(&st.acc_full[b], 1);
            ptx::mbar_init(&st.acc_empty[b], 4);
        }
        ptx::mbar_init(&st.drain, 1);
        st.abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map_a);
        ptx::prefetch_tmap(&map_b);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&st.tmem, S::kCols);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::griddep_launch_dependents();  // not before the tensor memory is allocated: the next launch's CTAs take some, too
    if (cs > 1) ptx::cluster_arrive_all();  // waited for before the first store to another CTA
    ptx::tc_fence_after();
    const uint32_t tmem = st.tmem;
    bool failed = false;
    auto fail = [&]() {
        failed = true;
        if (atomicExch(&st.abort, 1) == 0) record_status(p.status, kDevTimeoutGemmFp8);
    };
    auto all = [&](bool got) { return __all_sync(0xFFFFFFFFu, got) != 0; };
    bool good = true;
    float acc[kN];

    if (warp == 0) {
        const bool leader = ptx::elect_one();
        int s = 0;
        uint32_t ph = 0, fills = 0;
        bool ok = true;
        for (int kb = k0; kb < k1; ++kb) {
            ok = all(ptx::mbar_wait_near(&st.empty[s], ph ^ 1));
            if (!ok) break;
            uint8_t* b = smem + s * S::kStage;
            if (leader) {
                ptx::mbar_arrive_expect_tx(&st.full[s], S::kStage);
                ptx::tma_load_3d(b, &map_b, &st.full[s], kb * 128, tn * kFewM, 0);
                ptx::tma_load_3d(b + S::kA, &map_a, &st.full[s], kb * 128, tt * kN, 0);
            }
            ++fills;
            if (++s == kStages) { s = 0; ph ^= 1; }
        }
        if (!ok) fail();
        if (leader && !ptx::ring_drain(st.full, kStages, fills)) fail();
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_e4m3(kFewM, kN);
        const uint64_t dw = ptx::sdesc_sw128(ptx::smem_u32(smem)), dx = ptx::sdesc_sw128(ptx::smem_u32(smem + S::kA));
        const bool leader = ptx::elect_one();
        int s = 0;
        uint32_t ph = 0;
        const int hook = test_hook(p);
        bool ok = hook <= 0 || hook == kOneWarp || all(ptx::mbar_wait_us(&st.drain, 0, p.hooks->test_wait_us));
        for (int kb = k0; ok && kb < k1; ++kb) {
            const uint32_t it = kb - k0, buf = it % kFewBufs;
            ok = all(ptx::mbar_wait_near(&st.full[s], ph)) && all(ptx::mbar_wait_near(&st.acc_empty[buf], ((it / kFewBufs) & 1) ^ 1));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint64_t so = static_cast<uint64_t>(s) * (S::kStage >> 4);
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) mma_e4m3(tmem + buf * kN, dw + so + kk * 2, dx + so + kk * 2, idesc, kk > 0);
                ptx::tc_commit(&st.empty[s]);
                ptx::tc_commit(&st.acc_full[buf]);
            }
            if (++s == kStages) { s = 0; ph ^= 1; }
        }
        if (!ok) {
            fail();
            if (leader) ptx::tc_commit(&st.drain);  // what was issued ends before the tensor memory goes
            ptx::mbar_wait(&st.drain, 0);
        }
    } else {
        const int q = warp & 3, et = tid - 64;
        const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
        for (int i = 0; i < kN; ++i) acc[i] = 0.0f;
        const float* sb = p.b_scale + static_cast<int64_t>(tn) * nk;
        const int hook = rank == 0 && warp == 2 ? test_hook(p) : 0;
        for (int kb = k0; kb < k1; ++kb) {
            const uint32_t it = kb - k0, buf = it % kFewBufs;
            float* const sc = scales + (it / kChunk & 1) * kChunk * kN;
            if (it % kChunk == 0) {  // the products of both scales for the next blocks (the other half may still be read)
                for (int i = et; i < kChunk * kN; i += 128) {
                    const int t = tt * kN + i / kChunk, b = kb + i % kChunk;
                    sc[i % kChunk * kN + i / kChunk] = t < p.T && b < k1 ? __ldg(p.a_scale + static_cast<int64_t>(t) * nk + b) * __ldg(sb + b) : 0.0f;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            // a warp whose wait ran out goes on to the end all the same: the others wait for it at the barrier above
            if (!good) continue;
            good = !(it == 5 && hook == kOneWarp) && all(ptx::mbar_wait_near(&st.acc_full[buf], (it / kFewBufs) & 1));
            if (!good) continue;
            ptx::tc_fence_after();
            const float4* s4 = reinterpret_cast<const float4*>(sc + it % kChunk * kN);
#pragma unroll
            for (int c = 0; c < kN; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld16(tq + buf * kN + c, v);
                ptx::tmem_ld_wait();
                if (c + 16 == kN) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&st.acc_empty[buf]);
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 f = s4[(c + i) / 4];
                    acc[c + i] = fmaf(__uint_as_float(v[i]), f.x, acc[c + i]);
                    acc[c + i + 1] = fmaf(__uint_as_float(v[i + 1]), f.y, acc[c + i + 1]);
                    acc[c + i + 2] = fmaf(__uint_as_float(v[i + 2]), f.z, acc[c + i + 2]);
                    acc[c + i + 3] = fmaf(__uint_as_float(v[i + 3]), f.w, acc[c + i + 3]);
                }
            }
        }
        if (!good) fail();
    }
    __syncwarp();
    const int share_log2 = __ffs(kN / cs) - 1, share = 1 << share_log2;  // tokens whose parts this CTA adds (cs: 1, 2, 4 or 8)
    const int row = (warp & 3) * 32 + lane, n = tn * kFewM + row;
    auto store = [&](int c, float v) {
        const int t = tt * kN + c;
        if (t >= p.T || n >= p.N) return;
        const int64_t at = static_cast<int64_t>(t) * p.ld_out + n;
        if constexpr (kF32) static_cast<float*>(p.out)[at] = v;
        else static_cast<uint16_t*>(p.out)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
    };
    if (cs > 1) {
        ptx::cluster_wait();
        // without one CTA's part there is no sum: every CTA of the cluster hears of it
        if (__any_sync(0xFFFFFFFFu, failed) && lane < cs) ptx::cluster_store(ptx::cluster_addr(&st.abort, lane), __int_as_float(1));
        if (warp >= 2) {
#pragma unroll
            for (int c = 0; c < kN; ++c) {
                const uint32_t to = ptx::cluster_addr(part + ((rank << share_log2) + (c & (share - 1))) * kFewM + row, c >> share_log2);
                ptx::cluster_store(to, acc[c]);
            }
        }
        ptx::cluster_sync();
        if (warp >= 2 && !*reinterpret_cast<volatile int*>(&st.abort))
            for (int c = 0; c < share; ++c) {
                float v = 0.0f;
                for (int r = 0; r < cs; ++r) v += part[(r * share + c) * kFewM + row];
                store(rank * share + c, v);
            }
    } else if (warp >= 2 && good) {
#pragma unroll
        for (int c = 0; c < kN; ++c) store(c, acc[c]);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        ptx::tmem_dealloc(tmem, S::kCols);
    }
}

bool maps(const GemmFp8Args& p, CUtensorMap* a, CUtensorMap* b, uint32_t rows_a, uint32_t rows_b)
{
    return encode_tmap_3d_u8(a, p.a, p.K, p.T, 1, 128, rows_a) == CUDA_SUCCESS && encode_tmap_3d_u8(b, p.b, p.K, p.N, 1, 128, rows_b) == CUDA_SUCCESS;
}

template <bool kF32>
cudaError_t launch_big(const GemmFp8Args& p, int sms, cudaStream_t stream)
{
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(smem_set, reinterpret_cast<const void*>(k_gemm_fp8<kF32>), kBigSmem);
    if (e != cudaSuccess) return e;
    CUtensorMap a, b, out;
    if (!maps(p, &a, &b, kBigM, kBigN) || encode_tmap_2d_out(&out, p.out, kF32, p.N, p.T, p.ld_out, kF32 ? 32 : 64, 32) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const int tn = (p.N + kBigN - 1) / kBigN, tm = (p.T - 1) / kBigM + 1;
    const int64_t tiles = static_cast<int64_t>(tn) * tm;
    if (tiles > 0x7FFFFFFF - 65536) return cudaErrorInvalidValue;
    return launch_pdl(k_gemm_fp8<kF32>, dim3(tiles < sms ? static_cast<int>(tiles) : sms), dim3(kBigThreads), kBigSmem, stream, a, b, out, p, tn,
                      static_cast<int>(tiles));
}

// CTAs that share a tile: as many as all fit at the same time, two an SM
int few_cluster(int64_t tiles, int nk, int sms)
{
    int cs = 1;
    while (cs < 8 && tiles * cs * 2 <= sms * 2 && cs * 2 <= nk) cs *= 2;
    return cs;
}

template <int kN, bool kF32>
cudaError_t launch_few(const GemmFp8Args& p, int sms, cudaStream_t stream)
{
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_smem(smem_set, reinterpret_cast<const void*>(k_gemm_fp8_few<kN, kF32>), few_smem<kN>());
    if (e != cudaSuccess) return e;
    CUtensorMap a, b;
    if (!maps(p, &a, &b, kN, kFewM)) return cudaErrorInvalidValue;
    const int tt = (p.T - 1) / kN + 1, tn = (p.N + kFewM - 1) / kFewM, nk = (p.K + 127) / 128;
    const int64_t tiles = static_cast<int64_t>(tt) * tn;
    const int cs = few_cluster(tiles, nk, sms);
    if (tiles * cs > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * cs));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = few_smem<kN>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_gemm_fp8_few<kN, kF32>, a, b, p, tt);
}

template <bool kF32>
cudaError_t launch(const GemmFp8Args& p, int sms, cudaStream_t stream)
{
    if (p.T > 32) {
        // A multiprocessor passes a block of K in 0.5 to 0.6 us in either kernel, whatever its tile, and joining a cluster's
        // parts takes some 2 us: what has fewer rounds of tiles (512 x 4,096 x 2,048: 9 us with the wide tiles, 21 with 64
        // tokens; 512 x 1,024 x 4,096: 15 and 12; 128 x 1,024 x 4,096: 19 and 8).
        const int nk = (p.K + 127) / 128;
        const int64_t wide = static_cast<int64_t>((p.T - 1) / kBigM + 1) * ((p.N + kBigN - 1) / kBigN);
        const int64_t few = static_cast<int64_t>((p.T - 1) / 64 + 1) * ((p.N + kFewM - 1) / kFewM);
        const int cs = few_cluster(few, nk, sms);
        if ((wide + sms - 1) / sms * nk <= (few * cs + sms - 1) / sms * ((nk + cs - 1) / cs) + (cs > 1 ? 4 : 0)) return launch_big<kF32>(p, sms, stream);
    }
    if (p.T <= 16) return launch_few<16, kF32>(p, sms, stream);
    if (p.T <= 32) return launch_few<32, kF32>(p, sms, stream);
    return launch_few<64, kF32>(p, sms, stream);
}

}  // namespace

cudaError_t launch_gemm_fp8(const GemmFp8Args& p, int sms, cudaStream_t stream)
{
    return p.out_f32 ? launch<true>(p, sms, stream) : launch<false>(p, sms, stream);
}

}  // namespace moe
