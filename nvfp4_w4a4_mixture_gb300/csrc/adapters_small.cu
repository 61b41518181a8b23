// adapters_small.cu -- low-rank adapters where requests are short or the batch is: tiles of up to 8 rows
// of one request, bounded by reading A and B (from L2 where requests share an adapter).
//
// One CTA of eight warps a tile, or a cluster that shares K and then N. Both products are mma.sync
// m16n8k16 (bf16, FP32 sums) on operands loaded straight from global memory, 16 bytes a thread: a
// thread's eight neighbouring k take the places of the fragments' k pairs in both operands alike, so
// no operand passes through shared memory.
//   phase 1  h[j][t] = A_j . x_t: rank rows on M, tokens on N; the warps share rank rows and K; their
//            partial sums meet in shared memory (and through distributed shared memory in a cluster),
//            always added in the same order; h scale = hi + lo, two bf16 values
//   phase 2  d[t][c] = hi_t . B_c + lo_t . B_c: tokens on M, hi in rows 0..7 and lo in rows 8..15 (their
//            sums are added at the end), columns on N. Column 2q + e of product i stands for column 8q + 2i
//            + e of 32, so that a thread ends with eight neighbouring columns of a row: one 16-byte load of
//            y and one store of out. Ranks up to 16 take 8 bytes a thread and one product of 16.
// Measured, 2048 x 2048: 256 requests of one token, rank 32 10.2 us (52 MB of A and B from L2, 5 TB/s);
// 4 tokens, rank 16 4.3 us, the chain of one tile.
#include "adapters.cuh"

namespace moe {

namespace {

using namespace adapters;

constexpr int kM = 8;  // rows of a tile
constexpr int kWarps = 8, kThreads = 32 * kWarps;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d += a (rows g and g + 8) b over 32 k: two products of 16.
__device__ __forceinline__ void mma32(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& b)
{
    mma(d, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
    mma(d, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

__device__ __forceinline__ uint4 load16(const uint16_t* p, bool in)
{
    return in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

// y may be out: not through the path of data that the kernel does not change
__device__ __forceinline__ uint4 load16_y(const uint16_t* p, bool in)
{
    return in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
}

template <int kR>
__global__ void __launch_bounds__(kThreads, 2) k_adapter_add_small(const __grid_constant__ AdapterArgs p)
{
    constexpr int kBlocks = kR / 16, kSplit = kWarps / kBlocks;  // 16-row blocks of the rank, warps that share K
    constexpr int kSteps = (kR + 31) / 32;                       // 32 ranks each
    constexpr int kHld = kSteps * 32 + 8;                        // a token's h in shared memory (padded: other banks)
    constexpr int kUnroll1 = 8, kUnroll2 = kSteps <= 2 ? 4 / kSteps : 1;
    __shared__ float part[kSplit][kR * kM], sums[8][kR * kM];  // of the warps that share K, of the cluster's CTAs
    __shared__ __align__(16) uint16_t h_s[2][kM][kHld];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, q = lane % 4;
    const int cs = static_cast<int>(ptx::cluster_size()), rank = static_cast<int>(ptx::cluster_rank());
    const int cluster = blockIdx.x / cs, n_clusters = gridDim.x / cs;
    // A CTA's shared memory may be written by the others once that CTA has started: all arrive here, and wait
    // before their first store to another (as before each tile's, then for the readers of the tile before).
    if (cs > 1) ptx::cluster_arrive_all();
    // rows of h that no token fills, and columns past the rank, stay zero
    for (int i = tid; i < static_cast<int>(sizeof(h_s) / 4); i += kThreads) reinterpret_cast<uint32_t*>(h_s)[i] = 0u;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int nc = (p.N + 31) / 32, c0 = nc * rank / cs, c1 = nc * (rank + 1) / cs;  // this CTA's slices of 32 columns
    Walk<kM> walk;
    Tile t;
    const bool check = blockIdx.x == 0 && warp == 0;
    for (int number = cluster; walk.find(p, number, t, check); number += n_clusters) {
        if (t.adapter < 0) {
            const int w = min(c1 * 32, p.N) / 8 - c0 * 4;  // 16-byte pieces of a row
            for (int i = tid; i < w * t.rows; i += kThreads) {
                const int64_t row = t.row + i / w;
                const int col = c0 * 32 + i % w * 8;
                *reinterpret_cast<uint4*>(p.out + row * p.ld_out + col) = load16_y(p.y + row * p.ld_y + col, true);
            }
            continue;
        }
        {
            const int rb = warp % kBlocks, kw = warp / kBlocks;
            const int steps = (p.K + 31) / 32, share = cs * kSplit, me = rank * kSplit + kw;
            const int s0 = steps * me / share, s1 = steps * (me + 1) / share;
            const int j0 = rb * 16 + g;
            const uint16_t* a0 = p.a + (static_cast<int64_t>(t.adapter) * p.r + j0) * p.K;
            const uint16_t* x0 = p.x + (t.row + g) * p.ld_x;
            float d[4] = {};
            for (int s = s0; s < s1; s += kUnroll1) {
                uint4 av[kUnroll1][2], xv[kUnroll1];
#pragma unroll
                for (int u = 0; u < kUnroll1; ++u) {
                    const int k = (s + u) * 32 + q * 8;
                    const bool in = s + u < s1 && k < p.K;
                    av[u][0] = load16(a0 + k, in && j0 < p.r);
                    av[u][1] = load16(a0 + static_cast<int64_t>(8) * p.K + k, in && j0 + 8 < p.r);
                    xv[u] = load16(x0 + k, in && g < t.rows);
                }
#pragma unroll
                for (int u = 0; u < kUnroll1; ++u) mma32(d, av[u][0], av[u][1], xv[u]);
            }
            float* out = part[kw] + j0 * kM + 2 * q;
            *reinterpret_cast<float2*>(out) = make_float2(d[0], d[1]);
            *reinterpret_cast<float2*>(out + 8 * kM) = make_float2(d[2], d[3]);
        }
        // phase 2's first columns and their y come while the partial sums meet
        uint4 bv[kUnroll2][4][kSteps], yv[kUnroll2];
        const uint16_t* b0 = p.b + static_cast<int64_t>(t.adapter) * p.N * p.r;
        auto load_b = [&](int c) {
#pragma unroll
            for (int u = 0; u < kUnroll2; ++u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = (c + u) * 32 + g / 2 * 8 + 2 * i + g % 2;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const int k = kR == 16 ? q * 4 : s * 32 + q * 8;
                        const bool in = c + u < c1 && n < p.N && k < p.r;
                        if constexpr (kR == 16) {
                            const uint2 v = in ? __ldg(reinterpret_cast<const uint2*>(b0 + n * p.r + k)) : make_uint2(0, 0);
                            bv[u][i][s] = make_uint4(v.x, v.y, 0, 0);
                        } else {
                            bv[u][i][s] = load16(b0 + n * p.r + k, in);
                        }
                    }
                }
                const int col = (c + u) * 32 + q * 8;
                yv[u] = load16_y(p.y + (t.row + g) * p.ld_y + col, c + u < c1 && col < p.N && g < t.rows);
            }
        };
        load_b(c0 + warp * kUnroll2);
        __syncthreads();
        if (cs > 1) {  // this CTA's sum goes to every CTA of the cluster
            ptx::cluster_wait();  // all of them have started and have read the sums of the tile before
            for (int i = tid; i < kR * kM; i += kThreads) {
                float v = part[0][i];
#pragma unroll
                for (int w = 1; w < kSplit; ++w) v += part[w][i];
                for (int o = 0; o < cs; ++o) ptx::cluster_store(ptx::cluster_addr(&sums[rank][i], o), v);
            }
            ptx::cluster_sync();
        }
        const float f = __ldg(p.scale + t.adapter);
        for (int i = tid; i < kR * kM / 2; i += kThreads) {  // rank rows 2j and 2j + 1 of a token
            const int tok = i % kM, j = i / kM * 2;
            float u = 0.0f, v = 0.0f;
            if (cs > 1) {
                for (int o = 0; o < cs; ++o) {
                    u += sums[o][j * kM + tok];
                    v += sums[o][(j + 1) * kM + tok];
                }
            } else {
#pragma unroll
                for (int w = 0; w < kSplit; ++w) {
                    u += part[w][j * kM + tok];
                    v += part[w][(j + 1) * kM + tok];
                }
            }
            uint32_t hi, lo;
            split(j < p.r, u * f, v * f, hi, lo);
            *reinterpret_cast<uint32_t*>(&h_s[0][tok][j]) = hi;
            *reinterpret_cast<uint32_t*>(&h_s[1][tok][j]) = lo;
        }
        if (cs > 1) ptx::cluster_arrive_all();  // this CTA has read the cluster's sums
        __syncthreads();

        uint4 hi[kSteps], lo[kSteps];  // token g's h, in the order of the products' k
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if constexpr (kR == 16) {
                const uint2 a = *reinterpret_cast<const uint2*>(&h_s[0][g][q * 4]), b = *reinterpret_cast<const uint2*>(&h_s[1][g][q * 4]);
                hi[s] = make_uint4(a.x, a.y, 0, 0);
                lo[s] = make_uint4(b.x, b.y, 0, 0);
            } else {
                hi[s] = *reinterpret_cast<const uint4*>(&h_s[0][g][s * 32 + q * 8]);
                lo[s] = *reinterpret_cast<const uint4*>(&h_s[1][g][s * 32 + q * 8]);
            }
        }
        for (int c = c0 + warp * kUnroll2; c < c1; c += kWarps * kUnroll2) {
            if (c != c0 + warp * kUnroll2) load_b(c);
#pragma unroll
            for (int u = 0; u < kUnroll2; ++u) {
                const int col = (c + u) * 32 + q * 8;
                float d[4][4] = {};
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (kR == 16) mma(d[i], hi[s].x, lo[s].x, hi[s].y, lo[s].y, bv[u][i][s].x, bv[u][i][s].y);
                        else mma32(d[i], hi[s], lo[s], bv[u][i][s]);
                    }
                const uint32_t yy[4] = {yv[u].x, yv[u].y, yv[u].z, yv[u].w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = pack_bf16x2(bf16_to_f32(yy[i] & 0xFFFFu) + (d[i][0] + d[i][2]), bf16_to_f32(yy[i] >> 16) + (d[i][1] + d[i][3]));
                if (c + u < c1 && col < p.N && g < t.rows)
                    *reinterpret_cast<uint4*>(p.out + (t.row + g) * p.ld_out + col) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        __syncthreads();  // h is read
    }
    if (check) report(p, walk);
    if (cs > 1) ptx::cluster_wait();  // the last arrival's
}

template <int kR>
cudaError_t launch(const AdapterArgs& a, int cs, int64_t tiles, int sms, cudaStream_t stream)
{
    const int64_t room = 2LL * sms / cs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((tiles < room ? tiles : room) * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_adapter_add_small<kR>, a);
}

}  // namespace

cudaError_t launch_adapter_add_small(const AdapterArgs& a, int sms, cudaStream_t stream)
{
    // CTAs a tile: up to one round of two CTAs a multiprocessor, while a CTA keeps 64 KB of A and B to read
    // (32 KB where there is room for all in one CTA a multiprocessor): 64 requests of rank 64 14.1 us with one
    // CTA a tile, 9.5 with four; of rank 16 7.1 with one, 6.4 with two, 7.6 with four. Eight for a few tiles
    // alone: 4 tokens of rank 64 6.7 us against 7.2 with four, 256 tokens of one request 9.0 against 7.6.
    const int64_t tiles = adapter_tiles(a, kM), bytes = 2LL * a.r * (a.K + a.N);
    int cs = tiles * 16 <= sms ? 8 : 4;
    while (cs > 1 && (tiles * cs > 2LL * sms || bytes / cs < (tiles * cs > sms ? 65536 : 32768))) cs /= 2;
    if (a.r <= 16) return launch<16>(a, cs, tiles, sms, stream);
    if (a.r <= 32) return launch<32>(a, cs, tiles, sms, stream);
    if (a.r <= 64) return launch<64>(a, cs, tiles, sms, stream);
    return launch<128>(a, cs, tiles, sms, stream);
}

}  // namespace moe
