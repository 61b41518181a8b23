// adapters.cu -- low-rank adapters of many requests: out[t] = y[t] + scale_a B_a (A_a x[t]).
//
// The requests' rows are cut into tiles of up to tile_rows (<= 128) rows of one request. A tile is
// two tensor-core products (tcgen05 kind::f16, FP32 in tensor memory) of one CTA or of a cluster:
//   phase 1  h = x A^T over this CTA's share of K, in slices of 64 columns
//            (cluster: the partial h of all CTAs are added through distributed shared memory, in the
//            order of their ranks, so every CTA holds the same h)
//            h scale = hi + lo, two bf16 values (16 significant bits), written to shared memory as
//            the A operand of
//   phase 2  d = hi B^T + lo B^T over this CTA's share of N, in slices of 64 columns; out = y + d
// Warp 0 streams both phases through one ring by TMA (x and A slices, then y and B slices: phase 2's
// loads run while phase 1 ends), warp 1 issues the MMAs, warps 2-5 read the accumulators (one TMEM
// lane quarter each), add y in the ring's buffer and store rows of 128 bytes.
// Rows of a tile beyond its request's end hold whatever the buffers held; rows do not mix, and those
// are not stored. The zero fill of TMA pads K, N and the rank.
#include "block.cuh"
#include "ptx_cluster.cuh"

namespace moe {

namespace {

constexpr int kThreads = 192, kTileM = 128;
constexpr int kXBytes = kTileM * 128;  // 128 rows x 64 bf16
constexpr uint32_t kD2Col = 128;       // TMEM columns: h at 0..127, two phase-2 accumulators behind it

// kR: the rank, padded (16, 32, 64 or 128)
template <int kR>
struct Shape {
    static constexpr int kBlocks = (kR + 63) / 64;        // 64-column blocks of the rank
    static constexpr int kW = kBlocks * 64 * 128;         // bytes of a B slice (64 rows), >= the A slice (kR rows of 128)
    static_assert(kW >= kR * 128, "an A slice fits");
    static constexpr int kStage = kXBytes + kW;
    static constexpr int kH = kBlocks * kXBytes;          // hi (or lo)
    static constexpr int kStages = kR > 64 ? 4 : 7;
};

template <int kStages>
struct Tail {
    uint64_t full[kStages], empty[kStages];
    uint64_t d1_full, h_ready, d2_full[2], d2_empty[2], p_ready, p_done, drain;
    uint32_t tmem;
    int abort;
};

template <int kR>
constexpr size_t smem_bytes()
{
    return 1024 + static_cast<size_t>(Shape<kR>::kStages) * Shape<kR>::kStage + 2 * Shape<kR>::kH + sizeof(Tail<Shape<kR>::kStages>);
}

struct Tile {
    int row, rows, adapter;  // adapter -1: copy
};

// Walks the requests in order; every warp that needs the tiles has its own.
struct Walk {
    int base = 0, before = 0;  // first segment of the window, tiles before it

    // Warp-wide. The tile of the given number (numbers must not go down), false past the last.
    __device__ bool find(const AdapterArgs& p, int tile_rows, int number, Tile& t)
    {
        const int lane = threadIdx.x & 31;
        for (; base < p.S; base += 32) {
            const int s = base + lane;
            int beg = 0, end = 0, ad = -1, n = 0;
            if (s < p.S) {
                beg = __ldg(p.seg_offsets + s);
                end = __ldg(p.seg_offsets + s + 1);
                ad = __ldg(p.seg_adapter + s);
                const bool good = beg >= 0 && beg <= end && end <= p.T && ad >= -1 && ad < p.n;
                if (good && !(ad < 0 && p.out == p.y)) n = (end - beg + tile_rows - 1) / tile_rows;
            }
            int sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + sum > number);
            if (hit) {
                const int at = __ffs(hit) - 1;
                const int first = __shfl_sync(0xFFFFFFFFu, before + sum - n, at);
                beg = __shfl_sync(0xFFFFFFFFu, beg, at);
                end = __shfl_sync(0xFFFFFFFFu, end, at);
                t.adapter = __shfl_sync(0xFFFFFFFFu, ad, at);
                t.row = beg + (number - first) * tile_rows;
                t.rows = min(tile_rows, end - t.row);
                return true;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        return false;
    }
};

// Rows [row, row + rows) x 64 columns at column c into dst: boxes of 8 rows up to 32 rows, else of 32.
__device__ __forceinline__ uint32_t rows_bytes(int rows) { return rows <= 32 ? (rows + 7) / 8 * 1024u : (rows + 31) / 32 * 4096u; }
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* m8, const CUtensorMap* m32, uint64_t* bar, int c, int row,
                                          int rows)
{
    if (rows <= 32)
        for (int i = 0; i < rows; i += 8) ptx::tma_load_2d(dst + i * 128, m8, bar, c, row + i);
    else
        for (int i = 0; i < rows; i += 32) ptx::tma_load_2d(dst + i * 128, m32, bar, c, row + i);
}

// 16-byte piece j of row r in the 128-byte-swizzled layout
__device__ __forceinline__ uint32_t piece(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

template <int kR>
__global__ void __launch_bounds__(kThreads, 1)
    k_adapter_add(const __grid_constant__ AdapterArgs p, int tile_rows, const __grid_constant__ CUtensorMap map_x8,
                  const __grid_constant__ CUtensorMap map_x32, const __grid_constant__ CUtensorMap map_y8,
                  const __grid_constant__ CUtensorMap map_y32, const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b)
{
    using S = Shape<kR>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* hbuf = smem + kStages * S::kStage;  // hi, lo; before them the partial sums [kR][128] of a cluster
    Tail<kStages>& st = *reinterpret_cast<Tail<kStages>*>(hbuf + 2 * S::kH);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int cs = static_cast<int>(ptx::cluster_size()), rank = static_cast<int>(ptx::cluster_rank());
    const int cluster = blockIdx.x / cs, n_clusters = gridDim.x / cs;
    const int nk = (p.K + 63) / 64, nn = (p.N + 63) / 64;
    const int k0 = nk * rank / cs, k1 = nk * (rank + 1) / cs, n0 = nn * rank / cs, n1 = nn * (rank + 1) / cs;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&st.full[s], 1);
            ptx::mbar_init(&st.empty[s], 5);  // the MMA thread and four epilogue warps
        }
        ptx::mbar_init(&st.d1_full, 1);
        ptx::mbar_init(&st.drain, 1);
        ptx::mbar_init(&st.h_ready, 4);
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&st.d2_full[b], 1);
            ptx::mbar_init(&st.d2_empty[b], 4);
        }
        ptx::mbar_init(&st.p_ready, 4 * cs);
        ptx::mbar_init(&st.p_done, 4 * cs);
        st.abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map_a);
        ptx::prefetch_tmap(&map_b);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&st.tmem, 256);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before();
    __syncthreads();
    if (cs > 1) ptx::cluster_sync();  // the other CTAs' barriers are initialised
    ptx::tc_fence_after();
    const uint32_t tmem = st.tmem;
    auto fail = [&]() {
        if (atomicExch(&st.abort, 1) == 0) record_status(p.status, kDevTimeoutAdapter);
    };
    Walk walk;
    Tile t;

    if (warp == 0) {
        int s = 0;
        uint32_t ph = 0, fills = 0;
        bool ok = true;
        for (int number = cluster; ok && walk.find(p, tile_rows, number, t); number += n_clusters) {
            if (lane == 0) {
                const uint32_t xb = rows_bytes(t.rows);
                for (int kc = k0; ok && t.adapter >= 0 && kc < k1; ++kc) {
                    ok = ptx::mbar_wait(&st.empty[s], ph ^ 1);
                    if (!ok) break;
                    uint8_t* b = smem + s * S::kStage;
                    ptx::mbar_arrive_expect_tx(&st.full[s], xb + kR * 128);
                    load_rows(b, &map_x8, &map_x32, &st.full[s], kc * 64, t.row, t.rows);
                    ptx::tma_load_3d(b + kXBytes, &map_a, &st.full[s], kc * 64, 0, t.adapter);
                    ++fills;
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
                for (int nc = n0; ok && nc < n1; ++nc) {
                    ok = ptx::mbar_wait(&st.empty[s], ph ^ 1);
                    if (!ok) break;
                    uint8_t* b = smem + s * S::kStage;
                    ptx::mbar_arrive_expect_tx(&st.full[s], xb + (t.adapter >= 0 ? S::kW : 0));
                    load_rows(b, &map_y8, &map_y32, &st.full[s], nc * 64, t.row, t.rows);
                    if (t.adapter >= 0)
#pragma unroll
                        for (int kb = 0; kb < S::kBlocks; ++kb)
                            ptx::tma_load_3d(b + kXBytes + kb * 8192, &map_b, &st.full[s], kb * 64, nc * 64, t.adapter);
                    ++fills;
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
                if (!ok) fail();
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        }
        if (lane == 0 && !ptx::ring_drain(st.full, kStages, fills)) fail();
    } else if (warp == 1) {
        constexpr uint32_t idesc1 = ptx::idesc_bf16(kTileM, kR), idesc2 = ptx::idesc_bf16(kTileM, 64);
        const uint64_t dx = ptx::sdesc_sw128(ptx::smem_u32(smem)), dw = ptx::sdesc_sw128(ptx::smem_u32(smem + kXBytes));
        const uint64_t dh = ptx::sdesc_sw128(ptx::smem_u32(hbuf));
        const int ksteps = (p.r + 15) / 16;
        int s = 0;
        uint32_t ph = 0, it = 0, cc = 0;
        bool ok = true;
        for (int number = cluster; ok && walk.find(p, tile_rows, number, t); number += n_clusters) {
            if (lane == 0) {
                if (t.adapter >= 0) {
                    for (int kc = k0; kc < k1; ++kc) {
                        ok = ptx::mbar_wait(&st.full[s], ph);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint64_t so = static_cast<uint64_t>(s) * (S::kStage >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_bf16(tmem, dx + so + kk * 2, dw + so + kk * 2, idesc1, kc > k0 || kk > 0);
                        ptx::mbar_arrive_n(&st.empty[s], 4);
                        ptx::tc_commit(&st.empty[s]);
                        if (++s == kStages) { s = 0; ph ^= 1; }
                    }
                    ptx::tc_commit(&st.d1_full);
                    if (ok) ok = ptx::mbar_wait(&st.h_ready, it & 1);
                    ++it;
                    ptx::tc_fence_after();
                }
                for (int nc = n0; ok && nc < n1; ++nc) {
                    ok = ptx::mbar_wait(&st.full[s], ph);
                    if (!ok) break;
                    if (t.adapter >= 0) {
                        const uint32_t buf = cc & 1;
                        ok = ptx::mbar_wait(&st.d2_empty[buf], ((cc >> 1) & 1) ^ 1);
                        if (!ok) break;
                        ++cc;
                        ptx::tc_fence_after();
                        const uint64_t so = static_cast<uint64_t>(s) * (S::kStage >> 4);
                        const uint32_t d = tmem + kD2Col + buf * 64;
                        for (int kk = 0; kk < ksteps; ++kk) {
                            const uint64_t ho = (kk >> 2) * (kXBytes >> 4) + (kk & 3) * 2, bo = so + (kk >> 2) * (8192 >> 4) + (kk & 3) * 2;
                            ptx::mma_bf16(d, dh + ho, dw + bo, idesc2, kk > 0);
                            ptx::mma_bf16(d, dh + (S::kH >> 4) + ho, dw + bo, idesc2, 1);
                        }
                        ptx::tc_commit(&st.empty[s]);
                        ptx::tc_commit(&st.d2_full[buf]);
                    } else {
                        ptx::mbar_arrive(&st.empty[s]);
                    }
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
                if (!ok) {
                    fail();
                    ptx::tc_commit(&st.drain);  // what was issued ends before the tensor memory goes
                    ptx::mbar_wait(&st.drain, 0);
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        }
    } else {
        const int q = warp & 3, row = q * 32 + lane;  // TMEM lane quarter, row of the tile
        const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
        int s = 0;
        uint32_t ph = 0, it = 0, cc = 0;
        bool ok = true;
        // one lane's wait result may differ from another's only in time: the warp agrees on it
        auto all = [&](bool got) { return __all_sync(0xFFFFFFFFu, got) != 0; };
        if (cluster == 0 && rank == 0 && warp == 2) {
            bool bad = __ldg(p.seg_offsets) != 0 || __ldg(p.seg_offsets + p.S) != p.T;
            for (int i = lane; i < p.S; i += 32) {
                const int beg = __ldg(p.seg_offsets + i), end = __ldg(p.seg_offsets + i + 1), ad = __ldg(p.seg_adapter + i);
                bad |= beg < 0 || beg > end || end > p.T || ad < -1 || ad >= p.n;
            }
            if (bad) record_status(p.status, kDevBadSegment);
        }
        for (int number = cluster; ok && walk.find(p, tile_rows, number, t); number += n_clusters) {
            const bool live = q * 32 < t.rows;  // this warp has rows of the tile
            if (t.adapter >= 0) {
                for (s += k1 - k0; s >= kStages; s -= kStages) ph ^= 1;  // phase 1's stages are not its own
                float h[kR];
                ok = all(ptx::mbar_wait(&st.d1_full, it & 1));
                if (!ok) break;
                ptx::tc_fence_after();
                if (live && k0 < k1) {
#pragma unroll
                    for (int c = 0; c < kR; c += 16) {
                        uint32_t v[16];
                        ptx::tmem_ld16(tq + c, v);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) h[c + i] = __uint_as_float(v[i]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kR; ++c) h[c] = 0.0f;
                }
                ptx::tc_fence_before();
                if (cs > 1) {
                    float* part = reinterpret_cast<float*>(hbuf);  // [kR][128]
                    if (live)
#pragma unroll
                        for (int c = 0; c < kR; ++c) part[c * kTileM + row] = h[c];
                    __syncwarp();
                    if (lane < cs) ptx::cluster_arrive(ptx::cluster_addr(&st.p_ready, lane));
                    ok = all(ptx::mbar_wait_cluster(&st.p_ready, it & 1));
                    if (!ok) break;
                    if (live) {
#pragma unroll
                        for (int c = 0; c < kR; ++c) h[c] = 0.0f;
                        for (int o = 0; o < cs; ++o) {
                            const uint32_t at = ptx::cluster_addr(part + row, o);
#pragma unroll
                            for (int c = 0; c < kR; ++c) h[c] += ptx::cluster_load(at + c * kTileM * 4);
                        }
                    }
                    __syncwarp();
                    if (lane < cs) ptx::cluster_arrive(ptx::cluster_addr(&st.p_done, lane));
                    ok = all(ptx::mbar_wait_cluster(&st.p_done, it & 1));
                    if (!ok) break;
                }
                if (live) {
                    const float f = __ldg(p.scale + t.adapter);
#pragma unroll
                    for (int c = 0; c < kR; c += 8) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // r is even; the padded columns stay zero even where x is not finite
                            const float u = c + 2 * i < p.r ? h[c + 2 * i] * f : 0.0f, v = c + 2 * i < p.r ? h[c + 2 * i + 1] * f : 0.0f;
                            hi[i] = pack_bf16x2(u, v);
                            const float uh = bf16_to_f32(hi[i] & 0xFFFFu), vh = bf16_to_f32(hi[i] >> 16);
                            // an infinity has no remainder
                            lo[i] = pack_bf16x2(fabsf(uh) < INFINITY ? u - uh : 0.0f, fabsf(vh) < INFINITY ? v - vh : 0.0f);
                        }
                        uint8_t* d = hbuf + (c / 64) * kXBytes + piece(row, (c % 64) / 8);
                        *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(d + S::kH) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&st.h_ready);
                ++it;
            }
            for (int nc = n0; nc < n1; ++nc) {
                uint8_t* yb = smem + s * S::kStage;
                if (t.adapter >= 0) {
                    const uint32_t buf = cc & 1;
                    ok = all(ptx::mbar_wait(&st.d2_full[buf], (cc >> 1) & 1)) && all(ptx::mbar_wait(&st.full[s], ph));
                    if (!ok) break;
                    ++cc;
                    ptx::tc_fence_after();
                    if (live) {
                        uint32_t v[4][16];
#pragma unroll
                        for (int i = 0; i < 4; ++i) ptx::tmem_ld16(tq + kD2Col + buf * 64 + i * 16, v[i]);
                        ptx::tmem_ld_wait();
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&st.d2_empty[buf]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint4* at = reinterpret_cast<uint4*>(yb + piece(row, j));
                            const uint4 y = *at;
                            const uint32_t yy[4] = {y.x, y.y, y.z, y.w};
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int c = j * 8 + 2 * i;
                                o[i] = pack_bf16x2(bf16_to_f32(yy[i] & 0xFFFFu) + __uint_as_float(v[c / 16][c % 16]),
                                                   bf16_to_f32(yy[i] >> 16) + __uint_as_float(v[(c + 1) / 16][(c + 1) % 16]));
                            }
                            *at = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                        __syncwarp();
                    } else if (lane == 0) {
                        ptx::mbar_arrive(&st.d2_empty[buf]);
                    }
                } else {
                    ok = all(ptx::mbar_wait(&st.full[s], ph));
                    if (!ok) break;
                }
                if (live) {
                    const int col = nc * 64 + (lane & 7) * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = q * 32 + i * 4 + (lane >> 3);
                        if (r < t.rows && col < p.N)
                            *reinterpret_cast<uint4*>(p.out + (t.row + r) * p.ld_out + col) =
                                *reinterpret_cast<const uint4*>(yb + piece(r, lane & 7));
                    }
                    ptx::fence_proxy_async_smem();  // the next fill of this buffer comes through the async proxy
                    __syncwarp();
                }
                if (lane == 0) ptx::mbar_arrive(&st.empty[s]);
                if (++s == kStages) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) fail();
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        ptx::tmem_dealloc(tmem, 256);
    }
    if (cs > 1) ptx::cluster_sync();  // no CTA leaves while another reads its shared memory
}

CUresult map_rows(CUtensorMap* m, const uint16_t* base, int64_t cols, int64_t rows, int64_t ld, uint32_t box_rows)
{
    const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, strides[1] = {static_cast<uint64_t>(ld) * 2};
    const uint32_t box[2] = {64, box_rows};
    return encode_tmap_bf16(m, base, 2, dims, strides, box, 128);
}

CUresult map_bank(CUtensorMap* m, const uint16_t* base, int64_t cols, int64_t rows, int64_t n, uint32_t box_rows)
{
    const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(n)};
    const uint64_t strides[2] = {static_cast<uint64_t>(cols) * 2, static_cast<uint64_t>(cols * rows) * 2};
    const uint32_t box[3] = {64, box_rows, 1};
    return encode_tmap_bf16(m, base, 3, dims, strides, box, 128);
}

template <int kR>
cudaError_t launch(const AdapterArgs& a, int sms, cudaStream_t stream)
{
    static bool attr_set = false;
    if (!attr_set) {
        cudaError_t e = cudaFuncSetAttribute(k_adapter_add<kR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem_bytes<kR>()));
        if (e != cudaSuccess) return e;
        attr_set = true;
    }
    CUtensorMap x8, x32, y8, y32, ma, mb;
    if (map_rows(&x8, a.x, a.K, a.T, a.ld_x, 8) != CUDA_SUCCESS || map_rows(&x32, a.x, a.K, a.T, a.ld_x, 32) != CUDA_SUCCESS ||
        map_rows(&y8, a.y, a.N, a.T, a.ld_y, 8) != CUDA_SUCCESS || map_rows(&y32, a.y, a.N, a.T, a.ld_y, 32) != CUDA_SUCCESS ||
        map_bank(&ma, a.a, a.K, a.r, a.n, kR) != CUDA_SUCCESS || map_bank(&mb, a.b, a.r, a.N, a.n, 64) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const int tile_rows = kTileM;
    // a request of L rows has ceil(L / tile_rows) tiles: at most this many in all
    const int64_t tiles = a.T / tile_rows + (a.S < a.T ? a.S : a.T);
    int cs = 8;
    while (cs > 1 && tiles * cs > sms) cs /= 2;
    const int clusters = static_cast<int>(tiles * cs <= sms ? tiles : sms / cs);

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * cs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<kR>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_adapter_add<kR>, a, tile_rows, x8, x32, y8, y32, ma, mb);
}

}  // namespace

cudaError_t launch_adapter_add(const AdapterArgs& a, int sms, cudaStream_t stream)
{
    if (a.T <= 0) return cudaSuccess;
    if (a.r <= 16) return launch<16>(a, sms, stream);
    if (a.r <= 32) return launch<32>(a, sms, stream);
    if (a.r <= 64) return launch<64>(a, sms, stream);
    return launch<128>(a, sms, stream);
}

}  // namespace moe
