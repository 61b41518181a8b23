// adapters.cu -- low-rank adapters of many requests: out[t] = y[t] + scale_a B_a (A_a x[t]).
//
// The requests' rows are cut into tiles of up to 128 (or 64) rows of one request. A tile is
// two tensor-core products (tcgen05 kind::f16, FP32 in tensor memory) of one CTA or of a cluster:
//   phase 1  h = x A^T over this CTA's share of K, in slices of 64 columns
//            (cluster: the partial h of all CTAs are added through distributed shared memory, in the
//            order of their ranks, so every CTA holds the same h)
//            h scale = hi + lo, two bf16 values (16 significant bits), written to shared memory as
//            the A operand of
//   phase 2  d = hi B^T + lo B^T over this CTA's share of N, in slices of 64 columns; out = y + d
// Warps 0 and 2 stream both phases through one ring by TMA (x and A slices, then y and B slices: phase
// 2's loads run while phase 1 ends), warp 1 issues the MMAs, two groups of four warps (a TMEM lane
// quarter each) take phase 2's slices in turn: they read an accumulator, add y from the ring's buffer
// and store rows.
// Bounded by memory where the batch fills the multiprocessors (16,384 tokens of 24 requests, rank 64,
// 2048 x 2048: 38.0 us, 5.4 TB/s, 81 % of what a copy reaches), else by the chain of one tile (4,113
// tokens of 77 requests, rank 40, 2056 x 1032: 17.1 us, 141 CTAs).
// Rows of a tile beyond its request's end hold whatever the buffers held; rows do not mix, and those
// are not stored. The zero fill of TMA pads K, N and the rank.
#include "adapters.cuh"

namespace moe {

namespace {

using namespace adapters;

constexpr int kTileM = 128;            // rows of an MMA
constexpr int kGroups = 2;             // epilogue groups of four warps; they take phase 2's slices in turn
constexpr int kEpiWarps = 4 * kGroups, kFirstEpi = 3, kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kBufs = 2 * kGroups;     // phase-2 accumulators
constexpr uint32_t kD2Col = 128;       // TMEM columns: h at 0..127, the phase-2 accumulators behind it
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemMax = 227 * 1024;

// kR: the rank, padded (16, 32, 64 or 128); kRows: the most rows of a tile (128 or 64: of an MMA's other rows the
// operands are whatever lies behind in shared memory)
template <int kR, int kRows>
struct Shape {
    static constexpr int kBlocks = (kR + 63) / 64;        // 64-column blocks of the rank
    static constexpr int kX = kRows * 128;                // x or y slice: 64 bf16 a row
    static constexpr int kW = kBlocks * 64 * 128;         // bytes of a B slice (64 rows), >= the A slice (kR rows of 128)
    static_assert(kW >= kR * 128, "an A slice fits");
    static constexpr int kStage = kX + kW;
    static constexpr int kH = kBlocks * kX;               // hi (or lo)
    static constexpr int kOutStage = kGroups * kRows * 128;  // 32 rows x 128 bytes a warp that has rows
    static constexpr int kPart = kRows * kR * 4;          // a cluster's partial h, before the stores need their buffers
    static constexpr int kOut = kPart > kOutStage ? kPart : kOutStage;
    static constexpr int kStages = (kSmemMax - 2048 - 2 * kH - kOut) / kStage;
    static_assert(kStages >= 3, "buffers");
    static_assert(kX + kW >= kTileM * 128 && kX + kOut >= kTileM * 128, "an MMA's 128 rows stay inside");
};

template <int kStages>
struct Tail {
    uint64_t full[kStages], empty[kStages];
    uint64_t d1_full, h_ready, d2_full[kBufs], d2_empty[kBufs], p_ready, p_done, idle, drain;
    uint32_t tmem;
    int abort;
};

template <int kR, int kRows>
constexpr size_t smem_bytes()
{
    using S = Shape<kR, kRows>;
    constexpr size_t n = 1024 + static_cast<size_t>(S::kStages) * S::kStage + 2 * S::kH + S::kOut + sizeof(Tail<S::kStages>);
    static_assert(n <= kSmemMax, "shared memory");
    return n;
}

// Rows [row, row + rows) x 64 columns at column c into dst, by one thread: boxes of 8 rows up to 24
// rows, of 32 up to 32 less than a full tile, else one of a tile. box: the rows of a box, n: their number.
template <int kRows>
struct Boxes {
    int box, n;
    __device__ explicit Boxes(int rows) : box(rows <= 24 ? 8 : rows <= kRows - 32 ? 32 : kRows), n((rows + box - 1) / box) {}
    __device__ uint32_t bytes() const { return static_cast<uint32_t>(box * n) * 128u; }
    __device__ void load(uint8_t* dst, const CUtensorMap* m8, const CUtensorMap* m32, const CUtensorMap* m_all, uint64_t* bar, int c,
                         int row) const
    {
        const CUtensorMap* m = box == 8 ? m8 : box == 32 ? m32 : m_all;
        for (int i = 0; i < n; ++i) ptx::tma_load_2d(dst + i * box * 128, m, bar, c, row + i * box);
    }
};

// 16-byte piece j of row r in the 128-byte-swizzled layout
__device__ __forceinline__ uint32_t piece(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// Warp-wide: kN (a multiple of 4) columns of this warp's TMEM lanes.
template <int kN>
__device__ __forceinline__ void load_h(uint32_t taddr, uint32_t (&v)[kN])
{
#pragma unroll
    for (int c = 0; c < kN; c += 4) ptx::tmem_ld4(taddr + c, v + c);
    ptx::tmem_ld_wait();
}

template <int kR, int kRows>
__global__ void __launch_bounds__(kThreads, 1)
    k_adapter_add(const __grid_constant__ AdapterArgs p, const __grid_constant__ CUtensorMap map_x8,
                  const __grid_constant__ CUtensorMap map_x32, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_y8, const __grid_constant__ CUtensorMap map_y32,
                  const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b)
{
    using S = Shape<kR, kRows>;
    constexpr int kXBytes = S::kX;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* hbuf = smem + kStages * S::kStage;  // hi, lo
    uint8_t* obuf = hbuf + 2 * S::kH;            // rows to store, 4 KB a warp; before that a cluster's partial h
    Tail<kStages>& st = *reinterpret_cast<Tail<kStages>*>(obuf + S::kOut);
    const int tid = threadIdx.x, warp = __reduce_max_sync(0xFFFFFFFFu, tid / 32), lane = tid % 32;
    const int cs = static_cast<int>(ptx::cluster_size()), rank = static_cast<int>(ptx::cluster_rank());
    const int cluster = blockIdx.x / cs, n_clusters = gridDim.x / cs;
    const int nk = (p.K + 63) / 64, nn = (p.N + 63) / 64;
    const int k0 = nk * rank / cs, k1 = nk * (rank + 1) / cs, n0 = nn * rank / cs, n1 = nn * (rank + 1) / cs;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&st.full[s], 2);   // the two loading warps
            ptx::mbar_init(&st.empty[s], 5);  // the MMA thread and the four warps of an epilogue group
        }
        ptx::mbar_init(&st.d1_full, 1);
        ptx::mbar_init(&st.drain, 1);
        ptx::mbar_init(&st.h_ready, kEpiWarps);
        ptx::mbar_init(&st.idle, kEpiWarps);
        for (int b = 0; b < kBufs; ++b) {
            ptx::mbar_init(&st.d2_full[b], 1);
            ptx::mbar_init(&st.d2_empty[b], 4);
        }
        ptx::mbar_init(&st.p_ready, kEpiWarps * cs);
        ptx::mbar_init(&st.p_done, kEpiWarps * cs);
        st.abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&map_a);
        ptx::prefetch_tmap(&map_b);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&st.tmem, kTmemCols);
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
    Walk<kRows> walk;
    Tile t;

    // The issuing warps run their loops whole and one lane issues: loop counters, addresses and
    // descriptors stay uniform (a loop inside `if (lane == 0)` took 460 cycles a slice of two TMA
    // copies and 120 an MMA, for moving its operands to uniform registers).
    if (warp == 0 || warp == 2) {
        // warp 0 loads x and y, warp 2 A and B (one warp's issue of both took 320 cycles a slice)
        const bool leader = ptx::elect_one(), rows = warp == 0;
        int s = 0;
        uint32_t ph = 0, fills = 0;
        bool ok = true;
        for (int number = cluster; ok && walk.find(p, number, t); number += n_clusters) {
            const Boxes<kRows> boxes(t.rows);
            if (t.adapter >= 0)
                for (int kc = k0; kc < k1; ++kc) {
                    ok = __all_sync(0xFFFFFFFFu, ptx::mbar_wait_near(&st.empty[s], ph ^ 1));
                    if (!ok) break;
                    uint8_t* b = smem + s * S::kStage;
                    if (leader) {
                        ptx::mbar_arrive_expect_tx(&st.full[s], rows ? boxes.bytes() : kR * 128);
                        if (rows) boxes.load(b, &map_x8, &map_x32, &map_x, &st.full[s], kc * 64, t.row);
                        else ptx::tma_load_3d(b + kXBytes, &map_a, &st.full[s], kc * 64, 0, t.adapter);
                    }
                    ++fills;
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
            for (int nc = n0; ok && nc < n1; ++nc) {
                ok = __all_sync(0xFFFFFFFFu, ptx::mbar_wait_near(&st.empty[s], ph ^ 1));
                if (!ok) break;
                uint8_t* b = smem + s * S::kStage;
                if (leader) {
                    if (rows) {
                        ptx::mbar_arrive_expect_tx(&st.full[s], boxes.bytes());
                        boxes.load(b, &map_y8, &map_y32, &map_y, &st.full[s], nc * 64, t.row);
                    } else if (t.adapter >= 0) {
                        ptx::mbar_arrive_expect_tx(&st.full[s], S::kW);
#pragma unroll
                        for (int kb = 0; kb < S::kBlocks; ++kb)
                            ptx::tma_load_3d(b + kXBytes + kb * 8192, &map_b, &st.full[s], kb * 64, nc * 64, t.adapter);
                    } else {
                        ptx::mbar_arrive(&st.full[s]);
                    }
                }
                ++fills;
                if (++s == kStages) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) fail();
        if (leader && !ptx::ring_drain(st.full, kStages, fills)) fail();
    } else if (warp == 1) {
        constexpr uint32_t idesc1 = ptx::idesc_bf16(kTileM, kR), idesc2 = ptx::idesc_bf16(kTileM, 64);
        const uint64_t dx = ptx::sdesc_sw128(ptx::smem_u32(smem)), dw = ptx::sdesc_sw128(ptx::smem_u32(smem + kXBytes));
        const uint64_t dh = ptx::sdesc_sw128(ptx::smem_u32(hbuf));
        const int ksteps = (p.r + 15) / 16;
        const bool leader = ptx::elect_one();
        auto all = [&](bool got) { return __all_sync(0xFFFFFFFFu, got) != 0; };
        // a test makes the wait for h run out: then it is for a barrier that nobody arrives at
        const bool stuck = *reinterpret_cast<const volatile int*>(&p.hooks->test_ready_extra) > 0;
        int s = 0;
        uint32_t ph = 0, it = 0, cc = 0;
        bool ok = true;
        for (int number = cluster; ok && walk.find(p, number, t); number += n_clusters) {
            if (t.adapter >= 0) {
                for (int kc = k0; kc < k1; ++kc) {
                    ok = all(ptx::mbar_wait_near(&st.full[s], ph));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint64_t so = static_cast<uint64_t>(s) * (S::kStage >> 4);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_bf16(tmem, dx + so + kk * 2, dw + so + kk * 2, idesc1, kc > k0 || kk > 0);
                        ptx::mbar_arrive_n(&st.empty[s], 4);
                        ptx::tc_commit(&st.empty[s]);
                    }
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
                if (leader) ptx::tc_commit(&st.d1_full);
                if (stuck) ok = ok && all(ptx::mbar_wait_us(&st.drain, 0, p.hooks->test_wait_us));
                else ok = ok && all(ptx::mbar_wait(&st.h_ready, it & 1));
                ++it;
                ptx::tc_fence_after();
            }
            for (int nc = n0; ok && nc < n1; ++nc, ++cc) {
                const uint32_t buf = cc % kBufs;
                ok = all(ptx::mbar_wait_near(&st.full[s], ph)) && all(ptx::mbar_wait_near(&st.d2_empty[buf], ((cc / kBufs) & 1) ^ 1));
                if (!ok) break;
                if (t.adapter >= 0) {
                    ptx::tc_fence_after();
                    const uint64_t so = static_cast<uint64_t>(s) * (S::kStage >> 4);
                    const uint32_t d = tmem + kD2Col + buf * 64;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kR / 16; ++kk) {
                            if (kk >= ksteps) break;
                            const uint64_t ho = (kk >> 2) * (kXBytes >> 4) + (kk & 3) * 2, bo = so + (kk >> 2) * (8192 >> 4) + (kk & 3) * 2;
                            ptx::mma_bf16(d, dh + ho, dw + bo, idesc2, kk > 0);
                            ptx::mma_bf16(d, dh + (S::kH >> 4) + ho, dw + bo, idesc2, 1);
                        }
                        ptx::tc_commit(&st.empty[s]);
                        ptx::tc_commit(&st.d2_full[buf]);
                    }
                } else if (leader) {  // a tile to copy takes the same turns, without a product
                    ptx::mbar_arrive(&st.empty[s]);
                    ptx::mbar_arrive(&st.d2_full[buf]);
                }
                if (++s == kStages) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) {
            fail();
            if (leader) ptx::tc_commit(&st.drain);  // what was issued ends before the tensor memory goes
            ptx::mbar_wait(&st.drain, 0);
        }
    } else {
        // group g: its share of h's columns, every kGroups-th slice of phase 2; q: TMEM lane quarter
        const int ew = warp - kFirstEpi, g = ew / 4, q = warp & 3, row = q * 32 + lane;
        const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t ob = ptx::smem_u32(obuf) + (g * (kRows / 32) + q) * 4096;  // (of a warp that has rows)
        int s = 0;
        uint32_t ph = 0, it = 0, cc = 0, tiles = 0;
        bool ok = true;
        // one lane's wait result may differ from another's only in time: the warp agrees on it
        auto all = [&](bool got) { return __all_sync(0xFFFFFFFFu, got) != 0; };
        const bool check = cluster == 0 && rank == 0 && ew == 0;
        for (int number = cluster; ok && walk.find(p, number, t, check); number += n_clusters, ++tiles) {
            const bool live = q * 32 < t.rows;  // this warp has rows of the tile
            // a cluster: no warp is a tile ahead of another (their buffers are about to hold partial sums)
            if (cs > 1 && tiles > 0) ok = all(ptx::mbar_wait(&st.idle, (tiles - 1) & 1));
            if (!ok) break;
            if (t.adapter >= 0) {
                for (s += k1 - k0; s >= kStages; s -= kStages) ph ^= 1;  // phase 1's stages are not its own
                constexpr int kShare = kR / kGroups;
                const int c0 = g * kShare;
                const float f = __ldg(p.scale + t.adapter);
                ok = all(ptx::mbar_wait(&st.d1_full, it & 1));
                if (!ok) break;
                ptx::tc_fence_after();
                if (cs == 1) {
                    if (live) {
                        uint32_t v[kShare];
                        load_h<kShare>(tq + c0, v);
#pragma unroll
                        for (int c = 0; c < kShare; c += 4) {
                            uint32_t hi[2], lo[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                split(c0 + c + 2 * i < p.r, __uint_as_float(v[c + 2 * i]) * f, __uint_as_float(v[c + 2 * i + 1]) * f,
                                      hi[i], lo[i]);
                            uint8_t* d = hbuf + ((c0 + c) / 64) * kXBytes + piece(row, ((c0 + c) % 64) / 8) + (c0 + c) % 8 * 2;
                            ptx::shared_store8(ptx::smem_u32(d), hi[0], hi[1]);
                            ptx::shared_store8(ptx::smem_u32(d + S::kH), lo[0], lo[1]);
                        }
                    }
                    ptx::tc_fence_before();
                } else {
                    // each CTA's partial h, pieces of four columns; then CTA `rank` adds every cs-th row and
                    // writes it to all of the cluster
                    constexpr int kQuads = kR / 4, kMask = kQuads < 8 ? kQuads - 1 : 7;
                    if (live) {
                        uint32_t v[kShare];
                        if (k0 < k1) {
                            load_h<kShare>(tq + c0, v);
                        } else {
#pragma unroll
                            for (int c = 0; c < kShare; ++c) v[c] = 0u;
                        }
#pragma unroll
                        for (int c = 0; c < kShare; c += 4)
                            ptx::shared_store16(ptx::smem_u32(obuf) + (row * kQuads + (((c0 + c) / 4) ^ (row & kMask))) * 16,
                                                make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]));
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane < cs) ptx::cluster_arrive(ptx::cluster_addr(&st.p_ready, lane));
                    ok = all(ptx::mbar_wait_cluster(&st.p_ready, it & 1));
                    if (!ok) break;
                    const int n = t.rows > rank ? (t.rows - rank + cs - 1) / cs * kQuads : 0;
                    for (int u = ew * 32 + lane; u < n; u += kEpiWarps * 32) {
                        const int r = rank + u / kQuads * cs, c = u % kQuads * 4;
                        const uint8_t* at = obuf + (r * kQuads + ((c / 4) ^ (r & kMask))) * 16;
                        float4 h = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int o = 0; o < cs; ++o) {
                            const float4 v = ptx::cluster_load4(ptx::cluster_addr(at, o));
                            h.x += v.x, h.y += v.y, h.z += v.z, h.w += v.w;
                        }
                        uint32_t hi[2], lo[2];
                        split(c < p.r, h.x * f, h.y * f, hi[0], lo[0]);
                        split(c < p.r, h.z * f, h.w * f, hi[1], lo[1]);
                        const uint8_t* d = hbuf + (c / 64) * kXBytes + piece(r, (c % 64) / 8) + (c % 8) * 2;
                        for (int o = 0; o < cs; ++o) {
                            ptx::cluster_store2(ptx::cluster_addr(d, o), hi[0], hi[1]);
                            ptx::cluster_store2(ptx::cluster_addr(d + S::kH, o), lo[0], lo[1]);
                        }
                    }
                    ptx::fence_proxy_async();
                    __syncwarp();
                    if (lane < cs) ptx::cluster_arrive(ptx::cluster_addr(&st.p_done, lane));
                    ok = all(ptx::mbar_wait_cluster(&st.p_done, it & 1));
                    if (!ok) break;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&st.h_ready);
                ++it;
            }
            for (int nc = n0; nc < n1; ++nc) {
                const bool mine = cc % kGroups == static_cast<uint32_t>(g);
                const uint32_t buf = cc % kBufs, par = (cc / kBufs) & 1;
                ++cc;
                if (mine) {
                    // a stage or accumulator of another group may be a phase ahead: only its own are waited for
                    ok = all(ptx::mbar_wait_near(&st.d2_full[buf], par)) && all(ptx::mbar_wait_near(&st.full[s], ph));
                    if (!ok) break;
                    if (live) {
                        // this lane's row: 64 sums, then with y 128 bytes of out (o[j]: piece j)
                        uint32_t v[64], o[8][4], seen = 0;
                        if (t.adapter >= 0) {
                            ptx::tc_fence_after();
#pragma unroll
                            for (int c = 0; c < 64; c += 16)
                                ptx::tmem_ld16(tq + kD2Col + buf * 64 + c, *reinterpret_cast<uint32_t(*)[16]>(v + c));
                            ptx::tmem_ld_wait();
                            ptx::tc_fence_before();
                        } else {
#pragma unroll
                            for (int c = 0; c < 64; ++c) v[c] = 0x80000000u;  // -0: what leaves y's sign of zero as it is
                        }
                        const uint32_t yb = ptx::smem_u32(smem) + s * S::kStage;
                        uint4 y[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = ptx::shared_load16(yb + piece(row, j));
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t yy[4] = {y[j].x, y[j].y, y[j].z, y[j].w};
                            seen |= yy[0] | yy[1] | yy[2] | yy[3];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o[j][i] = pack_bf16x2(bf16_to_f32(yy[i] & 0xFFFFu) + __uint_as_float(v[j * 8 + 2 * i]),
                                                      bf16_to_f32(yy[i] >> 16) + __uint_as_float(v[j * 8 + 2 * i + 1]));
                        }
                        // y has to be in all lanes' registers before the stage goes back, or its next fill may be read: the
                        // arrival's address takes a zero from the loaded values, one that the compiler cannot know. (A fence
                        // would wait for the rows that were stored a slice ago, too.) Without it, 1 % of runs had 16-byte
                        // pieces of the stage's next fill.
                        const uint32_t zero = __reduce_or_sync(0xFFFFFFFFu, seen) & static_cast<uint32_t>(p.zero);
                        if (lane == 0) {
                            ptx::mbar_arrive(&st.empty[s + zero]);
                            ptx::mbar_arrive(&st.d2_empty[buf]);
                        }
                        // through this warp's buffer, so that a store instruction writes four rows of 128 bytes
#pragma unroll
                        for (int j = 0; j < 8; ++j) ptx::shared_store16(ob + piece(lane, j), make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]));
                        __syncwarp();
                        const int col = nc * 64 + (lane & 7) * 8, r0 = lane >> 3;
                        uint16_t* dst = p.out + (t.row + q * 32 + r0) * p.ld_out + col;
                        const uint32_t src = piece(r0, lane & 7);  // rows r0 + 4 i: every other one swaps halves of 64 bytes
                        const int left = col < p.N ? t.rows - q * 32 - r0 : 0;
                        uint4 w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = ptx::shared_load16(ob + i * 512 + (src ^ ((i & 1) * 64)));
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i * 4 < left) *reinterpret_cast<uint4*>(dst + i * 4 * p.ld_out) = w[i];
                        __syncwarp();
                    } else if (lane == 0) {
                        ptx::mbar_arrive(&st.empty[s]);
                        ptx::mbar_arrive(&st.d2_empty[buf]);
                    }
                }
                if (++s == kStages) { s = 0; ph ^= 1; }
            }
            if (lane == 0) ptx::mbar_arrive(&st.idle);
        }
        if (!ok) fail();
        if (check) report(p, walk);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        ptx::tmem_dealloc(tmem, kTmemCols);
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

template <int kR, int kRows>
cudaError_t launch_rows(const AdapterArgs& a, int cs, int64_t tiles, int sms, cudaStream_t stream)
{
    static bool attr_set = false;
    if (!attr_set) {
        cudaError_t e = cudaFuncSetAttribute(k_adapter_add<kR, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem_bytes<kR, kRows>()));
        if (e != cudaSuccess) return e;
        attr_set = true;
    }
    CUtensorMap x8, x32, x, y8, y32, y, ma, mb;
    if (map_rows(&x8, a.x, a.K, a.T, a.ld_x, 8) != CUDA_SUCCESS || map_rows(&x32, a.x, a.K, a.T, a.ld_x, 32) != CUDA_SUCCESS ||
        map_rows(&x, a.x, a.K, a.T, a.ld_x, kRows) != CUDA_SUCCESS || map_rows(&y, a.y, a.N, a.T, a.ld_y, kRows) != CUDA_SUCCESS ||
        map_rows(&y8, a.y, a.N, a.T, a.ld_y, 8) != CUDA_SUCCESS || map_rows(&y32, a.y, a.N, a.T, a.ld_y, 32) != CUDA_SUCCESS ||
        map_bank(&ma, a.a, a.K, a.r, a.n, kR) != CUDA_SUCCESS || map_bank(&mb, a.b, a.r, a.N, a.n, 64) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const int clusters = static_cast<int>(tiles * cs <= sms ? tiles : sms / cs);

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * cs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<kR, kRows>();
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_adapter_add<kR, kRows>, a, x8, x32, x, y8, y32, y, ma, mb);
}

template <int kR>
cudaError_t launch(const AdapterArgs& a, int cs, bool short_tiles, int sms, cudaStream_t stream)
{
    return short_tiles ? launch_rows<kR, 64>(a, cs, adapter_tiles(a, 64), sms, stream)
                       : launch_rows<kR, kTileM>(a, cs, adapter_tiles(a, kTileM), sms, stream);
}

}  // namespace

cudaError_t launch_adapter_add(const AdapterArgs& a, int sms, cudaStream_t stream)
{
    if (a.T <= 0) return cudaSuccess;
    // CTAs a tile of 128 rows: what fills the multiprocessors once. Clusters of eight need free multiprocessors
    // side by side (20 of them took 18.2 us where 20 clusters of four took 11.3); a batch hardly ever has all
    // the tiles that it could have, so a tenth more clusters of two are allowed.
    const int64_t tiles = adapter_tiles(a, kTileM);
    const int cs = tiles * 16 <= 2LL * (sms - sms / 8) ? 8 : tiles * 4 <= sms ? 4 : tiles * 20 <= 11LL * sms ? 2 : 1;
    // Estimated times in ns, from sweeps over 1 to 16,384 tokens of 1 to 256 requests, ranks 16 and 64, K x N
    // 2048 x 2048 and 512 x 1024 on 152 multiprocessors. Tiles of 8 rows: 4 us, 5 ns a tile and 105 ns a MB of
    // A and B (of padded rank) that the tiles read (256 single tokens, rank 64: 17.8 us against 36.9 with tiles
    // of 128; 4,113 tokens of 77 requests, rank 40: 30 against 17.0). Tiles of 128: the chain of one tile,
    // shorter the more CTAs share it, times the rounds of CTAs (4,113 tokens of 16 requests, rank 64: 18.4 us
    // against 33; 16,384 of 24: 38 against 130).
    const int64_t tiles8 = adapter_tiles(a, 8), width = a.K + a.N, padded = a.r <= 16 ? 16 : a.r <= 32 ? 32 : a.r <= 64 ? 64 : 128;
    const int64_t t8 = 4000 + tiles8 * (5 + 2 * padded * width / 9500);
    const int64_t chain = (cs == 8 ? 6500 : 8000) + width * (cs >= 4 ? 9 : cs == 2 ? 19 : 36) / 10 + 30 * a.r;
    // Tiles of 64 rows where one CTA a tile takes them in one round (4,113 tokens of 77 requests, rank 40: 17.0 us
    // against 23.4; 6,000 of 50, rank 64: 25.6 against 28.7; 10,000 of 20 need two rounds: 47.0 against 31.5).
    const bool short_tiles = cs == 1 && adapter_tiles(a, 64) <= sms + sms / 32;
    const int64_t ctas = 10 * tiles * cs, round = 11LL * sms;
    if (t8 <= (ctas <= round ? chain : chain * ctas / round)) return launch_adapter_add_small(a, sms, stream);
    if (a.r <= 16) return launch<16>(a, cs, short_tiles, sms, stream);
    if (a.r <= 32) return launch<32>(a, cs, short_tiles, sms, stream);
    if (a.r <= 64) return launch<64>(a, cs, short_tiles, sms, stream);
    return launch<128>(a, cs, short_tiles, sms, stream);
}

}  // namespace moe
