// adapters.cuh -- what the two adapter kernels share: the tiles of the requests and the two-value form
// of A x.
#pragma once
#include "block.cuh"
#include "ptx_cluster.cuh"

namespace moe {

// A request of L rows has ceil(L / rows) tiles of up to `rows` rows: at most this many in all.
inline int64_t adapter_tiles(const AdapterArgs& a, int rows) { return static_cast<int64_t>(a.T / rows) + (a.S < a.T ? a.S : a.T); }

// Tiles of up to rows (8 or 32) rows on mma.sync (adapters_small.cu).
cudaError_t launch_adapter_add_small(const AdapterArgs& a, int rows, int cs, int sms, cudaStream_t stream);

namespace adapters {

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
                // through warp reductions, whose results are uniform to the compiler: the addresses and loop
                // bounds that the issuing warps make of them then need no moves to uniform registers
                const bool me = lane == at;
                const int row = beg + (number - (before + sum - n)) * tile_rows;
                t.adapter = __reduce_max_sync(0xFFFFFFFFu, me ? ad : -1);
                t.row = __reduce_max_sync(0xFFFFFFFFu, me ? row : 0);
                t.rows = __reduce_max_sync(0xFFFFFFFFu, me ? min(tile_rows, end - row) : 0);
                return true;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        return false;
    }
};

// One warp: whether the requests follow the rules (in order, without gaps, adapters in range).
__device__ __forceinline__ void check_segments(const AdapterArgs& p)
{
    const int lane = threadIdx.x & 31;
    bool bad = __ldg(p.seg_offsets) != 0 || __ldg(p.seg_offsets + p.S) != p.T;
    for (int i = lane; i < p.S; i += 32) {
        const int beg = __ldg(p.seg_offsets + i), end = __ldg(p.seg_offsets + i + 1), ad = __ldg(p.seg_adapter + i);
        bad |= beg < 0 || beg > end || end > p.T || ad < -1 || ad >= p.n;
    }
    if (bad) record_status(p.status, kDevBadSegment);
}

// Two FP32 values (or zeros) as hi + lo, each two bf16: hi the nearest, lo the nearest to what is left.
__device__ __forceinline__ void split(bool in, float u, float v, uint32_t& hi, uint32_t& lo)
{
    if (!in) u = v = 0.0f;  // a padded column stays zero where x is not finite, too
    hi = pack_bf16x2(u, v);
    const float uh = bf16_to_f32(hi & 0xFFFFu), vh = bf16_to_f32(hi >> 16);
    // an infinity has no remainder
    lo = pack_bf16x2(fabsf(uh) < INFINITY ? u - uh : 0.0f, fabsf(vh) < INFINITY ? v - vh : 0.0f);
}

}  // namespace adapters
}  // namespace moe
