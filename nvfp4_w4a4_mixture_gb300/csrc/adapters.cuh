// adapters.cuh -- what the two adapter kernels share: the tiles of the requests and the two-value form
// of A x.
#pragma once
#include "block.cuh"
#include "ptx_cluster.cuh"

namespace moe {

// A request of L rows has ceil(L / rows) tiles of up to `rows` rows: at most this many in all.
__host__ __device__ inline int64_t adapter_tiles(const AdapterArgs& a, int rows) { return static_cast<int64_t>(a.T / rows) + (a.S < a.T ? a.S : a.T); }

// Tiles of up to 8 rows on mma.sync (adapters_small.cu).
cudaError_t launch_adapter_add_small(const AdapterArgs& a, int sms, cudaStream_t stream);

namespace adapters {

struct Tile {
    int row, rows, adapter;  // adapter -1: copy
};

// Walks the requests in order, 128 at a time (four neighbours a lane); every warp that needs the tiles
// has its own. kRows: the rows of a full tile.
template <int kRows>
struct Walk {
    int base = 0, before = 0;  // first request of the window, tiles before it
    bool bad = false;          // this lane has met a request that breaks the rules (where it looks for them)

    // Warp-wide. The tile of the given number (numbers must not go down), false past the last.
    __device__ bool find(const AdapterArgs& p, int number, Tile& t, bool check = false)
    {
        if (number >= adapter_tiles(p, kRows)) return false;
        const int lane = threadIdx.x & 31;
        for (; base < p.S; base += 128) {
            const int s = base + lane * 4;
            int off[5], ad[4], n[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 5; ++i) off[i] = s + i <= p.S ? __ldg(p.seg_offsets + s + i) : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) ad[i] = s + i < p.S ? __ldg(p.seg_adapter + s + i) : -2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool good = off[i] >= 0 && off[i] <= off[i + 1] && off[i + 1] <= p.T && ad[i] >= -1 && ad[i] < p.n;
                n[i] = good && !(ad[i] < 0 && p.out == p.y) ? static_cast<int>((static_cast<unsigned>(off[i + 1] - off[i]) + kRows - 1) / kRows) : 0;
                sum += n[i];
            }
            if (check) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    bad |= s + i < p.S && (off[i] < 0 || off[i] > off[i + 1] || ad[i] < -1 || ad[i] >= p.n || (s + i == 0 && off[i] != 0) ||
                                           (s + i + 1 == p.S && off[i + 1] != p.T));
            }
            const int mine = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + sum > number);
            if (hit) {
                int left = number - (before + sum - mine), row = 0, rows = 0, adapter = -1;
                if (lane == __ffs(hit) - 1) {
                    bool found = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (!found && left >= 0 && left < n[i]) {
                            found = true;
                            adapter = ad[i];
                            row = off[i] + left * kRows;
                            rows = min(kRows, off[i + 1] - row);
                        }
                        left -= n[i];
                    }
                }
                // through warp reductions, whose results are uniform to the compiler: the addresses and loop
                // bounds that the issuing warps make of them then need no moves to uniform registers
                t.adapter = __reduce_max_sync(0xFFFFFFFFu, adapter);
                t.row = __reduce_max_sync(0xFFFFFFFFu, row);
                t.rows = __reduce_max_sync(0xFFFFFFFFu, rows);
                return true;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        return false;
    }
};

// One warp that has called find with `check`: reports whether the requests follow the rules (in order,
// without gaps, adapters in range). The first 128 are known from its first find.
template <int kRows>
__device__ __forceinline__ void report(const AdapterArgs& p, Walk<kRows>& w)
{
    for (int i = 128 + static_cast<int>(threadIdx.x & 31); i < p.S; i += 32) {
        const int beg = __ldg(p.seg_offsets + i), end = __ldg(p.seg_offsets + i + 1), ad = __ldg(p.seg_adapter + i);
        w.bad |= beg < 0 || beg > end || ad < -1 || ad >= p.n || (i + 1 == p.S && end != p.T);
    }
    if (w.bad) record_status(p.status, kDevBadSegment);
}

// Two FP32 values (or zeros) as hi + lo, each two bf16: hi the nearest, lo the nearest to what is left, which keeps 16
// significant bits or more (2^-17 of the value; the output's own rounding is 2^-8). One bf16 value would add an error
// of that size wherever the adapter's part dominates; a third would cost half as many products again for bits that
// the output does not hold. Against FP32 all through, one output in some 1,000 rounds to the neighbouring bf16.
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
