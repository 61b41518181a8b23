// block.cuh -- internal launchers of the operators around the expert layer: norms with gate and
// residual, expert selection from given logits, and low-rank adapters (not part of the C ABI).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "kernels.cuh"

namespace moe {

// Device status bits of moe_adapter_add (the workspace header's status word).
enum : int {
    kDevTimeoutAdapter = 16,  // a bounded wait of the adapter kernel ran out
    kDevBadSegment = 32,      // seg_offsets or seg_adapter outside its range
};

// ---- norm_residual.cu
struct NormArgs {
    int T, H;
    const uint16_t* y;        // nullable
    int64_t ld_y;
    const void* res;          // nullable
    int64_t ld_res;
    bool res_f32;             // residual and residual_out are FP32, else bf16
    const uint16_t* w_post;   // nullable
    const uint16_t* w_pre;    // null exactly when x_out is
    float eps, w_offset, res_scale;
    const void* gate;         // nullable
    bool gate_f32, gate_per_channel;
    int64_t gate_ld;
    void* res_out;            // nullable
    int64_t ld_res_out;
    uint16_t* x_out;          // nullable
    int64_t ld_x;
};
cudaError_t launch_norm_residual(const NormArgs& a, int sms, cudaStream_t stream);

// ---- select_experts.cu
struct SelectArgs {
    int T, E, k;
    bool sigmoid;
    int n_group, topk_group;
    bool group_top2, renormalize;
    float scale;
    const float* bias;        // nullable
    const void* logits;
    bool logits_f32;
    int64_t ld;
    int32_t* ids;
    float* w;
    // set by the launcher: experts a group, log2 of the lanes that take a group, and the multiplier with
    // which (e * group_of_mul) >> 21 is expert e's group
    int group_size, group_lanes_log2;
    unsigned group_of_mul;
};
cudaError_t launch_select_experts(const SelectArgs& a, cudaStream_t stream);

// ---- adapters.cu
constexpr int kAdapterMaxRank = 128;
struct AdapterArgs {
    int T, S, n, r, K, N;
    const uint16_t* a;        // [n][r][K]
    const uint16_t* b;        // [n][N][r]
    const float* scale;       // [n]
    const uint16_t* x;
    int64_t ld_x;
    const int32_t* seg_offsets;
    const int32_t* seg_adapter;
    const uint16_t* y;
    int64_t ld_y;
    uint16_t* out;
    int64_t ld_out;
    int* status;
    const WsHeader* hooks;    // the workspace header whose test_* fields a wait reads
    int zero;                 // 0, which kernels do not know
};
cudaError_t launch_adapter_add(const AdapterArgs& a, int sms, cudaStream_t stream);

}  // namespace moe
