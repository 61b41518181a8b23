// The attention kernels of a cache in bf16 with heads of 64.
#include "paged_attention.cuh"

namespace moe {
namespace attention {

template cudaError_t launch_head_size<64, false>(const AttentionArgs&, int, cudaStream_t);

}  // namespace attention
}  // namespace moe
