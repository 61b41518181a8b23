// The attention kernels of a cache in e4m3 with heads of 128.
#include "paged_attention.cuh"

namespace moe {
namespace attention {

template cudaError_t launch_head_size<128, true>(const AttentionArgs&, int, cudaStream_t);

}  // namespace attention
}  // namespace moe
