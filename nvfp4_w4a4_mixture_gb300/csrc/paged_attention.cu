// paged_attention.cu -- moe_paged_attention's workspace and the choice of its kernels (paged_attention.cuh), which are
// compiled in a file for each type of cache and size of head.
#include <mutex>

#include "attention.cuh"

namespace moe {

namespace attention {

template <int kD, bool kE4M3>
cudaError_t launch_head_size(const AttentionArgs& a, int sms, cudaStream_t stream);

namespace {

template <bool kE4M3>
cudaError_t launch(const AttentionArgs& a, int sms, cudaStream_t stream)
{
    switch (a.c.D) {
    case 64: return launch_head_size<64, kE4M3>(a, sms, stream);
    case 128: return launch_head_size<128, kE4M3>(a, sms, stream);
    case 256: return launch_head_size<256, kE4M3>(a, sms, stream);
    default: return cudaErrorInvalidValue;
    }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// header, prefix, maxima and sums, partial outputs: two slots a CTA
size_t ml_at(int S) { return sizeof(WsHeader) + up256((static_cast<size_t>(S) + 3) * 8); }
size_t part_at(int S, int rows, int sms) { return ml_at(S) + up256(static_cast<size_t>(ctas_most(sms)) * 2 * rows * 8); }

}  // namespace
}  // namespace attention

size_t attention_workspace_bytes(int S, int n_q, int n_kv, int D, int max_new, int sms)
{
    const int rows = 8 * attention::row_eights(n_q / n_kv, max_new);
    return attention::part_at(S, rows, sms) + static_cast<size_t>(attention::ctas_most(sms)) * 2 * rows * D * 4;
}

cudaError_t launch_paged_attention(AttentionArgs a, void* ws, int sms, cudaStream_t stream)
{
    // Both launches of a call come one after the other: of two host threads that share a stream and a workspace, the join of
    // one would read the parts of the other.
    static std::mutex launches;
    std::lock_guard<std::mutex> lock(launches);
    char* const base = static_cast<char*>(ws);
    const int rows = 8 * attention::row_eights(a.group, a.max_new);
    a.prefix = reinterpret_cast<int64_t*>(base + sizeof(WsHeader));
    a.part_ml = reinterpret_cast<float*>(base + attention::ml_at(a.r.S));
    a.part = reinterpret_cast<float*>(base + attention::part_at(a.r.S, rows, sms));
    return a.c.e4m3 ? attention::launch<true>(a, sms, stream) : attention::launch<false>(a, sms, stream);
}

}  // namespace moe
