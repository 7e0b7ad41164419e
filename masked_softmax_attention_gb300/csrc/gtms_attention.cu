// gtms_attention.cu -- the attention forward and backward launches.
#include "gtms_attention_bwd.cuh"
#include "gtms_attention_fwd.cuh"
#include "gtms_attention_split.cuh"

namespace gtms {

template <typename T, int D>
cudaError_t launch_attention_forward(const AttentionArgs& a, cudaStream_t st)
{
    if (prefer_split<D>(a))
        return launch_attention_split<T, D>(a, st);
    return launch_attention_fwd_tc<T, D>(a, st);
}

template <typename T, int D>
cudaError_t launch_attention_backward(const AttentionArgs& a, cudaStream_t st)
{
    return launch_attention_bwd_tc<T, D>(a, st);
}

#define GTMS_ATTENTION(T, D)                                                             \
    template cudaError_t launch_attention_forward<T, D>(const AttentionArgs&, cudaStream_t);   \
    template cudaError_t launch_attention_backward<T, D>(const AttentionArgs&, cudaStream_t);
GTMS_ATTENTION(__nv_bfloat16, 64)
GTMS_ATTENTION(__nv_bfloat16, 128)
GTMS_ATTENTION(__half, 64)
GTMS_ATTENTION(__half, 128)

}  // namespace gtms
