// gtms_attention.cu -- the attention forward and backward launches.
#include "gtms_attention_fwd.cuh"
#include "gtms_attention_rows.cuh"

namespace gtms {

template <typename T, int D>
cudaError_t launch_attention_forward(const AttentionArgs& a, cudaStream_t st)
{
    return launch_attention_fwd_tc<T, D>(a, st);
}

template <typename T, int D>
cudaError_t launch_attention_backward(const AttentionArgs& a, cudaStream_t st)
{
    cudaError_t e = cudaSuccess;
    if (a.Sq > 0)
        e = launch_kernel(gtms_attention_rows_dq_kernel<T, D>, rows_grid(static_cast<int64_t>(a.B) * a.Hq * a.Sq),
                          kRowsThreads, 0, st, a);
    if (e == cudaSuccess && a.Skv > 0)
        e = launch_kernel(gtms_attention_rows_dkv_kernel<T, D>, rows_grid(static_cast<int64_t>(a.B) * a.Hkv * a.Skv),
                          kRowsThreads, 0, st, a);
    return e;
}

#define GTMS_ATTENTION(T, D)                                                             \
    template cudaError_t launch_attention_forward<T, D>(const AttentionArgs&, cudaStream_t);   \
    template cudaError_t launch_attention_backward<T, D>(const AttentionArgs&, cudaStream_t);
GTMS_ATTENTION(__nv_bfloat16, 64)
GTMS_ATTENTION(__nv_bfloat16, 128)
GTMS_ATTENTION(__half, 64)
GTMS_ATTENTION(__half, 128)

}  // namespace gtms
