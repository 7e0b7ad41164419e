// gtms_shared_prefix.cu -- the launches of attention over shared prefixes.
#include "gtms_shared_prefix.cuh"

namespace gtms {

extern template cudaError_t launch_attention_forward<__nv_bfloat16, 64>(const AttentionArgs&, cudaStream_t);
extern template cudaError_t launch_attention_forward<__nv_bfloat16, 128>(const AttentionArgs&, cudaStream_t);
extern template cudaError_t launch_attention_forward<__half, 64>(const AttentionArgs&, cudaStream_t);
extern template cudaError_t launch_attention_forward<__half, 128>(const AttentionArgs&, cudaStream_t);

namespace {

template <int D>
uint64_t workspace_bytes(const AttentionArgs& a, const PrefixArgs& p)
{
    const PackedPlan x = packed_plan<D>(a, p);
    return prefer_packed<D>(a, p, x) ? packed_bytes(a, p, x, D) : 0;
}

}  // namespace

uint64_t shared_prefix_workspace_bytes(const AttentionArgs& a, const PrefixArgs& p, int64_t D)
{
    return D == 64 ? workspace_bytes<64>(a, p) : workspace_bytes<128>(a, p);
}

template <typename T, int D>
cudaError_t launch_shared_prefix(const AttentionArgs& a, const PrefixArgs& p, void* workspace, cudaStream_t st)
{
    if (p.P == 0)
        return launch_attention_forward<T, D>(a, st);
    const PackedPlan x = packed_plan<D>(a, p);
    return prefer_packed<D>(a, p, x) ? launch_prefix_packed<T, D>(a, p, x, workspace, st) : launch_prefixed_whole<T, D>(a, p, st);
}

#define GTMS_SHARED_PREFIX(T, D) \
    template cudaError_t launch_shared_prefix<T, D>(const AttentionArgs&, const PrefixArgs&, void*, cudaStream_t);
GTMS_SHARED_PREFIX(__nv_bfloat16, 64)
GTMS_SHARED_PREFIX(__nv_bfloat16, 128)
GTMS_SHARED_PREFIX(__half, 64)
GTMS_SHARED_PREFIX(__half, 128)

}  // namespace gtms
