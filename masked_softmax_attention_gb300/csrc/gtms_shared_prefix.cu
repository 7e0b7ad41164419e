// gtms_shared_prefix.cu -- the launches of attention over shared prefixes.
#include "gtms_shared_prefix.cuh"

namespace gtms {

uint64_t shared_prefix_workspace_bytes(const AttentionArgs&, const PrefixArgs&, int64_t) { return 0; }

template <typename T, int D>
cudaError_t launch_shared_prefix(const AttentionArgs& a, const PrefixArgs& p, void*, cudaStream_t st)
{
    return launch_prefixed_whole<T, D>(a, p, st);
}

#define GTMS_SHARED_PREFIX(T, D) \
    template cudaError_t launch_shared_prefix<T, D>(const AttentionArgs&, const PrefixArgs&, void*, cudaStream_t);
GTMS_SHARED_PREFIX(__nv_bfloat16, 64)
GTMS_SHARED_PREFIX(__nv_bfloat16, 128)
GTMS_SHARED_PREFIX(__half, 64)
GTMS_SHARED_PREFIX(__half, 128)

}  // namespace gtms
