// gtms_key_weights.cu -- the key-weight launches.
#include "gtms_key_weights_few.cuh"

namespace gtms {

uint64_t key_weights_workspace_bytes(const AttentionArgs&) { return 0; }

template <typename T, int D>
cudaError_t launch_key_weights(const KeyWeightsArgs& w, cudaStream_t st)
{
    return launch_key_weights_few<T, D>(w, st);
}

#define GTMS_KEY_WEIGHTS(T, D) template cudaError_t launch_key_weights<T, D>(const KeyWeightsArgs&, cudaStream_t);
GTMS_KEY_WEIGHTS(__nv_bfloat16, 64)
GTMS_KEY_WEIGHTS(__nv_bfloat16, 128)
GTMS_KEY_WEIGHTS(__half, 64)
GTMS_KEY_WEIGHTS(__half, 128)

}  // namespace gtms
