// gtms_key_weights.cu -- the key-weight launches.
#include "gtms_key_weights_few.cuh"
#include "gtms_key_weights_tc.cuh"

namespace gtms {
namespace {

// Rows of a key/value head up to which the keys go straight to registers.
constexpr int64_t kFewRows = 32;

bool few(const AttentionArgs& a) { return static_cast<int64_t>(a.group) * a.Sq <= kFewRows; }

// Whether a map of q holds its heads: one that serves all (stride 0), or ones 2^40 bytes apart, it does not.
bool mapped(const AttentionArgs& a)
{
    return a.Hq == 1 || (a.q.sh > 0 && a.q.sh < (int64_t(1) << 39) / a.group);
}

}  // namespace

// By the shape alone, which does not say how q's heads stand: where they are broadcast the workspace is not used.
uint64_t key_weights_workspace_bytes(const AttentionArgs& a)
{
    const int32_t parts = few(a) ? 1 : key_plan(a).parts;
    return parts > 1 ? static_cast<uint64_t>(parts) * a.B * a.Hkv * a.Skv * 4 : 0;
}

template <typename T, int D>
cudaError_t launch_key_weights(const KeyWeightsArgs& w, cudaStream_t st)
{
    return few(w.a) || !mapped(w.a) ? launch_key_weights_few<T, D>(w, st) : launch_key_weights_tc<T, D>(w, st);
}

#define GTMS_KEY_WEIGHTS(T, D) template cudaError_t launch_key_weights<T, D>(const KeyWeightsArgs&, cudaStream_t);
GTMS_KEY_WEIGHTS(__nv_bfloat16, 64)
GTMS_KEY_WEIGHTS(__nv_bfloat16, 128)
GTMS_KEY_WEIGHTS(__half, 64)
GTMS_KEY_WEIGHTS(__half, 128)

}  // namespace gtms
