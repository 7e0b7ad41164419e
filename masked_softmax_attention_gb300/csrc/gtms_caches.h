// gtms_caches.h -- what the launches on key/value caches share: their arguments
// (shared prefixes, key weights, eviction) and the launch functions.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gtms_attention.h"

namespace gtms {

// Multiprocessors of the chip, for choices that size a workspace and so must not
// depend on a device being there.
constexpr int kChipSms = 152;

// k_out[j] = k[kept[j]] and so on for every (batch, head), kept ascending.
struct EvictArgs {
    HeadsRef in[2], out[2];       // k and v
    const float* weights;         // [B, H, S]
    float* weights_out;           // [B, H, S_out]
    const int32_t* positions;     // [B, H, S], or null: 0, 1, ...
    int32_t* positions_out;       // [B, H, S_out], or null
    const int32_t* seq_lens;
    int32_t* lens_out;
    int32_t* kept;                // workspace [B, H, keep]: indices, written where a sequence is longer than keep
    int32_t B, H, S, S_out, keep, first, recent;
    int32_t units;                // 16-byte units of a row
    int32_t moved;                // bits 0 to 2: k, v, weights and positions go elsewhere (otherwise they are compacted in place)

#ifdef __CUDACC__
    __device__ __forceinline__ int32_t length(int32_t b) const
    {
        const int32_t n = __ldg(seq_lens + b);
        return n < 0 ? 0 : (n > S ? S : n);
    }
#endif
};

inline uint64_t evict_workspace_bytes(int64_t B, int64_t H, int64_t keep)
{
    return (static_cast<uint64_t>(B) * H * keep * 4 + 15) / 16 * 16;
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st);

// attention_key_weights: a.q, a.k, a.lse and what says which entries are kept, and
struct KeyWeightsArgs {
    AttentionArgs a;
    float* weights;               // [B, Hkv, Skv]
    float* parts;                 // workspace: partial sums, see key_weights_parts
    int32_t accumulate;
};

uint64_t key_weights_workspace_bytes(const AttentionArgs& a);
template <typename T, int D>
cudaError_t launch_key_weights(const KeyWeightsArgs& w, cudaStream_t st);

// attention_shared_prefix: AttentionArgs of the sequences' own keys, and the
// prefixes [G, Hkv, P, D], sequence b of n * G under prefix b / n.
struct PrefixArgs {
    HeadsRef k, v;
    const int32_t* lens;          // [G], or null: all P
    int32_t G, P, n;

#ifdef __CUDACC__
    __device__ __forceinline__ int32_t length(int32_t g) const
    {
        const int32_t L = lens ? __ldg(lens + g) : P;
        return L < 0 ? 0 : (L > P ? P : L);
    }
#endif
};

uint64_t shared_prefix_workspace_bytes(const AttentionArgs& a, const PrefixArgs& p, int64_t D);
template <typename T, int D>
cudaError_t launch_shared_prefix(const AttentionArgs& a, const PrefixArgs& p, void* workspace, cudaStream_t st);

}  // namespace gtms
