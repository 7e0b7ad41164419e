// gtms_attention.h -- what the attention and rotary launches share: strided
// tensors and the kept set as the kernels see them, and the launch functions.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gtms.h"

namespace gtms {

// A strided [B, H, S, D] tensor on the device (strides in elements; 0 for a
// dimension of extent 1).
struct HeadsRef {
    void* data;
    int64_t sb, sh, ss;

    template <typename T>
    __host__ __device__ __forceinline__ T* row(int64_t b, int64_t h, int64_t s) const
    {
        return static_cast<T*>(data) + b * sb + h * sh + s * ss;
    }
};

// Offsets beyond this leave every row outside [0, L); the kernels clamp to it so
// that positions stay far inside 32 bits.
constexpr int32_t kMaxOffset = 1 << 25;
static_assert(kMaxOffset > GTMS_ATTENTION_MAX_S, "a clamped offset must leave no row alive");

struct AttentionArgs {
    HeadsRef q, k, v, o, dout, dq, dk, dv;
    float* lse;
    float *lse2, *delta, *norms;  // backward's workspace (see attention_workspace)
    int32_t Sq_pad, norm_blocks;
    const int32_t* seq_lens;
    const int32_t* q_offsets;
    int32_t* status;
    int32_t B, Hq, Hkv, group, Sq, Skv, window, mask_kind;
    float scale;

#ifdef __CUDACC__
    __device__ __forceinline__ int32_t length(int32_t b) const
    {
        const int32_t L = __ldg(seq_lens + b);
        return L < 0 ? 0 : (L > Skv ? Skv : L);
    }
    __device__ __forceinline__ int32_t offset(int32_t b) const
    {
        if (!q_offsets)
            return 0;
        const int32_t f = __ldg(q_offsets + b);
        return f < -kMaxOffset ? -kMaxOffset : (f > kMaxOffset ? kMaxOffset : f);
    }
    // Kept columns [c0, c1) of the row at position r.
    __device__ __forceinline__ void kept(int32_t r, int32_t L, int32_t& c0, int32_t& c1) const
    {
        c0 = c1 = 0;
        if (r >= 0 && r < L) {
            c1 = mask_kind == GTMS_MASK_LENGTH ? L : r + 1;
            if (mask_kind == GTMS_MASK_SLIDING_WINDOW && r - window + 1 > 0)
                c0 = r - window + 1;
        }
    }
#endif
};

// The backward's workspace: per query row, padded to whole tiles of 128, -lse in
// base 2 and -D; then the partial maxima of the norms of dout and v.
constexpr int64_t kWorkspaceNorms = 2 * 1024;

inline int64_t attention_padded_rows(int64_t B, int64_t Hq, int64_t Sq) { return B * Hq * ((Sq + 127) / 128 * 128); }
inline uint64_t attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Sq)
{
    return static_cast<uint64_t>(2 * attention_padded_rows(B, Hq, Sq) + kWorkspaceNorms) * 4;
}
inline void attention_workspace(AttentionArgs& a, void* workspace)
{
    a.Sq_pad = (a.Sq + 127) / 128 * 128;
    const int64_t rows = attention_padded_rows(a.B, a.Hq, a.Sq);
    a.lse2 = static_cast<float*>(workspace);
    a.delta = a.lse2 + rows;
    a.norms = a.delta + rows;
}

struct RotaryArgs {
    HeadsRef x[2], y[2];
    const int32_t* positions;
    int64_t position_stride;      // S, or 0 where one row serves every batch
    const float* inv_freq;
    int32_t B, H[2], S, D, R;
    float amplitude;
    int32_t interleaved, inverse, copy;   // copy: elements from R on go from x to y
};

template <typename T, int D>
cudaError_t launch_attention_forward(const AttentionArgs& a, cudaStream_t st);
template <typename T, int D>
cudaError_t launch_attention_backward(const AttentionArgs& a, cudaStream_t st);
template <typename T>
cudaError_t launch_rotary(const RotaryArgs& a, bool wide, cudaStream_t st);

}  // namespace gtms
