// gtms_attention_tc.cuh -- what the tensor-core attention kernels share: tensor
// maps of strided heads, the give-up protocol of their waits, tile loads.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gtms_attention.h"
#include "gtms_attn_tma.cuh"
#include "gtms_tcgen05.cuh"

namespace gtms {

constexpr int kTile = 128;   // rows and columns of one score tile

// A strided [B, H, S, D] tensor as a 4-D map (d, s, h, b) of 64-column boxes with
// the 128-byte swizzle. Rows past S read as zero. A broadcast dimension (stride 0)
// becomes an extent of one, and the kernels' coordinates along it are multiplied
// by 0 (mh, mb).
struct HeadsMap {
    CUtensorMap map;
    int32_t mh, mb;
};

template <typename T>
inline bool encode_heads(HeadsMap& m, const HeadsRef& t, int64_t B, int64_t H, int64_t S, int64_t D, uint32_t rows)
{
    const TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc)
        return false;
    m.mh = H > 1 && t.sh != 0;
    m.mb = B > 1 && t.sb != 0;
    // A stride that is never stepped over still has to be a legal one.
    const int64_t any = D;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(m.mh ? H : 1),
                                static_cast<cuuint64_t>(m.mb ? B : 1)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(S > 1 ? t.ss : any) * 2, static_cast<cuuint64_t>(m.mh ? t.sh : any) * 2,
                                   static_cast<cuuint64_t>(m.mb ? t.sb : any) * 2};
    const cuuint32_t box[4] = {64, rows, 1, 1}, estr[4] = {1, 1, 1, 1};
    return enc(&m.map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, t.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows row0 .. row0 + ROWS - 1 of head (h, b): D / 64 boxes of ROWS x 128 bytes.
template <int D, int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const HeadsMap& m, int32_t row0, int32_t h, int32_t b, uint64_t* bar)
{
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
        tc::tma_load_4d(dst + x * ROWS * 128, &m.map, x * 64, row0, h * m.mh, b * m.mb, bar);
}

// Every wait of these kernels is bounded: one that runs out raises the flag and
// the caller's status word, and every other role leaves its loop at the next wait
// that does not succeed at once.
struct GiveUp {
    int* flag;
    int32_t* status;
    uint64_t limit_ns;

    __device__ __forceinline__ bool raised() const { return *reinterpret_cast<const volatile int*>(flag) != 0; }
    __device__ __forceinline__ void raise() const
    {
        *reinterpret_cast<volatile int*>(flag) = 1;
        if (status)
            atomicOr(status, GTMS_ERR_TIMEOUT);
    }
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const
    {
        if (tc::mbar_try_wait(bar, parity))
            return true;
        const uint64_t t0 = tc::globaltimer_ns();
        for (;;) {
            if (tc::mbar_try_wait(bar, parity))
                return true;
            if (raised())
                return false;
            if (tc::globaltimer_ns() - t0 >= limit_ns) {
                raise();
                return false;
            }
        }
    }
    // All 32 lanes wait; the verdict is the warp's, so that warp-collective
    // instructions that follow stay converged.
    __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    }
};

// Zeroes rows [from, 128) of a swizzled tile of D / 64 boxes (a whole warp works).
template <int D>
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int32_t from, int lane)
{
    const int32_t per_box = (kTile - from) * 8;   // 16-byte chunks
    for (int32_t x = 0; x < D / 64; ++x)
        for (int32_t i = lane; i < per_box; i += 32)
            *reinterpret_cast<uint4*>(tile + x * kTile * 128 + from * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace gtms
