// gtms_attention_tc.cuh -- what the tensor-core attention kernels share: tensor
// maps of strided heads, the give-up protocol of their waits, tile loads.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gtms_attention.h"
#include "gtms_attn_tma.cuh"
#include "gtms_device.h"
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

// Makes the current device's context this thread's: the tensor-map encoder is a
// driver call, and a thread whose first CUDA call it is (autograd's, say) has none yet.
inline bool bind_context()
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

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

// Zeroes rows [from, to) of a swizzled 128-row tile of D / 64 boxes (a whole warp works).
template <int D>
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int32_t from, int32_t to, int lane)
{
    for (int32_t x = 0; x < D / 64; ++x)
        for (int32_t i = from * 8 + lane; i < to * 8; i += 32)   // 16-byte chunks, 8 to a row
            *reinterpret_cast<uint4*>(tile + x * kTile * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// The value of lane 0, for the compiler a warp's one value.
__device__ __forceinline__ int warp_value(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Work item of this CTA's round n: the items come costliest first, and every
// other round takes them the other way round, so that a CTA with a costly item
// in one round gets a cheap one in the next.
__device__ __forceinline__ int64_t snake_item(int64_t n)
{
    const int64_t g = gridDim.x, i = n & 1 ? g - 1 - blockIdx.x : blockIdx.x;
    return n * g + i;
}

// S (or dP) = A B^T: two K-major operands of 128 rows x D (a whole warp calls).
template <typename T, int D>
__device__ __forceinline__ void mma_abt(uint32_t d, uint32_t a, uint32_t b)
{
    constexpr uint32_t idesc = tc::idesc_f16<T>(kTile, kTile);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t at = (ks >> 2) * (kTile * 128) + (ks & 3) * 32;   // 16 columns of a swizzled 64-column box
        tc::mma_f16_warp(d, tc::smem_desc_sw128(a + at, 1024), tc::smem_desc_sw128(b + at, 1024), idesc, ks > 0);
    }
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
