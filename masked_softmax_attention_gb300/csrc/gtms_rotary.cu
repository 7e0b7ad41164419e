// gtms_rotary.cu -- rotary positions: pairs of a head's elements turned by
// angle = position * inv_freq (see gtms_rotary in include/gtms.h).
//
// The work is one read and one write of every element, so memory bounds it; the
// sine and cosine are the same for every head of a token, so a thread owns one
// 16-byte unit's pairs of one token, forms their rotations once and walks over
// heads with them. With few tokens the heads are split over more threads
// instead, which repeat the sines: there the launch's latency is the bound.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gtms_attention.h"
#include "gtms_kernels.cuh"

namespace gtms {
namespace {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// frequency / (2 pi) in turns, modulo one, as a 64-bit fixed-point fraction: the
// frequency's 24-bit mantissa times 1 / (2 pi) (64 significant bits), shifted by
// its exponent. Below 2^7 the fraction is off by less than 2^-57; the position
// multiplies that by at most 2^31.
__device__ __forceinline__ uint64_t turns_of(float frequency)
{
    constexpr uint64_t kInvTwoPi = 0xA2F9836E4E441529ull;   // floor(2^66 / (2 pi))
    const uint32_t bits = __float_as_uint(frequency);
    const int32_t e = static_cast<int32_t>((bits >> 23) & 0xFF);
    const uint64_t m = e ? (bits & 0x7FFFFFu) | 0x800000u : (bits & 0x7FFFFFu);
    const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
    const int32_t shift = 152 - (e ? e : 1);                // the product counts 2^-66 2^(e - 150), the fraction 2^-64
    uint64_t w = 0;
    if (shift <= 0)
        w = shift > -64 ? lo << -shift : 0;
    else if (shift < 64)
        w = (lo >> shift) | (hi << (64 - shift));
    else if (shift < 128)
        w = hi >> (shift - 64);
    return bits >> 31 ? 0 - w : w;
}

// cos and sin of position * frequency. The product is taken modulo one turn in
// 64-bit integers, exactly, so a far position loses nothing; what is left is
// rounded once to fp32, an error of at most 2^-25 half turns in the angle.
__device__ __forceinline__ void rotation(int32_t position, float frequency, float& c, float& s)
{
    const int64_t t = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(position)) * turns_of(frequency));
    const float poison = frequency * 0.0f;                  // NaN for a frequency that is no number
    sincospif(static_cast<float>(t) * 0x1p-63f + poison, &s, &c);
}

// VEC elements of one load: 16 bytes in the wide kernel, one element otherwise.
template <typename T, int VEC>
struct __align__(sizeof(T) * VEC) Unit {
    T e[VEC];
};

constexpr int kRotaryThreads = 128;
constexpr int kRotaryUnroll = 4;   // heads whose loads are in flight together

// Thread layout: unit fastest, then token, over x; y splits the heads. Units
// [0, n_rot) hold rotated pairs (VEC pairs from two places in the half layout,
// VEC / 2 neighbours in the interleaved one), the rest are copied.
template <typename T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads)
gtms_rotary_kernel(const RotaryArgs a, int32_t units, int32_t n_rot, int32_t heads_per_thread)
{
    using U = Unit<T, VEC>;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x;
    const int64_t token = idx / units;
    const int32_t unit = static_cast<int32_t>(idx - token * units);
    const int64_t b = token / a.S;
    const int32_t s = static_cast<int32_t>(token - b * a.S);
    if (b >= a.B)
        return;
    const int32_t heads = a.H[0] + a.H[1];
    const int32_t h0 = blockIdx.y * heads_per_thread;
    const int32_t h1 = h0 + heads_per_thread < heads ? h0 + heads_per_thread : heads;

    if (unit >= n_rot) {
        const int32_t at = a.R + (unit - n_rot) * VEC;
        for (int32_t h = h0; h < h1; ++h) {
            const int t = h >= a.H[0];
            const int32_t hh = t ? h - a.H[0] : h;
            *reinterpret_cast<U*>(a.y[t].row<T>(b, hh, s) + at) =
                *reinterpret_cast<const U*>(a.x[t].row<T>(b, hh, s) + at);
        }
        return;
    }

    constexpr int PAIRS = INTERLEAVED ? (VEC > 1 ? VEC / 2 : 1) : VEC;
    const int32_t pair0 = unit * PAIRS;
    float c[PAIRS], sn[PAIRS];
    const int32_t position = __ldg(a.positions + b * a.position_stride + s);
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
        rotation(position, __ldg(a.inv_freq + pair0 + i), c[i], sn[i]);
        c[i] *= a.amplitude;
        sn[i] *= a.inverse ? -a.amplitude : a.amplitude;
    }
    // Element offsets of the unit's two halves (the scalar interleaved kernel: a pair's two elements).
    const int32_t at1 = INTERLEAVED ? 2 * pair0 : pair0;
    const int32_t at2 = INTERLEAVED ? at1 + 1 : pair0 + a.R / 2;
    constexpr bool TWO = !INTERLEAVED || VEC == 1;   // the pairs' elements come from two units
    for (int32_t h = h0; h < h1; h += kRotaryUnroll) {
        U u[kRotaryUnroll], w[kRotaryUnroll];
#pragma unroll
        for (int k = 0; k < kRotaryUnroll; ++k)
            if (h + k < h1) {
                const int t = h + k >= a.H[0];
                const T* p = a.x[t].row<T>(b, t ? h + k - a.H[0] : h + k, s);
                u[k] = *reinterpret_cast<const U*>(p + at1);
                if constexpr (TWO)
                    w[k] = *reinterpret_cast<const U*>(p + at2);
            }
#pragma unroll
        for (int k = 0; k < kRotaryUnroll; ++k)
            if (h + k < h1) {
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    T& e1 = TWO ? u[k].e[i] : u[k].e[(2 * i) % VEC];
                    T& e2 = TWO ? w[k].e[i] : u[k].e[(2 * i + 1) % VEC];
                    const float x1 = to_float(e1), x2 = to_float(e2);
                    e1 = from_float<T>(x1 * c[i] - x2 * sn[i]);
                    e2 = from_float<T>(x2 * c[i] + x1 * sn[i]);
                }
                const int t = h + k >= a.H[0];
                T* p = a.y[t].row<T>(b, t ? h + k - a.H[0] : h + k, s);
                *reinterpret_cast<U*>(p + at1) = u[k];
                if constexpr (TWO)
                    *reinterpret_cast<U*>(p + at2) = w[k];
            }
    }
}

template <typename T, int VEC, bool INTERLEAVED>
cudaError_t launch(const RotaryArgs& a, cudaStream_t st)
{
    const int32_t pairs = INTERLEAVED ? (VEC > 1 ? VEC / 2 : 1) : VEC;
    const int32_t n_rot = a.R / 2 / pairs;
    const int32_t units = n_rot + (a.copy ? (a.D - a.R) / VEC : 0);
    if (units == 0)
        return cudaSuccess;   // in place, nothing rotated
    const int32_t heads = a.H[0] + a.H[1];
    const int64_t threads = static_cast<int64_t>(a.B) * a.S * units;
    const int64_t grid_x = (threads + kRotaryThreads - 1) / kRotaryThreads;
    if (grid_x > INT32_MAX)
        return cudaErrorNotSupported;
    int32_t per = heads;
    int32_t splits = (heads + per - 1) / per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid_x), static_cast<unsigned>(splits));
    cfg.blockDim = dim3(kRotaryThreads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, gtms_rotary_kernel<T, VEC, INTERLEAVED>, a, units, n_rot, per);
}

}  // namespace

template <typename T>
cudaError_t launch_rotary(const RotaryArgs& a, bool wide, cudaStream_t st)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    if (wide)
        return a.interleaved ? launch<T, V, true>(a, st) : launch<T, V, false>(a, st);
    return a.interleaved ? launch<T, 1, true>(a, st) : launch<T, 1, false>(a, st);
}

template cudaError_t launch_rotary<float>(const RotaryArgs&, bool, cudaStream_t);
template cudaError_t launch_rotary<__nv_bfloat16>(const RotaryArgs&, bool, cudaStream_t);
template cudaError_t launch_rotary<__half>(const RotaryArgs&, bool, cudaStream_t);

}  // namespace gtms
