// gtms_rotary.cu -- rotary positions: pairs of a head's elements turned by
// angle = position * inv_freq (see gtms_rotary in include/gtms.h).
//
// The work is one read and one write of every element, so memory bounds it. The
// sine and cosine are the same for every head of a token: a block takes one token,
// asks for its rows in L2, forms its rotations in shared memory meanwhile, and each
// thread then takes those of one 16-byte unit into registers and walks over the
// heads. q and k [4,40,4096,128] bf16: 52 us, 6.4 TB/s (70 without the L2 prefetch
// and with four tokens to a block of 128 threads).
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gtms_attention.h"
#include "gtms_device.h"
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

// 64 threads, 16 blocks to a multiprocessor, two heads in flight per thread: of 32 to
// 256 threads, 1 to 5 heads and 1 to 8 tokens the best at the size above (52 us;
// 128 threads 68, one head in flight 54, three 71, two tokens 60).
constexpr int kRotaryThreads = 64, kRotaryBlocks = 16;
constexpr int kRotaryUnroll = 2;      // heads whose loads are in flight together

// Units [0, n_rot) of a head hold rotated pairs (VEC pairs from two places in the
// half layout, VEC / 2 neighbours in the interleaved one), the rest are copied. A
// block takes one token and heads_per_block heads; consecutive threads take the
// units, then the heads.
template <typename T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads, kRotaryBlocks)
gtms_rotary_kernel(const RotaryArgs a, int32_t units, int32_t n_rot, int32_t heads_per_block)
{
    using U = Unit<T, VEC>;
    constexpr int PAIRS = INTERLEAVED ? (VEC > 1 ? VEC / 2 : 1) : VEC;
    constexpr bool TWO = !INTERLEAVED || VEC == 1;   // the pairs' elements come from two units
    extern __shared__ __align__(16) float2 turn[];   // [pair]: amplitude cos, amplitude sin
    const int32_t half = a.R / 2, heads = a.H[0] + a.H[1], h0 = blockIdx.y * heads_per_block;
    const int32_t h1 = h0 + heads_per_block < heads ? h0 + heads_per_block : heads;
    const int64_t b = blockIdx.x / a.S, s = blockIdx.x - b * a.S;
    auto row = [&](const HeadsRef& x, int32_t h) { return static_cast<T*>(x.data) + b * x.sb + s * x.ss + h * x.sh; };

    const int32_t lines = (a.D * static_cast<int32_t>(sizeof(T)) + 127) / 128;
    for (int32_t i = threadIdx.x; i < (h1 - h0) * lines; i += kRotaryThreads) {
        const int32_t n = i / lines, h = h0 + n, t = h >= a.H[0];
        const char* p = reinterpret_cast<const char*>(row(a.x[t], t ? h - a.H[0] : h)) + (i - n * lines) * 128;
        asm volatile("prefetch.global.L2 [%0];" :: "l"(p));
    }
    const int32_t position = __ldg(a.positions + b * a.position_stride + s);
    for (int32_t j = threadIdx.x; j < half; j += kRotaryThreads) {
        float c, sn;
        rotation(position, __ldg(a.inv_freq + j), c, sn);
        turn[j] = make_float2(c * a.amplitude, sn * (a.inverse ? -a.amplitude : a.amplitude));
    }
    __syncthreads();

    // A thread keeps one unit, its rotations in registers, and walks over the heads.
    const int32_t lanes = units < kRotaryThreads ? kRotaryThreads / units : 1, lane = threadIdx.x / units;
    if (lane >= lanes)
        return;
    for (int32_t unit = threadIdx.x - lane * units; unit < units; unit += kRotaryThreads) {
        const bool turned = unit < n_rot;
        const int32_t e = turned ? (INTERLEAVED ? 2 * PAIRS : PAIRS) * unit : a.R + (unit - n_rot) * VEC;
        float2 r[PAIRS];
        if (turned) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                r[i] = turn[unit * PAIRS + i];
        }
        const int32_t gap = INTERLEAVED ? 1 : half;   // from a pair's first element to its second
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // The block's heads of x[t].
            const int32_t before = t ? a.H[0] : 0;
            const int32_t last = h1 - before < a.H[t] ? h1 - before : a.H[t];
            int32_t h = (h0 > before ? h0 - before : 0) + lane;
            const int64_t in_step = lanes * a.x[t].sh, out_step = lanes * a.y[t].sh;
            const T* in = row(a.x[t], h) + e;
            T* out = row(a.y[t], h) + e;
            auto walk = [&](auto count) {   // `count` heads, their loads in flight together
                constexpr int N = decltype(count)::value;
                U u[N], w[N];
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    u[q] = *reinterpret_cast<const U*>(in + q * in_step);
                    if (TWO && turned)
                        w[q] = *reinterpret_cast<const U*>(in + q * in_step + gap);
                }
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    if (turned) {
#pragma unroll
                        for (int i = 0; i < PAIRS; ++i) {
                            T& e1 = TWO ? u[q].e[i] : u[q].e[(2 * i) % VEC];
                            T& e2 = TWO ? w[q].e[i] : u[q].e[(2 * i + 1) % VEC];
                            const float x1 = to_float(e1), x2 = to_float(e2);
                            e1 = from_float<T>(x1 * r[i].x - x2 * r[i].y);
                            e2 = from_float<T>(x2 * r[i].x + x1 * r[i].y);
                        }
                        if constexpr (TWO)
                            *reinterpret_cast<U*>(out + q * out_step + gap) = w[q];
                    }
                    *reinterpret_cast<U*>(out + q * out_step) = u[q];
                }
                in += N * in_step;
                out += N * out_step;
                h += N * lanes;
            };
            while (h + (kRotaryUnroll - 1) * lanes < last)
                walk(std::integral_constant<int, kRotaryUnroll>{});
            while (h < last)
                walk(std::integral_constant<int, 1>{});
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
    const int nsm = device_sms();
    if (nsm <= 0)
        return cudaErrorUnknown;
    // A block a token; where that leaves multiprocessors without work, the heads are split.
    const int32_t heads = a.H[0] + a.H[1];
    const int64_t tokens = static_cast<int64_t>(a.B) * a.S;
    int32_t splits = 1;
    while (tokens * splits < nsm && (heads / splits) * units > kRotaryThreads)
        splits *= 2;
    const int32_t per = (heads + splits - 1) / splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tokens), static_cast<unsigned>((heads + per - 1) / per));
    cfg.blockDim = dim3(kRotaryThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.R / 2) * sizeof(float2);
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
