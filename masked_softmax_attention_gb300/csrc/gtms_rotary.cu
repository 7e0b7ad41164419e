// gtms_rotary.cu -- rotary positions: pairs of a head's elements turned by
// angle = position * inv_freq (see gtms_rotary in include/gtms.h).
//
// The work is one read and one write of every element, so memory bounds it. The
// sine and cosine are the same for every head of a token: a block takes a few
// tokens and forms their rotations once, in shared memory; a thread then takes
// those of one 16-byte unit of one token into registers and walks over the heads.
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

// Blocks of 128 threads (six to a multiprocessor), four tokens each, two heads in
// flight per thread: of 128 to 512 threads, 2 to 5 heads and 2 to 8 tokens the
// best over the three measured sizes (q and k [4,40,4096,128] bf16 68 us, 4.9 TB/s;
// fewer, larger blocks hide less of the sines, more heads in flight cost occupancy).
constexpr int kRotaryThreads = 128;
constexpr int kRotaryUnroll = 2;      // heads whose loads are in flight together
constexpr int kRotaryBlocks = 6;
constexpr int kRotaryMaxTokens = 4;   // tokens of a block

// Units [0, n_rot) of a head hold rotated pairs (VEC pairs from two places in the
// half layout, VEC / 2 neighbours in the interleaved one), the rest are copied. A
// block takes 2^tokens_log tokens and heads_per_block heads; consecutive threads
// take the units of a token, then the tokens, then the heads.
template <typename T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads, kRotaryBlocks)
gtms_rotary_kernel(const RotaryArgs a, int32_t units, int32_t n_rot, int32_t tokens_log, int32_t heads_per_block)
{
    using U = Unit<T, VEC>;
    constexpr int PAIRS = INTERLEAVED ? (VEC > 1 ? VEC / 2 : 1) : VEC;
    constexpr bool TWO = !INTERLEAVED || VEC == 1;   // the pairs' elements come from two units
    extern __shared__ __align__(16) float2 turn[];   // [token][pair]: amplitude cos, amplitude sin
    __shared__ int64_t at[kRotaryMaxTokens][4];      // the token's offsets in x[0], y[0], x[1], y[1]
    const int32_t tokens = 1 << tokens_log, half = a.R / 2;
    const int64_t first = static_cast<int64_t>(blockIdx.x) << tokens_log, all = static_cast<int64_t>(a.B) * a.S;
    const int32_t live = all - first < tokens ? static_cast<int32_t>(all - first) : tokens;
    for (int32_t i = threadIdx.x; i < tokens * half; i += kRotaryThreads) {
        const int32_t k = i / half, j = i - k * half;
        if (k < live) {
            const int64_t b = (first + k) / a.S, s = first + k - b * a.S;
            float c, sn;
            rotation(__ldg(a.positions + b * a.position_stride + s), __ldg(a.inv_freq + j), c, sn);
            turn[i] = make_float2(c * a.amplitude, sn * (a.inverse ? -a.amplitude : a.amplitude));
        }
    }
    if (threadIdx.x < live) {
        const int64_t b = (first + threadIdx.x) / a.S, s = first + threadIdx.x - b * a.S;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            at[threadIdx.x][2 * k] = b * a.x[k].sb + s * a.x[k].ss;
            at[threadIdx.x][2 * k + 1] = b * a.y[k].sb + s * a.y[k].ss;
        }
    }
    __syncthreads();

    const int32_t heads = a.H[0] + a.H[1], h0 = blockIdx.y * heads_per_block;
    const int32_t h1 = h0 + heads_per_block < heads ? h0 + heads_per_block : heads;
    // A thread keeps one unit of one token, its rotations in registers, and walks over the heads.
    const int32_t places = units << tokens_log, lanes = places < kRotaryThreads ? kRotaryThreads / places : 1;
    const int32_t lane = threadIdx.x / places;
    if (lane >= lanes)
        return;
    for (int32_t place = threadIdx.x - lane * places; place < places; place += kRotaryThreads) {
        const int32_t k = place / units, unit = place - k * units;
        if (k >= live)
            break;
        const bool turned = unit < n_rot;
        const int32_t e = turned ? (INTERLEAVED ? 2 * PAIRS : PAIRS) * unit : a.R + (unit - n_rot) * VEC;
        float2 r[PAIRS];
        if (turned) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                r[i] = turn[k * half + unit * PAIRS + i];
        }
        const int32_t gap = INTERLEAVED ? 1 : half;   // from a pair's first element to its second
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // The block's heads of x[t].
            const int32_t before = t ? a.H[0] : 0;
            const int32_t last = h1 - before < a.H[t] ? h1 - before : a.H[t];
            int32_t h = (h0 > before ? h0 - before : 0) + lane;
            const int64_t in_step = lanes * a.x[t].sh, out_step = lanes * a.y[t].sh;
            const T* in = static_cast<const T*>(a.x[t].data) + at[k][2 * t] + h * a.x[t].sh + e;
            T* out = static_cast<T*>(a.y[t].data) + at[k][2 * t + 1] + h * a.y[t].sh + e;
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
    // Four tokens to a block; fewer, and then fewer heads, where that leaves multiprocessors without work.
    const int32_t heads = a.H[0] + a.H[1];
    const int64_t tokens = static_cast<int64_t>(a.B) * a.S;
    int32_t tokens_log = 2, splits = 1;
    while (tokens_log > 0 && ((tokens - 1) >> tokens_log) + 1 < 4 * nsm)
        --tokens_log;
    const int64_t grid_x = ((tokens - 1) >> tokens_log) + 1;
    while (grid_x * splits < nsm && (heads / splits) * units > kRotaryThreads)
        splits *= 2;
    if (grid_x > INT32_MAX)
        return cudaErrorNotSupported;
    const int32_t per = (heads + splits - 1) / splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid_x), static_cast<unsigned>((heads + per - 1) / per));
    cfg.blockDim = dim3(kRotaryThreads);
    cfg.dynamicSmemBytes = (static_cast<size_t>(a.R / 2) << tokens_log) * sizeof(float2);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, gtms_rotary_kernel<T, VEC, INTERLEAVED>, a, units, n_rot, tokens_log, per);
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
