// gtms_key_weights_few.cuh -- the weight that each key of a cache received, for few
// query rows over many keys (new tokens over a cache).
//
//   w_c = sum over the query heads of a key/value head and rows i with c in K(i) of
//         exp(scale q_i . k_c - lse_i)
//
// What bounds it is one read of the live keys. The keys are the M side of the product:
// a warp takes 16 of them at a time straight from memory into the registers that the
// tensor-core instruction reads them from, the next 16 in flight while it works, and a
// thread's results belong to two keys, so that a key's sum takes two shuffles. The rows
// (of all heads that share the keys, 8 to an instruction) stand in shared memory. The
// terms are probabilities: no running maximum, no barrier, no exchange between warps.
//
// Operand layout, as in the split attention kernel: lane 4 g + t holds 16 contiguous
// bytes of key g (elements 32 x + 8 t .. + 7), the order of a dot product's terms being
// free, and reads a row's elements in the same order.
//
// One token of 64 sequences over caches of 8192 keys, 8 key/value heads of 128, added to
// what stands there: 89 us, 6.7 TB/s, the rate of a copy.
#pragma once

#include "gtms_attention_tc.cuh"
#include "gtms_caches.h"

namespace gtms {

constexpr int kFewWarps = 8, kFewThreads = 32 * kFewWarps;
constexpr int kFewChunk = 1024;   // keys of a CTA at most
// Where q's heads are broadcast rows are many, and sums long: of a power of two of row tiles at a time, and of those, so
// that a key's sum is off by half a step for each of 128 and of 1 / 128 of its tiles at most (2^21 rows: 2^-14 of it).
// One after the other those were 2^-11.6.
constexpr int64_t kFewTiles = 128;

template <int D, int NT>
struct FewShared {
    uint4 q[8 * NT][D / 8 + 1];                 // + 1: rows start in different banks
    float shift[8 * NT];                        // -lse in base 2; -infinity for rows that do not count
    int32_t lo[8 * NT], hi[8 * NT];             // keys that a row keeps
    float sum[kFewChunk], total[kFewChunk];     // of the last tiles; of those before
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kFewThreads, NT <= 2 ? 3 : 2)
gtms_key_weights_few_kernel(const KeyWeightsArgs kw, int32_t chunks, int32_t chunk)
{
    constexpr int R = 8 * NT;
    const AttentionArgs& a = kw.a;
    __shared__ FewShared<D, NT> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t bg = blockIdx.x / chunks;
    const int32_t b = static_cast<int32_t>(bg / a.Hkv), hk = static_cast<int32_t>(bg - static_cast<int64_t>(b) * a.Hkv);
    const int32_t off = a.offset(b), L = a.length(b);
    const int32_t k0 = static_cast<int32_t>(blockIdx.x % chunks) * chunk;
    const int32_t end = k0 + chunk < a.Skv ? k0 + chunk : a.Skv, k1 = end < L ? end : L;   // live keys [k0, k1)
    float* out = kw.weights + bg * a.Skv;

    // Rows [ia, ie) that keep any of these keys.
    int32_t ia = 0, ie = 0;
    if (k0 < k1) {
        ia = off < 0 ? -off : 0;
        ie = L - off < a.Sq ? L - off : a.Sq;
        if (a.mask_kind != GTMS_MASK_LENGTH && k0 - off > ia)
            ia = k0 - off;
        if (a.mask_kind == GTMS_MASK_SLIDING_WINDOW && k1 - 1 + a.window - off < ie)
            ie = k1 - 1 + a.window - off;
    }
    const int64_t rows = ia < ie ? static_cast<int64_t>(ie - ia) * a.group : 0;
    if (rows == 0) {
        if (!kw.accumulate)
            for (int32_t c = k0 + threadIdx.x; c < end; c += kFewThreads)
                out[c] = 0.0f;
        return;
    }
    for (int32_t c = threadIdx.x; c < chunk; c += kFewThreads)
        sh.sum[c] = sh.total[c] = 0.0f;

    const float c2 = a.scale * kLog2e;
    const T* kbase = a.k.row<T>(b, hk, 0) + 8 * t;
    for (int64_t r0 = 0; r0 < rows; r0 += R) {
        __syncthreads();   // the last rows have been used
        // Row r of the tile is query row ia + (r0 + r) / group of shared head (r0 + r) % group.
        for (int32_t i = threadIdx.x; i < R * (D / 8); i += kFewThreads) {
            const int32_t r = i / (D / 8), x = i % (D / 8);
            const int64_t n = r0 + r;
            sh.q[r][x] = n < rows ? *(reinterpret_cast<const uint4*>(a.q.row<T>(b, hk * a.group + n % a.group, ia + n / a.group)) + x)
                                  : make_uint4(0, 0, 0, 0);
        }
        if (threadIdx.x < R) {
            const int64_t n = r0 + threadIdx.x;
            int32_t c0 = 0, c1 = 0;
            float shift = -INFINITY;
            if (n < rows) {
                const int32_t i = ia + static_cast<int32_t>(n / a.group), h = hk * a.group + static_cast<int32_t>(n % a.group);
                a.kept(off + i, L, c0, c1);
                const float lse = a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Sq + i];
                shift = lse == -INFINITY ? -INFINITY : -lse * kLog2e;   // a row that kept nothing gives nothing
            }
            sh.shift[threadIdx.x] = shift;
            sh.lo[threadIdx.x] = c0;
            sh.hi[threadIdx.x] = c1;
        }
        __syncthreads();
        // Keys [f0, f1) that every row of the tile keeps (those past the last row keep nothing but count as nothing).
        int32_t f0 = 0, f1 = INT32_MAX;
#pragma unroll
        for (int32_t r = 0; r < R; r += 32)
            if (r + lane < R && r0 + r + lane < rows) {
                f0 = sh.lo[r + lane] > f0 ? sh.lo[r + lane] : f0;
                f1 = sh.hi[r + lane] < f1 ? sh.hi[r + lane] : f1;
            }
        f0 = __reduce_max_sync(0xffffffffu, f0);
        f1 = __reduce_min_sync(0xffffffffu, f1);

        const bool carry = r0 / R % kFewTiles == kFewTiles - 1;
        uint4 kr[2][D / 32];
        auto load = [&](int32_t key0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int32_t key = key0 + 8 * k + g;
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    kr[k][x] = load_once(kbase + key * a.k.ss + 32 * x, key < k1);
            }
        };
        int32_t key0 = k0 + 16 * warp;
        load(key0);
        for (; key0 < k1; key0 += 16 * kFewWarps) {
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[n][j] = 0.0f;
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 q = sh.q[8 * n + g][4 * x + t];
                    mma_16816<T>(s[n], kr[0][x].x, kr[1][x].x, kr[0][x].y, kr[1][x].y, q.x, q.y);
                    mma_16816<T>(s[n], kr[0][x].z, kr[1][x].z, kr[0][x].w, kr[1][x].w, q.z, q.w);
                }
            load(key0 + 16 * kFewWarps);
            const bool full = key0 >= f0 && key0 + 16 <= f1;
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 shift = *reinterpret_cast<const float2*>(&sh.shift[8 * n + 2 * t]);
                float e[4] = {exp2_approx(fmaf(s[n][0], c2, shift.x)), exp2_approx(fmaf(s[n][1], c2, shift.y)),
                              exp2_approx(fmaf(s[n][2], c2, shift.x)), exp2_approx(fmaf(s[n][3], c2, shift.y))};
                if (!full) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int32_t r = 8 * n + 2 * t + (j & 1), key = key0 + g + 8 * (j >> 1);
                        e[j] = key >= sh.lo[r] && key < sh.hi[r] ? e[j] : 0.0f;
                    }
                }
                sum[0] += e[0] + e[1];
                sum[1] += e[2] + e[3];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
                sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
                const int32_t key = key0 + g + 8 * k;
                if (t == 0 && key < k1) {   // this warp's keys alone
                    const float so_far = sh.sum[key - k0] + sum[k];
                    sh.sum[key - k0] = carry ? 0.0f : so_far;
                    if (carry)
                        sh.total[key - k0] += so_far;
                }
            }
        }
    }
    __syncthreads();
    if (kw.accumulate) {   // what stands behind the length is not this call's: another stream may be writing there
        for (int32_t c = k0 + threadIdx.x; c < k1; c += kFewThreads)
            out[c] += sh.total[c - k0] + sh.sum[c - k0];
    } else {
        for (int32_t c = k0 + threadIdx.x; c < end; c += kFewThreads)
            out[c] = c < k1 ? sh.total[c - k0] + sh.sum[c - k0] : 0.0f;
    }
}

template <typename T, int D, int NT>
cudaError_t launch_key_weights_few_n(const KeyWeightsArgs& kw, cudaStream_t st)
{
    const AttentionArgs& a = kw.a;
    const int64_t units = static_cast<int64_t>(a.B) * a.Hkv;
    // Keys of a CTA: fewer until there are four CTAs to a multiprocessor.
    int32_t chunk = kFewChunk;
    while (chunk > 16 * kFewWarps && units * ((a.Skv + chunk - 1) / chunk) < 4 * kChipSms)
        chunk /= 2;
    const int64_t chunks = (a.Skv + chunk - 1) / chunk;
    if (units * chunks > INT32_MAX)
        return cudaErrorNotSupported;
    return launch_kernel(gtms_key_weights_few_kernel<T, D, NT>, static_cast<unsigned>(units * chunks), kFewThreads, 0, st, kw,
                         static_cast<int32_t>(chunks), chunk);
}

template <typename T, int D>
cudaError_t launch_key_weights_few(const KeyWeightsArgs& kw, cudaStream_t st)
{
    const int64_t rows = static_cast<int64_t>(kw.a.group) * kw.a.Sq;
    return rows <= 8    ? launch_key_weights_few_n<T, D, 1>(kw, st)
           : rows <= 16 ? launch_key_weights_few_n<T, D, 2>(kw, st)
                        : launch_key_weights_few_n<T, D, 4>(kw, st);
}

}  // namespace gtms
