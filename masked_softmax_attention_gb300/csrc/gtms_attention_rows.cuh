// gtms_attention_rows.cuh -- attention's backward pass, a warp per row.
//
// A warp owns one query row (or, for dk and dv, one key row), each lane D / 32
// of its elements, and walks over the row's kept entries: a dot product across
// the lanes, then the probability from the saved lse, everything in fp32. Nothing is shared between rows, so every masked entry is simply not
// visited. Bound by the shuffles of the dot products.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gtms_attention.h"
#include "gtms_kernels.cuh"

namespace gtms {

constexpr int kRowsThreads = 128;

template <typename T, int D>
struct RowVec {
    static constexpr int N = D / 32;
    float e[N];
    __device__ __forceinline__ void load(const T* p, int lane)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            e[i] = static_cast<float>(p[lane * N + i]);
    }
    __device__ __forceinline__ void store(T* p, int lane, float scale) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            p[lane * N + i] = static_cast<T>(e[i] * scale + 0.0f);   // a zero comes out as +0.0
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            e[i] = 0.0f;
    }
    __device__ __forceinline__ void scale_add(float f, float w, const RowVec& x)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            e[i] = e[i] * f + w * x.e[i];
    }
    __device__ __forceinline__ float dot(const RowVec& x) const
    {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            v += e[i] * x.e[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
};

// dq, and D_i for the key rows.
template <typename T, int D>
__global__ void __launch_bounds__(kRowsThreads)
gtms_attention_rows_dq_kernel(const AttentionArgs a)
{
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t bh = w / a.Sq;
    const int32_t i = static_cast<int32_t>(w - bh * a.Sq), b = static_cast<int32_t>(bh / a.Hq), h = static_cast<int32_t>(bh % a.Hq);
    if (b >= a.B)
        return;
    int32_t c0, c1;
    a.kept(a.offset(b) + i, a.length(b), c0, c1);
    RowVec<T, D> q, dout, dq, k, v;
    dq.zero();
    float lse = 0.0f, delta = 0.0f;
    if (c0 < c1) {
        q.load(a.q.row<T>(b, h, i), lane);
        dout.load(a.dout.row<T>(b, h, i), lane);
        v.load(a.o.row<T>(b, h, i), lane);
        delta = dout.dot(v);
        lse = a.lse[w];
    }
    if (lane == 0)
        a.delta[w] = delta;
    for (int32_t c = c0; c < c1; ++c) {
        k.load(a.k.row<T>(b, h / a.group, c), lane);
        v.load(a.v.row<T>(b, h / a.group, c), lane);
        dq.scale_add(1.0f, expf(q.dot(k) * a.scale - lse) * (dout.dot(v) - delta), k);
    }
    dq.store(a.dq.row<T>(b, h, i), lane, a.scale);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowsThreads)
gtms_attention_rows_dkv_kernel(const AttentionArgs a)
{
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int64_t bh = w / a.Skv;
    const int32_t c = static_cast<int32_t>(w - bh * a.Skv), b = static_cast<int32_t>(bh / a.Hkv), g = static_cast<int32_t>(bh % a.Hkv);
    if (b >= a.B)
        return;
    const int32_t L = a.length(b), off = a.offset(b);
    RowVec<T, D> k, v, dk, dv, q, dout;
    dk.zero();
    dv.zero();
    if (c < L) {
        k.load(a.k.row<T>(b, g, c), lane);
        v.load(a.v.row<T>(b, g, c), lane);
        for (int32_t h = g * a.group; h < (g + 1) * a.group; ++h)
            for (int32_t i = 0; i < a.Sq; ++i) {
                int32_t c0, c1;
                a.kept(off + i, L, c0, c1);
                if (c < c0 || c >= c1)
                    continue;
                const int64_t r = (static_cast<int64_t>(b) * a.Hq + h) * a.Sq + i;
                q.load(a.q.row<T>(b, h, i), lane);
                dout.load(a.dout.row<T>(b, h, i), lane);
                const float p = expf(q.dot(k) * a.scale - a.lse[r]);
                dv.scale_add(1.0f, p, dout);
                dk.scale_add(1.0f, p * (dout.dot(v) - a.delta[r]), q);
            }
    }
    dk.store(a.dk.row<T>(b, g, c), lane, a.scale);
    dv.store(a.dv.row<T>(b, g, c), lane, 1.0f);
}

inline unsigned rows_grid(int64_t rows) { return static_cast<unsigned>((rows + kRowsThreads / 32 - 1) / (kRowsThreads / 32)); }

}  // namespace gtms
