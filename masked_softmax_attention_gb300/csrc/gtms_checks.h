// gtms_checks.h -- host-side argument checks that the entry points on strided
// heads share (attention, rotary positions, caches).
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "gtms.h"
#include "gtms_attention.h"
#include "gtms_heads.h"

#define GTMS_EXPORT extern "C" __attribute__((visibility("default")))

namespace gtms {

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int status_of(cudaError_t e)
{
    if (e == cudaSuccess)
        return GTMS_OK;
    cudaGetLastError();   // reported through the returned code
    return e == cudaErrorNotSupported ? GTMS_ERR_UNSUPPORTED : GTMS_ERR_CUDA;
}

inline HeadsRef device_ref(const gtms_heads& t, const HeadsSpan& s, int elem)
{
    return {t.data, s.stride[0] / elem, s.stride[1] / elem, s.stride[2] / elem};
}

// Sizes and options that both directions share; *rows = B * Hq * Sq.
inline int check_shape(const gtms_attention_shape* p, int64_t* rows)
{
    if (!p || p->B < 0 || p->Hq < 0 || p->Hkv < 0 || p->Sq < 0 || p->Skv < 0 || p->head_dim < 0 ||
        !std::isfinite(p->scale))
        return GTMS_ERR_INVALID_ARG;
    if ((p->Hq == 0) != (p->Hkv == 0) || (p->Hkv > 0 && p->Hq % p->Hkv != 0))
        return GTMS_ERR_INVALID_ARG;
    if (p->mask_kind < 0 || p->mask_kind > 2)
        return GTMS_ERR_UNSUPPORTED;
    if (p->mask_kind == GTMS_MASK_SLIDING_WINDOW && p->window < 1)
        return GTMS_ERR_INVALID_ARG;
    if ((p->dtype != GTMS_BF16 && p->dtype != GTMS_F16) || (p->head_dim != 64 && p->head_dim != 128) ||
        p->Sq > GTMS_ATTENTION_MAX_S || p->Skv > GTMS_ATTENTION_MAX_S)
        return GTMS_ERR_UNSUPPORTED;
    // Every launch has at most one CTA per (batch, head, row or key): keep that, and the
    // fp32 row statistics' byte count, inside a grid dimension and 64 bits.
    int64_t heads = 0, ctas = 0;
    const int64_t s = p->Sq > p->Skv ? p->Sq : p->Skv;
    if (__builtin_mul_overflow(p->B, p->Hq, &heads) || __builtin_mul_overflow(heads, (s + 63) / 64, &ctas) ||
        ctas > INT32_MAX)
        return GTMS_ERR_UNSUPPORTED;
    *rows = heads * p->Sq;
    return GTMS_OK;
}

// Strides that a tensor map holds: a row's stride steps over the row, the others are 0 (a broadcast) or step
// over it too, all below 2^40 bytes.
inline int check_mapped(const HeadsSpan& t)
{
    for (int i = 0; i < 3; ++i)
        if (t.ext[i] > 1 && ((t.stride[i] < t.row && (i == 2 || t.stride[i] != 0)) || t.stride[i] >= (int64_t(1) << 40)))
            return GTMS_ERR_UNSUPPORTED;
    return GTMS_OK;
}

// One strided operand: pointer, alignment, strides, distinct elements of outputs.
inline int check_heads(const gtms_heads* t, int64_t B, int64_t H, int64_t S, int64_t D, int elem, int align, bool output,
                HeadsSpan& span)
{
    if (!t || !t->data)
        return GTMS_ERR_INVALID_ARG;
    if (!heads_span(*t, B, H, S, D, elem, span) || !aligned_to(t->data, elem))
        return GTMS_ERR_INVALID_ARG;
    if (output && !heads_distinct(span))
        return GTMS_ERR_INVALID_ARG;
    if (!aligned_to(t->data, align))
        return GTMS_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (span.stride[i] % align != 0)
            return GTMS_ERR_UNSUPPORTED;
    return align == 16 ? check_mapped(span) : GTMS_OK;   // 16: the attention calls
}

inline bool hits(const HeadsSpan& t, const void* p, uint64_t bytes)
{
    return p && ranges_overlap(t.base, t.bytes, reinterpret_cast<uint64_t>(p), bytes);
}

inline void fill_args(AttentionArgs& a, const gtms_attention_shape& p)
{
    a.B = static_cast<int32_t>(p.B);
    a.Hq = static_cast<int32_t>(p.Hq);
    a.Hkv = static_cast<int32_t>(p.Hkv);
    a.group = static_cast<int32_t>(p.Hq / p.Hkv);
    a.Sq = static_cast<int32_t>(p.Sq);
    a.Skv = static_cast<int32_t>(p.Skv);
    // Positions are below GTMS_ATTENTION_MAX_S: a wider window keeps the same entries.
    a.window = static_cast<int32_t>(p.window < GTMS_ATTENTION_MAX_S ? p.window : GTMS_ATTENTION_MAX_S);
    a.mask_kind = p.mask_kind;
    a.scale = p.scale;
}

}  // namespace gtms
