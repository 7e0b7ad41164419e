// gtms_heads.h -- host-side checks of strided [B, H, S, head_dim] tensors
// (gtms_heads), shared by the attention and rotary entry points.
#pragma once

#include <cstdint>

#include "gtms.h"

namespace gtms {

// A checked tensor: extents, byte strides (0 for a dimension of extent 1) and
// the bytes from the first element to one past the last.
struct HeadsSpan {
    uint64_t base = 0, bytes = 0;
    int64_t ext[3] = {0, 0, 0};      // B, H, S
    int64_t stride[3] = {0, 0, 0};   // bytes
    int64_t row = 0;                 // bytes of one head's vector
};

// Fills `out`; false where a stride is negative or the byte range overflows.
inline bool heads_span(const gtms_heads& t, int64_t B, int64_t H, int64_t S, int64_t D, int elem, HeadsSpan& out)
{
    const int64_t ext[3] = {B, H, S}, st[3] = {t.stride_b, t.stride_h, t.stride_s};
    out.base = reinterpret_cast<uint64_t>(t.data);
    out.row = D * elem;
    int64_t last = 0;
    for (int i = 0; i < 3; ++i) {
        out.ext[i] = ext[i];
        if (ext[i] <= 1) {
            out.stride[i] = 0;
            continue;
        }
        int64_t span;
        if (st[i] < 0 || __builtin_mul_overflow(st[i], static_cast<int64_t>(elem), &out.stride[i]) ||
            __builtin_mul_overflow(out.stride[i], ext[i] - 1, &span) || __builtin_add_overflow(last, span, &last))
            return false;
    }
    if (__builtin_add_overflow(last, out.row, &last) ||
        out.base + static_cast<uint64_t>(last) < out.base)
        return false;
    out.bytes = static_cast<uint64_t>(last);
    return true;
}

// Distinct elements: taken in the order of their strides, each dimension steps
// over everything the smaller ones span.
inline bool heads_distinct(const HeadsSpan& t)
{
    int64_t st[3], ex[3];
    int n = 0;
    for (int i = 0; i < 3; ++i)
        if (t.ext[i] > 1) {
            int j = n++;
            for (; j > 0 && st[j - 1] > t.stride[i]; --j) {
                st[j] = st[j - 1];
                ex[j] = ex[j - 1];
            }
            st[j] = t.stride[i];
            ex[j] = t.ext[i];
        }
    int64_t span = t.row;
    for (int i = 0; i < n; ++i) {
        if (st[i] < span)
            return false;
        span += st[i] * (ex[i] - 1);
    }
    return true;
}

inline bool ranges_overlap(uint64_t a, uint64_t an, uint64_t b, uint64_t bn) { return a < b + bn && b < a + an; }

// False only where no element of a can be one of b: the byte ranges are apart,
// or both tensors repeat with one common period and stand apart inside it (the
// parts of one fused projection).
inline bool heads_may_overlap(const HeadsSpan& a, const HeadsSpan& b)
{
    if (!ranges_overlap(a.base, a.bytes, b.base, b.bytes))
        return false;
    for (int c = 0; c < 3; ++c) {
        const int64_t period = a.stride[c];
        if (period <= 0)
            continue;
        int64_t span[2];
        bool fits = true;
        for (int k = 0; k < 2 && fits; ++k) {
            const HeadsSpan& t = k == 0 ? a : b;
            span[k] = t.row;
            for (int i = 0; i < 3; ++i) {
                if (t.stride[i] >= period)
                    fits = fits && t.stride[i] % period == 0;
                else if (t.ext[i] > 1)
                    span[k] += t.stride[i] * (t.ext[i] - 1);
            }
            fits = fits && span[k] <= period;
        }
        if (!fits)
            continue;
        const uint64_t p = static_cast<uint64_t>(period);
        const uint64_t delta = b.base >= a.base ? (b.base - a.base) % p : (p - (a.base - b.base) % p) % p;
        if (delta >= static_cast<uint64_t>(span[0]) && delta + static_cast<uint64_t>(span[1]) <= p)
            return false;
    }
    return true;
}

inline bool heads_same(const HeadsSpan& a, const HeadsSpan& b)
{
    if (a.base != b.base || a.row != b.row)
        return false;
    for (int i = 0; i < 3; ++i)
        if (a.ext[i] != b.ext[i] || a.stride[i] != b.stride[i])
            return false;
    return true;
}

}  // namespace gtms
