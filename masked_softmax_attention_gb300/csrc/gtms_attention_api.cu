// gtms_attention_api.cu -- the attention and rotary entry points of
// include/gtms.h: host-side argument checks and dispatch on type and head dim.
// No allocation, no synchronisation, no host read of device memory.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gtms.h"
#include "gtms_attention.h"
#include "gtms_heads.h"

#define GTMS_EXPORT extern "C" __attribute__((visibility("default")))

namespace gtms {
#define GTMS_EXTERN_ATTENTION(T, D)                                                            \
    extern template cudaError_t launch_attention_forward<T, D>(const AttentionArgs&, cudaStream_t);  \
    extern template cudaError_t launch_attention_backward<T, D>(const AttentionArgs&, cudaStream_t);
GTMS_EXTERN_ATTENTION(__nv_bfloat16, 64)
GTMS_EXTERN_ATTENTION(__nv_bfloat16, 128)
GTMS_EXTERN_ATTENTION(__half, 64)
GTMS_EXTERN_ATTENTION(__half, 128)
#undef GTMS_EXTERN_ATTENTION
extern template cudaError_t launch_rotary<float>(const RotaryArgs&, bool, cudaStream_t);
extern template cudaError_t launch_rotary<__nv_bfloat16>(const RotaryArgs&, bool, cudaStream_t);
extern template cudaError_t launch_rotary<__half>(const RotaryArgs&, bool, cudaStream_t);
}  // namespace gtms

namespace {

using gtms::HeadsSpan;

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int status_of(cudaError_t e)
{
    if (e == cudaSuccess)
        return GTMS_OK;
    cudaGetLastError();   // reported through the returned code
    return e == cudaErrorNotSupported ? GTMS_ERR_UNSUPPORTED : GTMS_ERR_CUDA;
}

gtms::HeadsRef device_ref(const gtms_heads& t, const HeadsSpan& s, int elem)
{
    return {t.data, s.stride[0] / elem, s.stride[1] / elem, s.stride[2] / elem};
}

// Sizes and options that both directions share; *rows = B * Hq * Sq.
int check_shape(const gtms_attention_shape* p, int64_t* rows)
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
int check_mapped(const HeadsSpan& t)
{
    for (int i = 0; i < 3; ++i)
        if (t.ext[i] > 1 && ((t.stride[i] < t.row && (i == 2 || t.stride[i] != 0)) || t.stride[i] >= (int64_t(1) << 40)))
            return GTMS_ERR_UNSUPPORTED;
    return GTMS_OK;
}

// One strided operand: pointer, alignment, strides, distinct elements of outputs.
int check_heads(const gtms_heads* t, int64_t B, int64_t H, int64_t S, int64_t D, int elem, int align, bool output,
                HeadsSpan& span)
{
    if (!t || !t->data)
        return GTMS_ERR_INVALID_ARG;
    if (!gtms::heads_span(*t, B, H, S, D, elem, span) || !aligned_to(t->data, elem))
        return GTMS_ERR_INVALID_ARG;
    if (output && !gtms::heads_distinct(span))
        return GTMS_ERR_INVALID_ARG;
    if (!aligned_to(t->data, align))
        return GTMS_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (span.stride[i] % align != 0)
            return GTMS_ERR_UNSUPPORTED;
    return align == 16 ? check_mapped(span) : GTMS_OK;   // 16: the attention calls
}

bool hits(const HeadsSpan& t, const void* p, uint64_t bytes)
{
    return p && gtms::ranges_overlap(t.base, t.bytes, reinterpret_cast<uint64_t>(p), bytes);
}

void fill_args(gtms::AttentionArgs& a, const gtms_attention_shape& p)
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

template <template <typename, int> class Launch>
cudaError_t dispatch(const gtms_attention_shape& p, const gtms::AttentionArgs& a, cudaStream_t st)
{
    if (p.dtype == GTMS_BF16)
        return p.head_dim == 64 ? Launch<__nv_bfloat16, 64>::run(a, st) : Launch<__nv_bfloat16, 128>::run(a, st);
    return p.head_dim == 64 ? Launch<__half, 64>::run(a, st) : Launch<__half, 128>::run(a, st);
}

template <typename T, int D>
struct Forward {
    static cudaError_t run(const gtms::AttentionArgs& a, cudaStream_t st) { return gtms::launch_attention_forward<T, D>(a, st); }
};
template <typename T, int D>
struct Backward {
    static cudaError_t run(const gtms::AttentionArgs& a, cudaStream_t st) { return gtms::launch_attention_backward<T, D>(a, st); }
};

}  // namespace

GTMS_EXPORT int gtms_attention_forward(const gtms_attention_shape* shape, const gtms_heads* q, const gtms_heads* k,
                                       const gtms_heads* v, const gtms_heads* o, float* lse, const int32_t* seq_lens,
                                       const int32_t* q_offsets, int32_t* status, void* stream)
{
    int64_t rows = 0;
    int rc = check_shape(shape, &rows);
    if (rc != GTMS_OK || rows == 0)
        return rc;
    const gtms_attention_shape& p = *shape;
    HeadsSpan sq, sk, sv, so;
    if ((rc = check_heads(q, p.B, p.Hq, p.Sq, p.head_dim, 2, 16, false, sq)) != GTMS_OK ||
        (rc = check_heads(o, p.B, p.Hq, p.Sq, p.head_dim, 2, 16, true, so)) != GTMS_OK)
        return rc;
    if (p.Skv > 0 && ((rc = check_heads(k, p.B, p.Hkv, p.Skv, p.head_dim, 2, 16, false, sk)) != GTMS_OK ||
                      (rc = check_heads(v, p.B, p.Hkv, p.Skv, p.head_dim, 2, 16, false, sv)) != GTMS_OK))
        return rc;
    if (!seq_lens || !aligned_to(seq_lens, 4) || !aligned_to(q_offsets, 4) || !aligned_to(lse, 4) ||
        !aligned_to(status, 4))
        return GTMS_ERR_INVALID_ARG;
    const uint64_t lens = static_cast<uint64_t>(p.B) * 4, lse_bytes = static_cast<uint64_t>(rows) * 4;
    if (gtms::heads_may_overlap(so, sq) || (p.Skv > 0 && (gtms::heads_may_overlap(so, sk) || gtms::heads_may_overlap(so, sv))))
        return GTMS_ERR_INVALID_ARG;
    if (hits(so, seq_lens, lens) || hits(so, q_offsets, lens) || hits(so, status, 4) || hits(so, lse, lse_bytes))
        return GTMS_ERR_INVALID_ARG;
    if (lse) {
        HeadsSpan sl;
        sl.base = reinterpret_cast<uint64_t>(lse);
        sl.bytes = lse_bytes;
        if (hits(sl, seq_lens, lens) || hits(sl, q_offsets, lens) || hits(sl, status, 4) || hits(sq, lse, lse_bytes) ||
            (p.Skv > 0 && (hits(sk, lse, lse_bytes) || hits(sv, lse, lse_bytes))))
            return GTMS_ERR_INVALID_ARG;
    }
    gtms::AttentionArgs a{};
    fill_args(a, p);
    a.q = device_ref(*q, sq, 2);
    a.o = device_ref(*o, so, 2);
    if (p.Skv > 0) {
        a.k = device_ref(*k, sk, 2);
        a.v = device_ref(*v, sv, 2);
    }
    a.lse = lse;
    a.seq_lens = seq_lens;
    a.q_offsets = q_offsets;
    a.status = status;
    return status_of(dispatch<Forward>(p, a, static_cast<cudaStream_t>(stream)));
}

GTMS_EXPORT int gtms_attention_backward_workspace(const gtms_attention_shape* shape, uint64_t* bytes)
{
    int64_t rows = 0;
    const int rc = check_shape(shape, &rows);
    if (rc != GTMS_OK)
        return rc;
    if (!bytes)
        return GTMS_ERR_INVALID_ARG;
    *bytes = gtms::attention_workspace_bytes(shape->B, shape->Hq, shape->Sq);
    return GTMS_OK;
}

GTMS_EXPORT int gtms_attention_backward(const gtms_attention_shape* shape, const gtms_heads* q, const gtms_heads* k,
                                        const gtms_heads* v, const gtms_heads* o, const float* lse,
                                        const gtms_heads* dout, const gtms_heads* dq, const gtms_heads* dk,
                                        const gtms_heads* dv, const int32_t* seq_lens, const int32_t* q_offsets,
                                        void* workspace, uint64_t workspace_bytes, int32_t* status, void* stream)
{
    int64_t rows = 0;
    int rc = check_shape(shape, &rows);
    if (rc != GTMS_OK)
        return rc;
    const gtms_attention_shape& p = *shape;
    const int64_t keys = p.B * p.Hkv * p.Skv;
    if (rows == 0 && keys == 0)
        return GTMS_OK;
    // inputs q, o, dout, k, v; outputs dq, dk, dv (an empty side has no operands to check)
    const gtms_heads* const ptr[8] = {q, o, dout, dq, k, v, dk, dv};
    HeadsSpan span[8];
    for (int i = 0; i < 8; ++i) {
        const bool of_q = i < 4;
        if ((of_q ? rows : keys) == 0)
            continue;
        rc = check_heads(ptr[i], p.B, of_q ? p.Hq : p.Hkv, of_q ? p.Sq : p.Skv, p.head_dim, 2, 16,
                         i == 3 || i >= 6, span[i]);
        if (rc != GTMS_OK)
            return rc;
    }
    const uint64_t need = gtms::attention_workspace_bytes(p.B, p.Hq, p.Sq);
    if (!seq_lens || !aligned_to(seq_lens, 4) || !aligned_to(q_offsets, 4) || !aligned_to(status, 4) ||
        (rows > 0 && (!lse || !aligned_to(lse, 4))) || !workspace || workspace_bytes < need ||
        !aligned_to(workspace, 16))
        return GTMS_ERR_INVALID_ARG;
    const uint64_t lens = static_cast<uint64_t>(p.B) * 4, lse_bytes = static_cast<uint64_t>(rows) * 4;
    for (int i = 0; i < 8; ++i) {
        if (span[i].bytes == 0)
            continue;
        const bool output = i == 3 || i >= 6;
        if (hits(span[i], workspace, need))
            return GTMS_ERR_INVALID_ARG;
        if (!output)
            continue;
        if (hits(span[i], seq_lens, lens) || hits(span[i], q_offsets, lens) || hits(span[i], status, 4) ||
            hits(span[i], lse, lse_bytes))
            return GTMS_ERR_INVALID_ARG;
        for (int j = 0; j < 8; ++j)
            if (j != i && span[j].bytes != 0 && gtms::heads_may_overlap(span[i], span[j]))
                return GTMS_ERR_INVALID_ARG;
    }
    HeadsSpan w;
    w.base = reinterpret_cast<uint64_t>(workspace);
    w.bytes = need;
    if (hits(w, seq_lens, lens) || hits(w, q_offsets, lens) || hits(w, status, 4) || hits(w, lse, lse_bytes))
        return GTMS_ERR_INVALID_ARG;
    gtms::AttentionArgs a{};
    fill_args(a, p);
    gtms::HeadsRef* const ref[8] = {&a.q, &a.o, &a.dout, &a.dq, &a.k, &a.v, &a.dk, &a.dv};
    for (int i = 0; i < 8; ++i)
        if (span[i].bytes != 0)
            *ref[i] = device_ref(*ptr[i], span[i], 2);
    a.lse = const_cast<float*>(lse);
    gtms::attention_workspace(a, workspace);
    a.seq_lens = seq_lens;
    a.q_offsets = q_offsets;
    a.status = status;
    return status_of(dispatch<Backward>(p, a, static_cast<cudaStream_t>(stream)));
}

GTMS_EXPORT int gtms_rotary(const gtms_heads* x, const gtms_heads* y, const gtms_heads* x2, const gtms_heads* y2,
                            int64_t B, int64_t H, int64_t H2, int64_t S, int64_t head_dim, int64_t rot_dim,
                            const int32_t* positions, int64_t position_batches, const float* inv_freq,
                            int interleaved, float amplitude, int inverse, int dtype, void* stream)
{
    if (B < 0 || H < 0 || H2 < 0 || S < 0 || head_dim < 0 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0 ||
        !std::isfinite(amplitude) || (x2 == nullptr) != (y2 == nullptr) || (x2 == nullptr && H2 != 0))
        return GTMS_ERR_INVALID_ARG;
    const int elem = dtype == GTMS_F32 ? 4 : 2;
    if ((dtype != GTMS_F32 && dtype != GTMS_BF16 && dtype != GTMS_F16) || head_dim > 1024 || S > GTMS_ATTENTION_MAX_S)
        return GTMS_ERR_UNSUPPORTED;
    int64_t heads = 0, vectors = 0;
    if (__builtin_add_overflow(H, H2, &heads) || __builtin_mul_overflow(heads, B, &vectors) ||
        __builtin_mul_overflow(vectors, S, &vectors) || vectors > (int64_t(1) << 40) || heads > GTMS_ATTENTION_MAX_S)
        return GTMS_ERR_UNSUPPORTED;
    if (vectors == 0 || head_dim == 0)
        return GTMS_OK;
    if (B * S > INT32_MAX)   // a block each
        return GTMS_ERR_UNSUPPORTED;
    if (!positions || !aligned_to(positions, 4) || (position_batches != 1 && position_batches != B) ||
        (rot_dim > 0 && !inv_freq) || !aligned_to(inv_freq, 4))
        return GTMS_ERR_INVALID_ARG;
    const gtms_heads* const in[2] = {x, x2};
    const gtms_heads* const out[2] = {y, y2};
    const int64_t count[2] = {H, H2};
    HeadsSpan si[2], so[2];
    gtms::RotaryArgs a{};
    const int64_t half = interleaved ? rot_dim : rot_dim / 2;   // elements that a 16-byte unit must not straddle
    bool wide = (half * elem) % 16 == 0 && ((head_dim - rot_dim) * elem) % 16 == 0;
    for (int t = 0; t < 2; ++t) {
        a.H[t] = static_cast<int32_t>(count[t]);
        if (count[t] == 0)
            continue;
        int rc;
        if ((rc = check_heads(in[t], B, count[t], S, head_dim, elem, elem, false, si[t])) != GTMS_OK ||
            (rc = check_heads(out[t], B, count[t], S, head_dim, elem, elem, true, so[t])) != GTMS_OK)
            return rc;
        a.x[t] = device_ref(*in[t], si[t], elem);
        a.y[t] = device_ref(*out[t], so[t], elem);
        if (!gtms::heads_same(si[t], so[t]))
            a.copy = 1;
        for (const HeadsSpan* s : {&si[t], &so[t]})
            wide = wide && s->base % 16 == 0 && s->stride[0] % 16 == 0 && s->stride[1] % 16 == 0 && s->stride[2] % 16 == 0;
    }
    const uint64_t pos_bytes = static_cast<uint64_t>(position_batches) * S * 4, freq_bytes = static_cast<uint64_t>(rot_dim) * 2;
    for (int t = 0; t < 2; ++t) {
        if (count[t] == 0)
            continue;
        if (hits(so[t], positions, pos_bytes) || hits(so[t], inv_freq, freq_bytes))
            return GTMS_ERR_INVALID_ARG;
        for (int u = 0; u < 2; ++u) {
            if (count[u] == 0)
                continue;
            if (!(u == t && gtms::heads_same(si[u], so[t])) && gtms::heads_may_overlap(so[t], si[u]))
                return GTMS_ERR_INVALID_ARG;
            if (u != t && gtms::heads_may_overlap(so[t], so[u]))
                return GTMS_ERR_INVALID_ARG;
        }
    }
    a.positions = positions;
    a.position_stride = position_batches == 1 ? 0 : S;
    a.inv_freq = inv_freq;
    a.B = static_cast<int32_t>(B);
    a.S = static_cast<int32_t>(S);
    a.D = static_cast<int32_t>(head_dim);
    a.R = static_cast<int32_t>(rot_dim);
    a.amplitude = amplitude;
    a.interleaved = interleaved != 0;
    a.inverse = inverse != 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
    case GTMS_F32: return status_of(gtms::launch_rotary<float>(a, wide, st));
    case GTMS_BF16: return status_of(gtms::launch_rotary<__nv_bfloat16>(a, wide, st));
    default: return status_of(gtms::launch_rotary<__half>(a, wide, st));
    }
}

GTMS_EXPORT int gtms_rotary_frequencies(int64_t rot_dim, double base, int scaling, double factor, double low_turns,
                                        double high_turns, int64_t original_length, float* inv_freq)
{
    if (rot_dim < 0 || rot_dim % 2 != 0 || !(base > 0) || !std::isfinite(base) || !(factor > 0) ||
        !std::isfinite(factor) || (rot_dim > 0 && !inv_freq))
        return GTMS_ERR_INVALID_ARG;
    if (scaling < GTMS_ROTARY_PLAIN || scaling > GTMS_ROTARY_BY_PARTS)
        return GTMS_ERR_UNSUPPORTED;
    if (scaling == GTMS_ROTARY_BY_PARTS &&
        (!(high_turns > low_turns) || !std::isfinite(high_turns) || !std::isfinite(low_turns) || original_length < 1))
        return GTMS_ERR_INVALID_ARG;
    for (int64_t j = 0; j < rot_dim / 2; ++j) {
        double f = std::pow(base, -2.0 * static_cast<double>(j) / static_cast<double>(rot_dim));
        if (scaling == GTMS_ROTARY_LINEAR) {
            f /= factor;
        } else if (scaling == GTMS_ROTARY_BY_PARTS) {
            const double turns = static_cast<double>(original_length) * f / (2.0 * 3.14159265358979323846);
            double m = (turns - low_turns) / (high_turns - low_turns);
            m = m < 0.0 ? 0.0 : (m > 1.0 ? 1.0 : m);
            f = (1.0 - m) * f / factor + m * f;
        }
        inv_freq[j] = static_cast<float>(f);
    }
    return GTMS_OK;
}
