// gtms_caches_api.cu -- the entry points of include/gtms.h on key/value caches
// (shared prefixes, key weights, eviction): host-side argument checks and dispatch.
// No allocation, no synchronisation, no host read of device memory.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gtms.h"
#include "gtms_caches.h"
#include "gtms_checks.h"

namespace gtms {
#define GTMS_EXTERN_CACHES(T, D)                                                        \
    extern template cudaError_t launch_key_weights<T, D>(const KeyWeightsArgs&, cudaStream_t); \
    extern template cudaError_t launch_shared_prefix<T, D>(const AttentionArgs&, const PrefixArgs&, void*, cudaStream_t);
GTMS_EXTERN_CACHES(__nv_bfloat16, 64)
GTMS_EXTERN_CACHES(__nv_bfloat16, 128)
GTMS_EXTERN_CACHES(__half, 64)
GTMS_EXTERN_CACHES(__half, 128)
#undef GTMS_EXTERN_CACHES
}  // namespace gtms

namespace {

using namespace gtms;

// A plain array as a span, to be held against others.
HeadsSpan array_span(const void* p, uint64_t bytes)
{
    HeadsSpan s;
    s.base = reinterpret_cast<uint64_t>(p);
    s.bytes = p ? bytes : 0;
    return s;
}

bool meet(const HeadsSpan& a, const HeadsSpan& b)
{
    return a.bytes != 0 && b.bytes != 0 && ranges_overlap(a.base, a.bytes, b.base, b.bytes);
}

// The call's function for its type and head dim.
template <typename Call>
cudaError_t dispatch(const gtms_attention_shape& p, Call call)
{
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (p.dtype == GTMS_BF16)
        return p.head_dim == 64 ? call(__nv_bfloat16(), D64()) : call(__nv_bfloat16(), D128());
    return p.head_dim == 64 ? call(__half(), D64()) : call(__half(), D128());
}

// Sizes of a call over shared prefixes; *rows = B Hq Sq.
int check_prefix_shape(const gtms_attention_shape* p, int64_t groups, int64_t prefix, int64_t* rows)
{
    const int rc = check_shape(p, rows);
    if (rc != GTMS_OK)
        return rc;
    if (groups < 0 || prefix < 0 || (p->B > 0 && (groups == 0 || p->B % groups != 0)))
        return GTMS_ERR_INVALID_ARG;
    if (p->mask_kind == GTMS_MASK_SLIDING_WINDOW || prefix > GTMS_ATTENTION_MAX_S)
        return GTMS_ERR_UNSUPPORTED;
    return GTMS_OK;
}

void fill_prefix(AttentionArgs& a, PrefixArgs& x, const gtms_attention_shape& p, int64_t groups, int64_t prefix)
{
    fill_args(a, p);
    x.G = static_cast<int32_t>(groups);
    x.P = static_cast<int32_t>(prefix);
    x.n = static_cast<int32_t>(p.B / groups);
}

}  // namespace

GTMS_EXPORT int gtms_attention_shared_prefix_workspace(const gtms_attention_shape* shape, int64_t groups, int64_t prefix,
                                                       uint64_t* bytes)
{
    int64_t rows = 0;
    const int rc = check_prefix_shape(shape, groups, prefix, &rows);
    if (rc != GTMS_OK)
        return rc;
    if (!bytes)
        return GTMS_ERR_INVALID_ARG;
    *bytes = 0;
    if (rows == 0)
        return GTMS_OK;
    AttentionArgs a{};
    PrefixArgs x{};
    fill_prefix(a, x, *shape, groups, prefix);
    *bytes = shared_prefix_workspace_bytes(a, x, shape->head_dim);
    return GTMS_OK;
}

GTMS_EXPORT int gtms_attention_shared_prefix(const gtms_attention_shape* shape, int64_t groups, int64_t prefix,
                                             const gtms_heads* q, const gtms_heads* k_prefix, const gtms_heads* v_prefix,
                                             const gtms_heads* k, const gtms_heads* v, const gtms_heads* o, float* lse,
                                             const int32_t* prefix_lens, const int32_t* seq_lens, const int32_t* q_offsets,
                                             void* workspace, uint64_t workspace_bytes, int32_t* status, void* stream)
{
    int64_t rows = 0;
    int rc = check_prefix_shape(shape, groups, prefix, &rows);
    if (rc != GTMS_OK || rows == 0)
        return rc;
    const gtms_attention_shape& p = *shape;
    // q, prefix k and v, k, v (an empty side has no operands to check), o
    const gtms_heads* const ptr[6] = {q, k_prefix, v_prefix, k, v, o};
    const int64_t B[6] = {p.B, groups, groups, p.B, p.B, p.B}, H[6] = {p.Hq, p.Hkv, p.Hkv, p.Hkv, p.Hkv, p.Hq};
    const int64_t S[6] = {p.Sq, prefix, prefix, p.Skv, p.Skv, p.Sq};
    HeadsSpan span[6];
    for (int i = 0; i < 6; ++i)
        if (S[i] > 0 && (rc = check_heads(ptr[i], B[i], H[i], S[i], p.head_dim, 2, 16, i == 5, span[i])) != GTMS_OK)
            return rc;
    AttentionArgs a{};
    PrefixArgs x{};
    fill_prefix(a, x, p, groups, prefix);
    const uint64_t need = shared_prefix_workspace_bytes(a, x, p.head_dim);
    if (!seq_lens || !aligned_to(seq_lens, 4) || !aligned_to(prefix_lens, 4) || !aligned_to(q_offsets, 4) ||
        !aligned_to(lse, 4) || !aligned_to(status, 4) ||
        (need > 0 && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16))))
        return GTMS_ERR_INVALID_ARG;
    // What is written must not meet anything else.
    const uint64_t lens = static_cast<uint64_t>(p.B) * 4;
    const HeadsSpan small[4] = {array_span(seq_lens, lens), array_span(q_offsets, lens),
                                array_span(prefix_lens, static_cast<uint64_t>(groups) * 4), array_span(status, 4)};
    const HeadsSpan out[3] = {span[5], array_span(lse, static_cast<uint64_t>(rows) * 4), array_span(workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 4; ++j)
            if (meet(out[i], small[j]))
                return GTMS_ERR_INVALID_ARG;
        for (int j = 0; j < 5; ++j)
            if (i == 0 ? span[j].bytes != 0 && heads_may_overlap(out[0], span[j]) : meet(out[i], span[j]))
                return GTMS_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j]))
                return GTMS_ERR_INVALID_ARG;
    }
    a.q = device_ref(*q, span[0], 2);
    a.o = device_ref(*o, span[5], 2);
    if (prefix > 0) {
        x.k = device_ref(*k_prefix, span[1], 2);
        x.v = device_ref(*v_prefix, span[2], 2);
    }
    if (p.Skv > 0) {
        a.k = device_ref(*k, span[3], 2);
        a.v = device_ref(*v, span[4], 2);
    }
    a.lse = lse;
    a.seq_lens = seq_lens;
    a.q_offsets = q_offsets;
    a.status = status;
    x.lens = prefix_lens;
    return status_of(dispatch(p, [&](auto type, auto dim) {
        return launch_shared_prefix<decltype(type), dim()>(a, x, workspace, static_cast<cudaStream_t>(stream));
    }));
}

GTMS_EXPORT int gtms_attention_key_weights_workspace(const gtms_attention_shape* shape, uint64_t* bytes)
{
    int64_t rows = 0;
    const int rc = check_shape(shape, &rows);
    if (rc != GTMS_OK)
        return rc;
    if (!bytes)
        return GTMS_ERR_INVALID_ARG;
    *bytes = 0;
    if (rows == 0 || shape->Skv == 0)
        return GTMS_OK;
    AttentionArgs a{};
    fill_args(a, *shape);
    *bytes = key_weights_workspace_bytes(a);
    return GTMS_OK;
}

GTMS_EXPORT int gtms_attention_key_weights(const gtms_attention_shape* shape, const gtms_heads* q, const gtms_heads* k,
                                           const float* lse, float* weights, int accumulate, const int32_t* seq_lens,
                                           const int32_t* q_offsets, void* workspace, uint64_t workspace_bytes,
                                           int32_t* status, void* stream)
{
    int64_t rows = 0;
    int rc = check_shape(shape, &rows);
    if (rc != GTMS_OK)
        return rc;
    const gtms_attention_shape& p = *shape;
    const int64_t keys = p.B * p.Hkv * p.Skv;
    if (keys == 0)
        return GTMS_OK;
    HeadsSpan sq, sk;
    if (rows > 0 && ((rc = check_heads(q, p.B, p.Hq, p.Sq, p.head_dim, 2, 16, false, sq)) != GTMS_OK ||
                     (rc = check_heads(k, p.B, p.Hkv, p.Skv, p.head_dim, 2, 16, false, sk)) != GTMS_OK))
        return rc;
    AttentionArgs a{};
    fill_args(a, p);
    const uint64_t need = rows > 0 ? key_weights_workspace_bytes(a) : 0;
    if (!weights || !aligned_to(weights, 4) || !seq_lens || !aligned_to(seq_lens, 4) || !aligned_to(q_offsets, 4) ||
        !aligned_to(status, 4) || (rows > 0 && (!lse || !aligned_to(lse, 4))) ||
        (need > 0 && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16))))
        return GTMS_ERR_INVALID_ARG;
    const uint64_t lens = static_cast<uint64_t>(p.B) * 4;
    const HeadsSpan in[6] = {array_span(seq_lens, lens), array_span(q_offsets, lens), array_span(status, 4),
                             array_span(lse, static_cast<uint64_t>(rows) * 4), sq, sk};
    const HeadsSpan out[2] = {array_span(weights, static_cast<uint64_t>(keys) * 4), array_span(workspace, need)};
    for (const HeadsSpan& t : in)
        if (meet(out[0], t) || meet(out[1], t))
            return GTMS_ERR_INVALID_ARG;
    if (meet(out[0], out[1]))
        return GTMS_ERR_INVALID_ARG;
    KeyWeightsArgs w{};
    if (rows > 0) {
        a.q = device_ref(*q, sq, 2);
        a.k = device_ref(*k, sk, 2);
    }
    a.lse = const_cast<float*>(lse);
    a.seq_lens = seq_lens;
    a.q_offsets = q_offsets;
    a.status = status;
    w.a = a;
    w.weights = weights;
    w.parts = static_cast<float*>(workspace);
    w.accumulate = accumulate != 0;
    return status_of(dispatch(p, [&](auto type, auto dim) {
        return launch_key_weights<decltype(type), dim()>(w, static_cast<cudaStream_t>(stream));
    }));
}

namespace {

// Sizes of an eviction; *keep = the entries of a sequence that can stay.
int check_evict_shape(const gtms_evict_shape* p, int64_t* keep)
{
    if (!p || p->B < 0 || p->H < 0 || p->S < 0 || p->S_out < 0 || p->head_dim < 0 || p->keep < 0 || p->first < 0 ||
        p->recent < 0 || p->first > p->keep || p->recent > p->keep - p->first)
        return GTMS_ERR_INVALID_ARG;
    *keep = p->keep < p->S ? p->keep : p->S;
    if (p->S_out < *keep)
        return GTMS_ERR_INVALID_ARG;
    const int elem = p->dtype == GTMS_F32 ? 4 : 2;
    if ((p->dtype != GTMS_F32 && p->dtype != GTMS_BF16 && p->dtype != GTMS_F16) || p->head_dim > 1024 ||
        (p->head_dim * elem) % 16 != 0 || p->S > GTMS_ATTENTION_MAX_S || p->S_out > GTMS_ATTENTION_MAX_S)
        return GTMS_ERR_UNSUPPORTED;
    // Clusters of up to 8 CTAs to a (batch, head), and a CTA to 8 rows of 4 KB, more shorter ones, of those that stay (to
    // fewer only while CTAs are few beside the multiprocessors).
    int64_t heads = 0, ctas = 0;
    if (__builtin_mul_overflow(p->B, p->H, &heads) || __builtin_mul_overflow(heads, *keep / 8 + 129, &ctas) ||
        ctas > INT32_MAX)
        return GTMS_ERR_UNSUPPORTED;
    return GTMS_OK;
}

}  // namespace

GTMS_EXPORT int gtms_cache_evict_workspace(const gtms_evict_shape* shape, uint64_t* bytes)
{
    int64_t keep = 0;
    const int rc = check_evict_shape(shape, &keep);
    if (rc != GTMS_OK)
        return rc;
    if (!bytes)
        return GTMS_ERR_INVALID_ARG;
    *bytes = evict_workspace_bytes(shape->B, shape->H, keep);
    return GTMS_OK;
}

GTMS_EXPORT int gtms_cache_evict(const gtms_evict_shape* shape, const gtms_heads* k, const gtms_heads* v, const float* weights,
                                 const int32_t* positions, const gtms_heads* k_out, const gtms_heads* v_out,
                                 float* weights_out, int32_t* positions_out, const int32_t* seq_lens, int32_t* lens_out,
                                 void* workspace, uint64_t workspace_bytes, void* stream)
{
    int64_t keep = 0;
    int rc = check_evict_shape(shape, &keep);
    if (rc != GTMS_OK)
        return rc;
    const gtms_evict_shape& p = *shape;
    const int64_t heads = p.B * p.H;
    if (heads == 0 || p.head_dim == 0)
        return p.B == 0 ? GTMS_OK : GTMS_ERR_INVALID_ARG;   // without heads nothing would write the lengths
    const int elem = p.dtype == GTMS_F32 ? 4 : 2;
    const uint64_t need = evict_workspace_bytes(p.B, p.H, keep), lens = static_cast<uint64_t>(p.B) * 4;
    if (!seq_lens || !aligned_to(seq_lens, 4) || !lens_out || !aligned_to(lens_out, 4) ||
        (need > 0 && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16))))
        return GTMS_ERR_INVALID_ARG;
    const gtms_heads* const ptr[4] = {k, v, k_out, v_out};
    HeadsSpan span[4], label[4];   // weights, positions, in and out
    EvictArgs a{};
    if (keep > 0) {
        for (int i = 0; i < 4; ++i)
            if ((rc = check_heads(ptr[i], p.B, p.H, i < 2 ? p.S : p.S_out, p.head_dim, elem, 16, i >= 2, span[i])) != GTMS_OK)
                return rc;
        if (!weights || !aligned_to(weights, 4) || !weights_out || !aligned_to(weights_out, 4) || !aligned_to(positions, 4) ||
            !aligned_to(positions_out, 4))
            return GTMS_ERR_INVALID_ARG;
        const uint64_t in = static_cast<uint64_t>(heads) * p.S * 4, out = static_cast<uint64_t>(heads) * p.S_out * 4;
        label[0] = array_span(weights, in);
        label[1] = array_span(positions, in);
        label[2] = array_span(weights_out, out);
        label[3] = array_span(positions_out, out);
    }
    // What is written meets nothing, save that a tensor may be compacted where it stands.
    const HeadsSpan small[3] = {array_span(seq_lens, lens), array_span(lens_out, lens), array_span(workspace, need)};
    if (meet(small[1], small[0]) || meet(small[2], small[0]) || meet(small[2], small[1]))
        return GTMS_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i) {
        if (meet(span[i], small[1]) || meet(span[i], small[2]) || meet(label[i], small[1]) || meet(label[i], small[2]))
            return GTMS_ERR_INVALID_ARG;
        if (i < 2)
            continue;
        if (meet(span[i], small[0]) || meet(label[i], small[0]))
            return GTMS_ERR_INVALID_ARG;
        for (int j = 0; j < 4; ++j) {
            if (meet(span[i], label[j]) || meet(label[i], span[j]))
                return GTMS_ERR_INVALID_ARG;
            const bool same = j == i - 2 && p.S == p.S_out;
            if (j < i && span[j].bytes != 0 && !(same && heads_same(span[i], span[j])) && heads_may_overlap(span[i], span[j]))
                return GTMS_ERR_INVALID_ARG;
            if (j < i && !(same && label[i].base == label[j].base) && meet(label[i], label[j]))
                return GTMS_ERR_INVALID_ARG;
        }
    }
    for (int i = 0; i < 2 && keep > 0; ++i) {
        a.in[i] = device_ref(*ptr[i], span[i], 16);
        a.out[i] = device_ref(*ptr[2 + i], span[2 + i], 16);
        a.moved |= (p.S == p.S_out && heads_same(span[i], span[2 + i]) ? 0 : 1) << i;
    }
    a.weights = weights;
    a.weights_out = weights_out;
    a.positions = positions;
    a.positions_out = positions_out;
    a.seq_lens = seq_lens;
    a.lens_out = lens_out;
    a.kept = static_cast<int32_t*>(workspace);
    a.B = static_cast<int32_t>(p.B);
    a.H = static_cast<int32_t>(p.H);
    a.S = static_cast<int32_t>(p.S);
    a.S_out = static_cast<int32_t>(p.S_out);
    a.keep = static_cast<int32_t>(keep);
    a.first = static_cast<int32_t>(p.first);
    a.recent = static_cast<int32_t>(p.recent);
    a.units = static_cast<int32_t>(p.head_dim * elem / 16);
    return status_of(launch_cache_evict(a, static_cast<cudaStream_t>(stream)));
}
