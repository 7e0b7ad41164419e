// gtms_shared_prefix.cuh -- attention for a batch whose sequences share long prefixes.
//
// Sequence b of n G keeps, beside its own keys, all keys of prefix b / n:
//   o_i = sum_c exp(s_ic - lse_i) v_c over the prefix's keys and its own kept ones.
//
// Two forms, of the two attention kernels:
//   rows of their own   (prompts, long chunks) a tile of query rows walks over the
//                       tiles of the prefix and then its own, as over one cache
//                       (PrefixedCache). One launch; a prefix tile is read once for 128
//                       or 256 rows of one head, from L2 mostly;
//   rows packed         (new tokens) the rows of all sequences and heads that share a
//                       prefix's head stand in one matrix, 128 to a tile, so that its
//                       keys are read once for all of them and by the tensor cores'
//                       full width. The keys are dealt out in parts, each part's sums
//                       (m, l, O) go to the workspace in fp32 (PrefixRows), and the
//                       split kernel joins them with what it finds in the sequences'
//                       own caches (PrefixParts).
#pragma once

#include "gtms_attention_fwd.cuh"
#include "gtms_attention_split.cuh"
#include "gtms_caches.h"

namespace gtms {

// Tiles [0, prefix_tiles) of an item are the prefix's, those behind them its own.
struct PrefixedCache {
    static constexpr bool prefixed = true, packed = false;
    HeadsMap mk, mv;
    PrefixArgs p;

    template <int W>
    struct Item : FwdItem<W> {
        int32_t g, prefix, prefix_tiles;
    };
    template <int W>
    __device__ __forceinline__ void set(Item<W>& it, const AttentionArgs& a, uint32_t item, uint32_t heads, int32_t blocks) const
    {
        it.set(a, item, heads, blocks);
        it.g = it.b / p.n;
        it.prefix = p.length(it.g);
        it.prefix_tiles = (it.prefix + kTile - 1) / kTile;
#pragma unroll
        for (int w = 0; w < W; ++w)
            it.hi[w] += it.hi[w] > 0 ? it.prefix_tiles : 0;   // lo is 0: no windows here
    }
};

// The partial sums of a prefix's keys: row R of (prefix g, key/value head h) is query
// row (R / group) % Sq, shared head R % group of its sequence R / (group Sq).
struct PrefixParts {
    static constexpr bool any = true;
    float* o;        // [parts, G Hkv, rows, D], not divided by l
    float2* ml;      // [parts, G Hkv, rows]: maximum in base 2 and sum; (-inf, 0) without keys, and o is zero
    int32_t parts, n, G, Hkv, per;   // per: rows of a sequence (group Sq)

    __host__ __device__ __forceinline__ int64_t stride() const { return static_cast<int64_t>(G) * Hkv * n * per; }
    __device__ __forceinline__ int64_t at(int32_t b, int32_t hk, int32_t r) const
    {
        const int32_t g = b / n;
        return (static_cast<int64_t>(g) * Hkv + hk) * (static_cast<int64_t>(n) * per) + static_cast<int64_t>(b - g * n) * per + r;
    }
    // Adds them to a row's sums at maximum `top`: l, and the elements d and d + 1. Eight parts at a time, their loads
    // in flight together (one after the other the parts took most of the call).
    template <int D>
    __device__ __forceinline__ void add(int32_t b, int32_t hk, int32_t r, int32_t d, float& top, float& l, float& x, float& y) const
    {
        constexpr int N = 8;
        const int64_t i = at(b, hk, r), step = stride();
        for (int32_t k = 0; k < parts; k += N) {
            float2 s[N], e[N];
#pragma unroll
            for (int u = 0; u < N; ++u) {
                s[u] = make_float2(-INFINITY, 0.0f);
                e[u] = make_float2(0.0f, 0.0f);
                if (k + u < parts) {
                    s[u] = ml[i + (k + u) * step];
                    e[u] = *reinterpret_cast<const float2*>(o + (i + (k + u) * step) * D + d);
                }
            }
            float t = top;
#pragma unroll
            for (int u = 0; u < N; ++u)
                t = fmaxf(t, s[u].x);
            const float base = t == -INFINITY ? 0.0f : t, f = exp2_approx(top - base);
            l *= f;
            x *= f;
            y *= f;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const float g = exp2_approx(s[u].x - base);
                l += g * s[u].y;
                x += g * e[u].x;
                y += g * e[u].y;
            }
            top = t;
        }
    }
};

// Work items (prefix, head, rows, part of the keys) of the packed rows. The kernel's
// AttentionArgs are those of one batch of G over the prefixes, Sq its packed rows.
struct PrefixRows {
    static constexpr bool prefixed = false, packed = true;
    HeadsRef q;
    PrefixArgs p;
    PrefixParts out;
    int32_t Sq, group;

    template <int W>
    struct Item : FwdItem<W> {
        int32_t part;
    };
    template <int W>
    __device__ __forceinline__ void set(Item<W>& it, const AttentionArgs& a, uint32_t item, uint32_t heads, int32_t) const
    {
        const int32_t gh = static_cast<int32_t>(item % heads), rest = static_cast<int32_t>(item / heads);
        it.part = rest % out.parts;
        it.b = gh / a.Hkv;
        it.h = gh - it.b * a.Hkv;
        it.i0 = rest / out.parts * W * kTile;
        it.off = 0;
        it.L = p.length(it.b);
        const int32_t tiles = (it.L + kTile - 1) / kTile, per = (tiles + out.parts - 1) / out.parts;   // of this prefix
        const int32_t lo = it.part * per, hi = lo + per < tiles ? lo + per : tiles;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const bool any = lo < hi && it.i0 + w * kTile < a.Sq;
            it.lo[w] = any ? lo : 0;
            it.hi[w] = any ? hi : 0;
            it.full0[w] = 0;
            it.full1[w] = it.L;
        }
    }
    template <typename T>
    __device__ __forceinline__ const T* row(int32_t g, int32_t h, int32_t r) const
    {
        const int32_t b = r / out.per, i = r - b * out.per, s = i / group;
        return q.row<T>(g * p.n + b, h * group + (i - s * group), s);
    }
    __device__ __forceinline__ int64_t index(int32_t part, int32_t g, int32_t h, int32_t r) const
    {
        return part * out.stride() + (static_cast<int64_t>(g) * out.Hkv + h) * (static_cast<int64_t>(p.n) * out.per) + r;
    }
};

template <typename T, int D>
cudaError_t launch_prefixed_whole(const AttentionArgs& a, const PrefixArgs& p, cudaStream_t st, uint64_t wait_ns = kAttnWaitNs)
{
    using TL = FwdTile<D>;
    if (!bind_context())
        return cudaErrorUnknown;
    // Without keys no tile is loaded, and q stands in for k and v in the maps.
    const bool keys = a.Skv > 0, shared = p.P > 0;
    HeadsMap mq, mk, mv;
    PrefixedCache source;
    source.p = p;
    if (!encode_heads<T>(mq, a.q, a.B, a.Hq, a.Sq, D, kTile) ||
        !encode_heads<T>(mk, keys ? a.k : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile) ||
        !encode_heads<T>(mv, keys ? a.v : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile) ||
        !encode_heads<T>(source.mk, shared ? p.k : a.q, p.G, a.Hkv, shared ? p.P : 1, D, kTile) ||
        !encode_heads<T>(source.mv, shared ? p.v : a.q, p.G, a.Hkv, shared ? p.P : 1, D, kTile))
        return cudaErrorInvalidValue;
    const int32_t blocks = (a.Sq + TL::rows - 1) / TL::rows;
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hq;
    auto launch = [&](auto is_long) {
        constexpr auto* kern = gtms_attention_fwd_kernel<T, D, is_long(), PrefixedCache>;
        constexpr int smem = static_cast<int>(TL::smem);
        const cudaError_t e = allow_smem<kern>(smem);
        return e != cudaSuccess ? e
                                : launch_kernel(kern, static_cast<unsigned>(heads * blocks), TL::threads, smem, st, mq, mk, mv, a,
                                                static_cast<uint32_t>(heads), blocks, wait_ns, source);
    };
    // A tile counts as whole even where the prefix ends inside it.
    const int64_t most = static_cast<int64_t>(p.P) + kTile + a.Skv;
    return most > kCarryTerms<T> ? launch(std::true_type()) : launch(std::false_type());
}

// How a call's packed rows are dealt out: tiles of rows, parts of the keys.
struct PackedPlan {
    int64_t rows;     // of one prefix and key/value head
    int64_t blocks;   // items of rows
    int32_t parts;
    double us;        // of the first launch
};

// Microseconds of an item of rows x keys, and of 128 keys of one (with both CTAs of a
// multiprocessor busy at head dim 64), as measured for the forward kernel.
template <int D>
constexpr double kItemUs = D == 64 ? 4.0 : 5.0;
template <int D>
constexpr double kTileUs = D == 64 ? 1.0 : 1.15;

// Parts: as many as take the least time. A part's keys are below kCarryTerms of either
// type, so that no sum in an accumulator is long.
template <int D>
PackedPlan packed_plan(const AttentionArgs& a, const PrefixArgs& p)
{
    using TL = FwdTile<D>;
    PackedPlan x;
    x.rows = static_cast<int64_t>(p.n) * a.Sq * a.group;
    x.blocks = (x.rows + TL::rows - 1) / TL::rows;
    const int64_t items = static_cast<int64_t>(p.G) * a.Hkv * x.blocks, slots = int64_t(kChipSms) * TL::ctas;
    const int64_t tiles = (static_cast<int64_t>(p.P) + kTile - 1) / kTile, least = (tiles + 255) / 256;
    x.parts = 1;
    x.us = 0.0;
    for (int64_t parts = least; parts <= tiles && parts <= least + 63; ++parts) {
        const int64_t turns = (items * parts + slots - 1) / slots, per = (tiles + parts - 1) / parts;
        // Each part is written once and read once by the second launch, in fp32, at about 10 TB/s (L2).
        const double us = static_cast<double>(turns) * (kItemUs<D> + kTileUs<D> * static_cast<double>(per)) +
                          static_cast<double>(items * parts) * TL::rows * D * 8 * 1e-7;
        if (parts == least || us < x.us) {
            x.us = us;
            x.parts = static_cast<int32_t>(parts);
        }
    }
    return x;
}

// Whether to pack: always where the rows of a sequence's head fill one tile of the
// split kernel, otherwise by the time that both forms take (see prefer_split).
template <int D>
bool prefer_packed(const AttentionArgs& a, const PrefixArgs& p, const PackedPlan& x)
{
    const int64_t rows = static_cast<int64_t>(a.group) * a.Sq;
    if (p.P == 0 || rows > kSplitMaxRows || x.rows > (1 << 24) || x.blocks * x.parts * p.G * a.Hkv > INT32_MAX)
        return false;
    if (rows <= kSplitRows)
        return true;
    const double items = static_cast<double>(a.B) * a.Hq * ((a.Sq + FwdTile<D>::rows - 1) / FwdTile<D>::rows);
    const double loads = items / (static_cast<double>(kChipSms) * FwdTile<D>::ctas);
    const int64_t tiles = (static_cast<int64_t>(p.P) + kTile - 1) / kTile + (static_cast<int64_t>(a.Skv) + kTile - 1) / kTile;
    const double whole = (loads > 1.0 ? loads : 1.0) * (kItemUs<D> + kTileUs<D> * static_cast<double>(tiles));
    const int64_t units = split_units(a), ranks = split_ranks(units, a.Skv, kChipSms);
    const double turns = static_cast<double>(units * ranks) / (3 * kChipSms);
    const double block = turns > 1.0 ? (D == 64 ? 1.3 : 2.3) : (D == 64 ? 1.0 : 1.8);
    const double split = (turns > 1.0 ? turns : 1.0) * (6.0 + block * static_cast<double>((a.Skv + ranks * 64 - 1) / (ranks * 64)));
    return x.us + split < whole;
}

inline uint64_t packed_bytes(const AttentionArgs& a, const PrefixArgs& p, const PackedPlan& x, int64_t D)
{
    return static_cast<uint64_t>(x.parts) * p.G * a.Hkv * x.rows * (D * 4 + 8);
}

template <typename T, int D>
cudaError_t launch_prefix_packed(const AttentionArgs& a, const PrefixArgs& p, const PackedPlan& x, void* workspace,
                                 cudaStream_t st, uint64_t wait_ns = kAttnWaitNs)
{
    using TL = FwdTile<D>;
    if (!bind_context())
        return cudaErrorUnknown;
    const int64_t heads = static_cast<int64_t>(p.G) * a.Hkv;
    HeadsMap mk, mv;
    if (!encode_heads<T>(mk, p.k, p.G, a.Hkv, p.P, D, kTile) || !encode_heads<T>(mv, p.v, p.G, a.Hkv, p.P, D, kTile))
        return cudaErrorInvalidValue;
    PrefixRows source;
    source.q = a.q;
    source.p = p;
    source.Sq = a.Sq;
    source.group = a.group;
    source.out.o = static_cast<float*>(workspace);
    source.out.ml = reinterpret_cast<float2*>(source.out.o + x.parts * heads * x.rows * D);
    source.out.parts = x.parts;
    source.out.n = p.n;
    source.out.G = p.G;
    source.out.Hkv = a.Hkv;
    source.out.per = a.group * a.Sq;
    AttentionArgs rows = a;   // one batch of G, its queries the packed rows
    rows.B = p.G;
    rows.Hq = a.Hkv;
    rows.group = 1;
    rows.Sq = static_cast<int32_t>(x.rows);
    rows.Skv = p.P;
    rows.mask_kind = GTMS_MASK_LENGTH;
    constexpr auto* kern = gtms_attention_fwd_kernel<T, D, false, PrefixRows>;
    constexpr int smem = static_cast<int>(TL::smem);
    cudaError_t e = allow_smem<kern>(smem);
    if (e == cudaSuccess)
        e = launch_kernel(kern, static_cast<unsigned>(heads * x.blocks * x.parts), TL::threads, smem, st, mk, mk, mv, rows,
                          static_cast<uint32_t>(heads), static_cast<int32_t>(x.blocks), wait_ns, source);
    return e != cudaSuccess ? e : launch_attention_split<T, D>(a, st, source.out);
}

}  // namespace gtms
