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
//                       (m, l, O) go to the workspace in fp32 (PrefixRows). The
//                       sequences' own caches: of few sequences, by the split kernel,
//                       which joins its sums with the parts (PrefixParts); of many,
//                       which are short beside the prefix, a chunk to a warp, more parts
//                       to be joined by a last launch. The split kernel spends 6 to 8 us
//                       of a CTA on its start and its joins, whatever the keys are, and
//                       starts when the prefix is done: 64 sequences of 100 to 1024 keys
//                       over a prefix of 8192, 8 key/value heads of 128, 71 us; so 47.
#pragma once

#include "gtms_attention_fwd.cuh"
#include "gtms_attention_split.cuh"
#include "gtms_caches.h"

namespace gtms {

// Tiles [0, prefix_tiles) of an item are the prefix's, those behind them its own.
template <bool FINE>
struct PrefixedCache {
    static constexpr bool prefixed = true, packed = false, fine = FINE;
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

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Shared memory of a warp that works on a chunk: stages of 16 keys and values, the queries.
template <int D, int NT>
struct ChunkWarp {
    static constexpr int ST = 3, R = 8 * NT;
    static constexpr int KC = 2 * (D / 32), VC = 4 * (D / 64);   // 16-byte chunks a lane takes of 16 keys, of their values
    uint4 kv[ST][KC + VC][32];        // [chunk][lane]: every lane reads back what it asked for itself
    uint4 q[R][D / 8];                // chunk x of row r at x ^ r % 8
};

// A chunk of a sequence's own keys to a warp (a CTA), which shares nothing with any other:
// a part more of its rows' sums. Copies run through three stages of 16 keys in shared
// memory, two of them ahead of the products: 8 warps of 26.6 KB to a multiprocessor at head
// dim 128, 16 at 64, have 128 KB in flight, where the 2 to 3 us of a busy memory want 150.
// The keys are the M side of both products (S^T = K Q^T, O^T = V^T P^T), so that a tile is
// 8 rows per NT, which one token's heads fill. P^T comes out of the first product with a
// key to a row and goes into the second with a row to a column: an 8 x 8 transposition.
// Operand layouts as in the split kernel. A maximum is raised only where a score exceeds
// it by 2^8. 64 sequences of 100 to 1024 keys, 8 key/value heads of 128 (147 MB): 30 us by
// itself (4.9 TB/s); as a fixed number of warps that go from chunk to chunk without a
// pause it takes the start of the call 8 to 14 us longer, since whose multiprocessor the
// prefix still has starts late.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(32)
gtms_attention_chunks_kernel(const AttentionArgs a, const PrefixParts out, int32_t chunk, int32_t chunks, int32_t tiles)
{
    using W = ChunkWarp<D, NT>;
    constexpr int R = W::R, ST = W::ST, KC = W::KC;
    constexpr float kRaise = 8.0f;
    extern __shared__ __align__(16) uint4 raw[];
    W& sh = *reinterpret_cast<W*>(raw);
    let_next_launch_start();
    const int lane = threadIdx.x, g = lane >> 2, t = lane & 3;
    const int32_t unit = blockIdx.x / chunks, part = blockIdx.x - unit * chunks, bg = unit / tiles, tile = unit - bg * tiles;
    const int32_t b = bg / a.Hkv, hk = bg - b * a.Hkv, rows = a.group * a.Sq;
    const int32_t off = a.offset(b), L = a.length(b);
    // Keys [0, hi) are kept by row r of the tile: this thread's rows are 8 n + 2 t and the next.
    int32_t hi[NT][2], most = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int32_t r = tile * R + 8 * n + 2 * t + e;
            int32_t c0 = 0;
            hi[n][e] = 0;
            if (r < rows)
                a.kept(off + r / a.group, L, c0, hi[n][e]);
            most = hi[n][e] > most ? hi[n][e] : most;
        }
    most = __reduce_max_sync(0xffffffffu, most);
    const int32_t k0 = part * chunk, k1 = k0 + chunk < most ? k0 + chunk : most;
    if (k0 < k1) {
#pragma unroll
        for (int i = lane; i < R * (D / 8); i += 32) {
            const int32_t r = i / (D / 8), x = i % (D / 8), n = tile * R + r;
            const bool exists = n < rows;
            tc::cp_async16(tc::smem_u32(&sh.q[r][x ^ (r & 7)]),
                           a.q.row<T>(b, hk * a.group + (exists ? n % a.group : 0), exists ? n / a.group : 0) + 8 * x, exists ? 16 : 0);
        }
        const T* kbase = a.k.row<T>(b, hk, 0) + 8 * t;
        const T* vbase = a.v.row<T>(b, hk, 0) + 8 * g;
        auto ask = [&](int32_t key0, int32_t s) {   // a block, a group of its own (an empty one at the end)
            if (key0 < k1) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int32_t c = key0 + 8 * y + g;
                    const bool live = c < k1;
#pragma unroll
                    for (int x = 0; x < D / 32; ++x)
                        tc::cp_async16(tc::smem_u32(&sh.kv[s][y * (D / 32) + x][lane]), kbase + (live ? c : key0) * a.k.ss + 32 * x,
                                       live ? 16 : 0);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int32_t c = key0 + 2 * t + (y & 1) + 8 * (y >> 1);
                    const bool live = c < k1;
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tc::cp_async16(tc::smem_u32(&sh.kv[s][KC + y * (D / 64) + x][lane]), vbase + (live ? c : key0) * a.v.ss + 64 * x,
                                       live ? 16 : 0);
                }
            }
            tc::cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < ST - 1; ++s)
            ask(k0 + 16 * s, s);

        const float c = a.scale * kLog2e;
        float m[NT][2], l[NT][2], o[NT][D / 64][4][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                l[n][e] = 0.0f;
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[n][y][j][e] = o[n][y][j][2 + e] = 0.0f;
            }
        int32_t stage = 0;
        for (int32_t key0 = k0; key0 < k1; key0 += 16, stage = stage == ST - 1 ? 0 : stage + 1) {
            ask(key0 + 16 * (ST - 1), stage == 0 ? ST - 1 : stage - 1);   // into the stage that the last block has left
            asm volatile("cp.async.wait_group %0;" :: "n"(ST - 1) : "memory");
            __syncwarp();   // the queries are other lanes' copies too
            const uint4(&kv)[KC + W::VC][32] = sh.kv[stage];
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s[n][k] = 0.0f;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                const uint4 ka = kv[x][lane], kb = kv[D / 32 + x][lane];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 y = sh.q[8 * n + g][(4 * x + t) ^ g];
                    mma_16816<T>(s[n], ka.x, kb.x, ka.y, kb.y, y.x, y.y);
                    mma_16816<T>(s[n], ka.z, kb.z, ka.w, kb.w, y.z, y.w);
                }
            }
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // key g + 8 (k / 2), row 2 t + k % 2
                    s[n][k] = key0 + g + 8 * (k >> 1) < hi[n][k & 1] ? s[n][k] * c : -INFINITY;
                    raise = raise || s[n][k] > m[n][k & 1] + kRaise;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(m[n][e], fmaxf(s[n][e], s[n][2 + e]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                        const float f = top == -INFINITY ? 1.0f : exp2_approx(m[n][e] - top);
                        m[n][e] = top;
                        l[n][e] *= f;
#pragma unroll
                        for (int y = 0; y < D / 64; ++y)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                o[n][y][j][e] *= f;
                                o[n][y][j][2 + e] *= f;
                            }
                    }
            }
            uint32_t p[NT][2];   // [half of the keys]
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s[n][k] = exp2_approx(s[n][k] - (m[n][k & 1] == -INFINITY ? 0.0f : m[n][k & 1]));
                    l[n][k & 1] += s[n][k];
                }
                // 16 bits, as the products with V take them; l sums them as they were.
                p[n][0] = transpose_8x8(pack2<T>(s[n][0], s[n][1]));
                p[n][1] = transpose_8x8(pack2<T>(s[n][2], s[n][3]));
            }
#pragma unroll
            for (int y = 0; y < D / 64; ++y) {
                uint32_t r[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 v = kv[KC + k * (D / 64) + y][lane];
                    r[k][0] = v.x;
                    r[k][1] = v.y;
                    r[k][2] = v.z;
                    r[k][3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {   // elements 64 y + 8 g + 2 j and the next
                    const uint32_t a0 = __byte_perm(r[0][j], r[1][j], 0x5410), a1 = __byte_perm(r[0][j], r[1][j], 0x7632);
                    const uint32_t a2 = __byte_perm(r[2][j], r[3][j], 0x5410), a3 = __byte_perm(r[2][j], r[3][j], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_16816<T>(o[n][y][j], a0, a1, a2, a3, p[n][0], p[n][1]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
                const int32_t r = tile * R + 8 * n + 2 * t + e;
                if (r < rows) {
                    const int64_t at = (out.parts + part) * out.stride() + out.at(b, hk, r);
                    if (g == 0)
                        out.ml[at] = make_float2(m[n][e], l[n][e]);
#pragma unroll
                    for (int y = 0; y < D / 64; ++y) {
                        float4* to = reinterpret_cast<float4*>(out.o + at * D + 64 * y + 8 * g);
                        to[0] = make_float4(o[n][y][0][e], o[n][y][0][2 + e], o[n][y][1][e], o[n][y][1][2 + e]);
                        to[1] = make_float4(o[n][y][2][e], o[n][y][2][2 + e], o[n][y][3][e], o[n][y][3][2 + e]);
                    }
                }
            }
    }
    // One CTA alone waits for the prefix's launch to end, so that this one ends after it and the next waits for both;
    // the others would hold the places of those that have not started.
    if (blockIdx.x == 0)
        await_last_launch();
}

// The parts of a row, the prefix's and those of its own keys, which follow them: four
// elements a thread, four parts in flight. Where parts are many, a CTA's four warps take
// every fourth one of the same rows and meet in shared memory (one thread that walks over
// all parts waits for memory as often as it has fours of them: 4 x 8 sequences over prefixes
// of 32768 keys, 12 us instead of 6); where they are few or rows many, each has rows of its own
// (88 x 16 rows of 32 heads over prefixes of 1700 keys: the call 133 -> 80 us).
constexpr int kJoinThreads = 128;
template <typename T, int D, bool SHARED>
__global__ void __launch_bounds__(kJoinThreads)
gtms_attention_parts_kernel(const AttentionArgs a, const PrefixParts in, int32_t chunk)
{
    constexpr int LANES = D / 4, ROWS = 32 / LANES, WARPS = SHARED ? kJoinThreads / 32 : 1, N = 4;
    __shared__ float2 ml[WARPS][ROWS];
    __shared__ float4 sums[WARPS][32];
    const int warp = SHARED ? threadIdx.x >> 5 : 0, lane = threadIdx.x & 31, d = lane % LANES * 4;
    const int64_t group = SHARED ? blockIdx.x : blockIdx.x * static_cast<int64_t>(kJoinThreads / 32) + (threadIdx.x >> 5);
    const int64_t x = group * ROWS + lane / LANES;   // (batch, key/value head, row of it)
    const int64_t bg = x / in.per;
    const int32_t r = static_cast<int32_t>(x - bg * in.per), b = static_cast<int32_t>(bg / a.Hkv);
    const int32_t hk = static_cast<int32_t>(bg - static_cast<int64_t>(b) * a.Hkv);
    int32_t c0 = 0, c1 = 0;
    if (b < a.B)
        a.kept(a.offset(b) + r / a.group, a.length(b), c0, c1);
    await_last_launch();
    float top = -INFINITY, l = 0.0f;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float m, float n, float4 e) {
        const float next = fmaxf(top, m), base = next == -INFINITY ? 0.0f : next;
        const float f = exp2_approx(top - base), h = exp2_approx(m - base);
        l = l * f + h * n;
        y = make_float4(y.x * f + h * e.x, y.y * f + h * e.y, y.z * f + h * e.z, y.w * f + h * e.w);
        top = next;
    };
    const int32_t parts = c1 > 0 ? in.parts + (c1 + chunk - 1) / chunk : 0;
    const int64_t i = in.at(b, hk, r), step = in.stride();
    for (int32_t k = warp; k < parts; k += N * WARPS) {
        float2 s[N];
        float4 e[N];
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (k + u * WARPS < parts) {
                s[u] = in.ml[i + (k + u * WARPS) * step];
                e[u] = *reinterpret_cast<const float4*>(in.o + (i + (k + u * WARPS) * step) * D + d);
            }
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (k + u * WARPS < parts)
                add(s[u].x, s[u].y, e[u]);
    }
    if (SHARED) {
        sums[warp][lane] = y;
        if (d == 0)
            ml[warp][lane / LANES] = make_float2(top, l);
        __syncthreads();
        if (warp != 0)
            return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
            add(ml[w][lane / LANES].x, ml[w][lane / LANES].y, sums[w][lane]);
    }
    if (b >= a.B)
        return;
    const float inv = parts > 0 ? 1.0f / l : 0.0f;
    const int32_t h = hk * a.group + r % a.group, row = r / a.group;
    *reinterpret_cast<uint2*>(a.o.row<T>(b, h, row) + d) =
        parts > 0 ? make_uint2(pack2<T>(y.x * inv, y.y * inv), pack2<T>(y.z * inv, y.w * inv)) : make_uint2(0u, 0u);
    if (a.lse && d == 0)
        a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Sq + row] = parts > 0 ? top * 0.6931471805599453f + logf(l) : -INFINITY;
}

// Work items (prefix, head, rows, part of the keys) of the packed rows. The kernel's
// AttentionArgs are those of one batch of G over the prefixes, Sq its packed rows.
struct PrefixRows {
    static constexpr bool prefixed = false, packed = true, fine = false;
    HeadsRef q;
    PrefixArgs p;
    PrefixParts out;
    int32_t Sq, group;
    // Where one tile holds all rows, a CTA's two work on alternate tiles of keys, a part each, instead of one on all of
    // them, waiting for itself (4 x 8 sequences of 8 heads to a key over prefixes of 32768 keys in 8 items each: 51 us,
    // 46 so; in 12: 41, 40).
    bool alternate;

    template <int W>
    struct Item : FwdItem<W> {
        int32_t part;
        bool alternate;

        __device__ __forceinline__ bool has(int w, int32_t t) const
        {
            return FwdItem<W>::has(w, t) && (!alternate || (t & 1) == w);
        }
        __device__ __forceinline__ bool alternating() const { return alternate; }
    };
    template <int W>
    __device__ __forceinline__ void set(Item<W>& it, const AttentionArgs& a, uint32_t item, uint32_t heads, int32_t) const
    {
        const int32_t gh = static_cast<int32_t>(item % heads), rest = static_cast<int32_t>(item / heads);
        const int32_t parts = alternate ? out.parts / 2 : out.parts;   // items
        it.alternate = alternate;
        it.part = rest % parts;
        it.b = gh / a.Hkv;
        it.h = gh - it.b * a.Hkv;
        it.i0 = rest / parts * W * kTile;
        it.off = 0;
        it.L = p.length(it.b);
        const int32_t tiles = (it.L + kTile - 1) / kTile, per = (tiles + parts - 1) / parts;   // of this prefix
        const int32_t lo = it.part * per, hi = lo + per < tiles ? lo + per : tiles;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            // Its first and its last tile, where they alternate those whose number is w modulo 2.
            const int32_t lo_w = alternate ? lo + ((w - lo) & 1) : lo, hi_w = alternate ? hi - ((hi - 1 - w) & 1) : hi;
            const bool any = lo_w < hi_w && (alternate || it.i0 + w * kTile < a.Sq);
            it.lo[w] = any ? lo_w : 0;
            it.hi[w] = any ? hi_w : 0;
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

// Calls of few items and keys have P as two numbers, so that o is its own rounding. One
// rounding of P, the forward kernel's, adds an error of that size, 1.4 times it together;
// but a row's outputs share P's errors, so that over few rows of few keys the figure
// scatters (12 draws each): one row of 36 keys 1.1 to 1.9, 4 rows 1.2 to 1.5, 32 rows 1.24 to
// 1.41. More than 32 items are more rows, more keys even it out within a row (36 rows of 564
// keys 1.34 to 1.45, 4 rows of 2064, packed, 1.25 to 1.46), and those have the one rounding.
// The price of the other (32 rows on the device; through the call 22 to 24 us either way): 36
// keys of head dim 64 7.1 -> 8.3 us, 564 10.3 -> 13.1, of 128 11.8 -> 15.7, 864 15.3 -> 21.5; 2 sequences
// of 16 heads and 128 rows, 32 items too, 11.7 -> 15.2. fp16 spills 184 and 160 bytes there.
constexpr int64_t kFineItems = 32, kFineKeys = 1024;

template <typename T, int D>
cudaError_t launch_prefixed_whole(const AttentionArgs& a, const PrefixArgs& p, cudaStream_t st, uint64_t wait_ns = kAttnWaitNs)
{
    using TL = FwdTile<D>;
    if (!bind_context())
        return cudaErrorUnknown;
    // Without keys no tile is loaded, and q stands in for k and v in the maps.
    const bool keys = a.Skv > 0, shared = p.P > 0;
    HeadsMap mq, mk, mv, mkp, mvp;
    if (!encode_heads<T>(mq, a.q, a.B, a.Hq, a.Sq, D, kTile) ||
        !encode_heads<T>(mk, keys ? a.k : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile) ||
        !encode_heads<T>(mv, keys ? a.v : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile) ||
        !encode_heads<T>(mkp, shared ? p.k : a.q, p.G, a.Hkv, shared ? p.P : 1, D, kTile) ||
        !encode_heads<T>(mvp, shared ? p.v : a.q, p.G, a.Hkv, shared ? p.P : 1, D, kTile))
        return cudaErrorInvalidValue;
    const int32_t blocks = (a.Sq + TL::rows - 1) / TL::rows;
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hq;
    auto launch = [&](auto is_long, auto fine) {
        constexpr auto* kern = gtms_attention_fwd_kernel<T, D, is_long(), PrefixedCache<fine()>>;
        constexpr int smem = static_cast<int>(TL::smem);
        const cudaError_t e = allow_smem<kern>(smem);
        return e != cudaSuccess ? e
                                : launch_kernel(kern, static_cast<unsigned>(heads * blocks), TL::threads, smem, st, mq, mk, mv, a,
                                                static_cast<uint32_t>(heads), blocks, wait_ns,
                                                PrefixedCache<fine()>{mkp, mvp, p});
    };
    // A tile counts as whole even where the prefix ends inside it.
    const int64_t most = static_cast<int64_t>(p.P) + kTile + a.Skv;
    constexpr std::true_type yes;
    constexpr std::false_type no;
    if (heads * blocks <= kFineItems && most <= kFineKeys)
        return launch(no, yes);
    return most > kCarryTerms<T> ? launch(yes, no) : launch(no, no);
}

// How a call's packed rows are dealt out: tiles of rows, parts of the keys; and the
// sequences' own keys.
struct PackedPlan {
    int64_t rows;            // of one prefix and key/value head
    int64_t blocks;          // items of rows
    bool alternate;          // see PrefixRows
    int32_t parts;           // of the keys: items, two parts each where they alternate
    int32_t tile;            // rows of a warp's chunk
    int32_t chunk, chunks;   // keys of a chunk, chunks of a sequence's own cache; 0: the split kernel takes them
    double us;               // of the call, about
};

// Microseconds of an item of rows x keys, and of 128 keys of one (with both CTAs of a
// multiprocessor busy at head dim 64), as measured for the forward kernel.
template <int D>
constexpr double kItemUs = D == 64 ? 4.0 : 5.0;
template <int D>
constexpr double kTileUs = D == 64 ? 1.0 : 1.15;

// Rows of a call up to which a CTA each joins its parts.
constexpr int64_t kJoinRows = 8192;

// Own keys go in chunks of 128 (64 to 256 of them differ by 1 to 5 %), longer ones where a
// cache would make more than 64; long caches of a few sequences, whose chunks would not
// fill the chip, are the split kernel's.
constexpr int32_t kChunk = 128;

// Parts of the prefix: as many as make the call shortest, since the prefix's items and the
// chunks share the chip. Microseconds, measured (parts: time):
//   64 sequences of 100 to 1024 keys, 8 heads of 128, prefix 8192:    4: 47, 8: 49, 12: 53, 16: 57
//   64 sequences of 128 keys, the same:                               4: 38, 8: 27, 12: 27, 16: 36
//   4 x 8 of 300 to 2048, 2 heads of 128 (8 to a key), prefixes 32768: 8: 46, 12: 40, 14: 38, 16: 42
//   24 x 5 rows of 50 to 333, 4 heads of 64, prefix 5003:              4: 18, 8: 14, 12: 15, 16: 15
// A part's keys are below kCarryTerms of either type, so that no sum in an accumulator is long.
template <int D>
PackedPlan packed_plan(const AttentionArgs& a, const PrefixArgs& p)
{
    using TL = FwdTile<D>;
    PackedPlan x;
    x.rows = static_cast<int64_t>(p.n) * a.Sq * a.group;
    x.blocks = (x.rows + TL::rows - 1) / TL::rows;
    x.alternate = TL::W == 2 && x.rows <= kTile;

    const int64_t rows = a.group * int64_t(a.Sq);
    x.tile = rows <= 8 ? 8 : 16;
    const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * ((rows + x.tile - 1) / x.tile);
    int64_t chunk = (static_cast<int64_t>(a.Skv) + 63) / 64;
    chunk = chunk > kChunk ? (chunk + 15) / 16 * 16 : kChunk;
    const int64_t chunks = (static_cast<int64_t>(a.Skv) + chunk - 1) / chunk;
    x.chunk = x.chunks = 0;
    if (units <= INT32_MAX / 64 && chunk <= kCarryTerms<__half> && (units * chunks >= 2 * kChipSms || chunks <= 16)) {
        x.chunk = static_cast<int32_t>(chunk);
        x.chunks = static_cast<int32_t>(chunks);
    }

    const int64_t items = static_cast<int64_t>(p.G) * a.Hkv * x.blocks, slots = int64_t(kChipSms) * TL::ctas;
    const int64_t tiles = p.P > 0 ? (static_cast<int64_t>(p.P) + kTile - 1) / kTile : 1, least = (tiles + 255) / 256;
    // The own keys take the whole chip this long, caches half filled: 5 TB/s, once for each tile of rows.
    const double own = 0.5 * static_cast<double>(units) * a.Skv * D * 4 / 5e6;
    x.parts = 1;
    x.us = 0.0;
    for (int64_t parts = least; parts <= tiles && parts <= least + 31; ++parts) {
        const int64_t turns = (items * parts + slots - 1) / slots, per = (tiles + parts - 1) / parts;
        const double item = kItemUs<D> + (x.alternate ? 0.7 : 1.0) * kTileUs<D> * static_cast<double>(per);
        const double first = static_cast<double>(turns) * item;
        const double both = own + static_cast<double>(items * parts) * item / static_cast<double>(slots);
        const double us = (first > both ? first : both) + 0.1 * first + 3.0 + 0.25 * static_cast<double>(x.alternate ? 2 * parts : parts);
        // A third of the chip is left to the chunks from the start (64 x 128 keys, prefix 8192: 12 parts, 96 of 152
        // multiprocessors, 27 us; 13, 104 of them: 36).
        if (parts == least || (us < x.us && (x.chunks == 0 || 3 * items * parts <= 2 * slots))) {
            x.us = us;
            x.parts = static_cast<int32_t>(parts);
        }
    }
    return x;
}

// Whether to pack, by the time that both forms take (see prefer_split). Its two launches
// more cost the host as much as some tiles cost the chip: 4 sequences, 16 / 4 heads of 64, a
// prefix of 500 keys, 8 us on the device either way, through the call 34 us packed, 25 whole.
constexpr double kLaunchesUs = 4.0;

template <int D>
bool prefer_packed(const AttentionArgs& a, const PrefixArgs& p, const PackedPlan& x)
{
    if (p.P == 0 || static_cast<int64_t>(a.group) * a.Sq > kSplitMaxRows || x.rows > (1 << 24) ||
        x.blocks * x.parts * p.G * a.Hkv > INT32_MAX)
        return false;
    const double items = static_cast<double>(a.B) * a.Hq * ((a.Sq + FwdTile<D>::rows - 1) / FwdTile<D>::rows);
    const double loads = items / (static_cast<double>(kChipSms) * FwdTile<D>::ctas);
    const int64_t tiles = (static_cast<int64_t>(p.P) + kTile - 1) / kTile + (static_cast<int64_t>(a.Skv) + kTile - 1) / kTile;
    const double whole = (loads > 1.0 ? loads : 1.0) * (kItemUs<D> + kTileUs<D> * static_cast<double>(tiles));
    return x.us + kLaunchesUs < whole;
}

inline uint64_t packed_bytes(const AttentionArgs& a, const PrefixArgs& p, const PackedPlan& x, int64_t D)
{
    return static_cast<uint64_t>((x.alternate ? 2 : 1) * x.parts + x.chunks) * p.G * a.Hkv * x.rows * (D * 4 + 8);
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
    source.alternate = x.alternate;
    source.out.parts = x.alternate ? 2 * x.parts : x.parts;
    source.out.ml = reinterpret_cast<float2*>(source.out.o + (source.out.parts + x.chunks) * heads * x.rows * D);
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
    if (e != cudaSuccess || x.chunks == 0)
        return e != cudaSuccess ? e : launch_attention_split<T, D>(a, st, source.out);
    auto chunks = [&](auto nt) {
        constexpr auto* kern = gtms_attention_chunks_kernel<T, D, nt()>;
        constexpr int smem = static_cast<int>(sizeof(ChunkWarp<D, nt()>));
        const int64_t tiles = (a.group * int64_t(a.Sq) + x.tile - 1) / x.tile, items = static_cast<int64_t>(a.B) * a.Hkv * tiles * x.chunks;
        const cudaError_t err = allow_smem<kern>(smem);
        return err != cudaSuccess ? err
                                  : launch_beside_last(true, kern, static_cast<unsigned>(items), 32, smem, st, a, source.out,
                                                       x.chunk, x.chunks, static_cast<int32_t>(tiles));
    };
    e = x.tile == 8 ? chunks(std::integral_constant<int, 1>()) : chunks(std::integral_constant<int, 2>());
    if (e != cudaSuccess)
        return e;
    const int64_t all = static_cast<int64_t>(a.B) * a.Hkv * source.out.per;
    auto join = [&](auto shared) {
        constexpr int rows_of_cta = 128 / D * (shared() ? 1 : kJoinThreads / 32);
        return launch_beside_last(true, gtms_attention_parts_kernel<T, D, shared()>,
                                  static_cast<unsigned>((all + rows_of_cta - 1) / rows_of_cta), kJoinThreads, 0, st, a, source.out,
                                  x.chunk);
    };
    return source.out.parts + x.chunks > 8 && all <= kJoinRows ? join(std::true_type()) : join(std::false_type());
}

}  // namespace gtms
