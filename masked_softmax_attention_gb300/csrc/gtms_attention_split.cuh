// gtms_attention_split.cuh -- attention forward for few query rows over many keys
// (new tokens over a cache), the keys split over the CTAs of a cluster.
//
// What bounds it is one read of the live keys and values. The rows of the query
// heads that share a key/value head are packed into tiles of 16, so that every
// key is read once for all of them. A warp takes 16 keys at a time straight from
// memory into the registers that the tensor-core instruction reads them from, the
// next 16 in flight while it works, with a running maximum and sum per row; no
// shared memory and no barrier until the end, where the warps' (m, l, O) are
// joined in shared memory and the CTAs' through the cluster's. One launch, no
// workspace.
//
// Operand layouts. A dot product does not care in which order its terms come, so
// the k indices of S = Q K^T are dealt out such that a thread's share of a key is
// 16 contiguous bytes (lane 4 g + t: key g, elements 32 x + 8 t .. + 7), and q is
// dealt out likewise. For O += P V a thread reads 16 contiguous bytes (elements
// 64 y + 8 g .. + 7) of the keys 2t, 2t + 1, 2t + 8, 2t + 9 and pairs up the keys
// with byte permutations: column n of product j is element 64 y + 8 n + j.
#pragma once

#include <atomic>
#include <cooperative_groups.h>

#include "gtms_attention_fwd.cuh"

namespace gtms {

constexpr int kSplitRows = 16, kSplitKeys = 16;   // rows of a tile; keys a warp takes at a time
// Batches are taken longest first where the grid takes more than one turn, up to this
// many of them: every CTA ranks the lengths by itself (64 sequences of 700 to 8192 keys,
// 8 key/value heads, head dim 128: 210 -> 187 us; 24 of 819 to 8192: 90 -> 75, of equal
// lengths 135 -> 136).
constexpr int kSplitOrdered = 256;
constexpr int kSplitMaxCluster = 8;               // the largest portable cluster
constexpr int kSplitLarge[] = {16, 12, 10};          // larger ones, where the chip has room for all of them at once
// Warps of a CTA: four, three CTAs to a multiprocessor; eight and one CTA where all
// clusters then run at once (one token, 10 key/value heads of 8192 keys, 80 CTAs: head
// dim 128 23.8 -> 17.5 us, 64 16.5 -> 11.6; 16 heads, whose 128 CTAs do not: 27.9, 32.4).

template <int D, int WARPS>
struct SplitShared {
    uint4 q[kSplitRows][D / 8 + 1];                  // + 1: rows start in different banks
    float m[WARPS][kSplitRows], l[WARPS][kSplitRows];
    float o[WARPS][kSplitRows][D + 4];
    float cta_m[kSplitRows], cta_l[kSplitRows];      // joined over the warps; o[0] then holds the CTA's O
    int32_t length[kSplitOrdered], batch;            // of all batches; the one this CTA takes
};

// What the rows' sums are joined with at the end: nothing, or the parts of a shared
// prefix (gtms_shared_prefix.cuh).
struct NoParts {
    static constexpr bool any = false;
};

// LONG: where a warp may have more than kCarryTerms keys (code of its own, whose registers
// the others would spill for).
template <typename T, int D, int WARPS, bool LONG, typename Parts = NoParts>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 4 ? 3 : 1)
gtms_attention_split_kernel(const AttentionArgs a, int32_t tiles, int32_t ordered, const Parts parts)
{
    namespace cg = cooperative_groups;
    constexpr int THREADS = 32 * WARPS;
    const cg::cluster_group cluster = cg::this_cluster();
    const int32_t ranks = static_cast<int32_t>(cluster.num_blocks()), rank = static_cast<int32_t>(cluster.block_rank());
    extern __shared__ __align__(128) uint8_t smem_raw[];
    using Shared = SplitShared<D, WARPS>;
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    const int64_t unit = blockIdx.x / ranks;
    const int32_t tile = static_cast<int32_t>(unit % tiles);
    const int64_t bg = unit / tiles;
    int32_t b = static_cast<int32_t>(bg / a.Hkv);
    const int32_t hk = static_cast<int32_t>(bg - static_cast<int64_t>(b) * a.Hkv);
    if (ordered) {   // the b-th longest of the batches
        for (int32_t i = threadIdx.x; i < a.B; i += THREADS)
            sh.length[i] = a.length(i);
        __syncthreads();
        for (int32_t i = threadIdx.x; i < a.B; i += THREADS) {
            const int32_t mine = sh.length[i];
            int32_t longer = 0;
            for (int32_t j = 0; j < a.B; ++j)
                longer += sh.length[j] > mine || (sh.length[j] == mine && j < i);
            if (longer == b)
                sh.batch = i;
        }
        __syncthreads();
        b = sh.batch;
    }
    const int32_t off = a.offset(b), L = a.length(b), rows = a.group * a.Sq;
    // Row r of a tile is query row r / group of shared head r % group: neighbouring rows keep nearly the same keys.
    auto head_of = [&](int32_t r) { return hk * a.group + (tile * kSplitRows + r) % a.group; };
    auto row_of = [&](int32_t r) { return (tile * kSplitRows + r) / a.group; };
    auto exists = [&](int32_t r) { return tile * kSplitRows + r < rows; };

    int32_t c0[2] = {0, 0}, c1[2] = {0, 0}, lo = INT32_MAX, hi = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int32_t r = g + 8 * k;
        if (exists(r))
            a.kept(off + row_of(r), L, c0[k], c1[k]);
        if (c0[k] < c1[k]) {
            lo = c0[k] < lo ? c0[k] : lo;
            hi = c1[k] > hi ? c1[k] : hi;
        }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        const int32_t x = __shfl_xor_sync(0xffffffffu, lo, o), y = __shfl_xor_sync(0xffffffffu, hi, o);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
    }

    // q into shared memory; rows that do not exist are zero.
    for (int32_t i = threadIdx.x; i < kSplitRows * (D / 8); i += THREADS) {
        const int32_t r = i / (D / 8), x = i % (D / 8);
        sh.q[r][x] = exists(r) ? *(reinterpret_cast<const uint4*>(a.q.row<T>(b, head_of(r), row_of(r))) + x) : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();

    // This CTA's share of the 16-key blocks, contiguous; its warps take them in turn.
    const int32_t first = hi > 0 ? lo / kSplitKeys : 0, blocks = hi > 0 ? (hi + kSplitKeys - 1) / kSplitKeys - first : 0;
    const int32_t per = (blocks + ranks - 1) / ranks;
    const int32_t end = first + (per * (rank + 1) < blocks ? per * (rank + 1) : blocks);
    int32_t blk = first + per * rank + warp;

    const T* kbase = a.k.row<T>(b, hk, 0) + 8 * t;
    const T* vbase = a.v.row<T>(b, hk, 0) + 8 * g;
    uint4 kr[2][D / 32], vr[4][D / 64];
    auto load_k = [&](int32_t n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int32_t key = n * kSplitKeys + 8 * k + g;
            const bool use = n < end && key >= lo && key < hi;
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
                kr[k][x] = load_once(kbase + key * a.k.ss + 32 * x, use);
        }
    };
    auto load_v = [&](int32_t n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int32_t key = n * kSplitKeys + 2 * t + (k & 1) + 8 * (k >> 1);
            const bool use = n < end && key >= lo && key < hi;
#pragma unroll
            for (int y = 0; y < D / 64; ++y)
                vr[k][y] = load_once(vbase + key * a.v.ss + 64 * y, use);
        }
    };

    const float c = a.scale * kLog2e;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float o[D / 64][8][4];
#pragma unroll
    for (int y = 0; y < D / 64; ++y)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[y][j][k] = 0.0f;

    // Long sums (see kCarryTerms): the warp's O is added up in fp32 in its place in shared
    // memory, at the maxima that stand in sh.m.
    constexpr int kCarryBlocks = kCarryTerms<T> / kSplitKeys;
    const int32_t start = blk;
    auto kept_o = [&](int y, int h, int n, int j) { return reinterpret_cast<float4*>(&sh.o[warp][g + 8 * h][64 * y + 16 * t + 8 * n + j]); };
    auto add_kept = [&] {   // o += what is kept
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float f = m[h] == -INFINITY ? 0.0f : exp2_approx(sh.m[warp][g + 8 * h] - m[h]);
#pragma unroll
            for (int y = 0; y < D / 64; ++y)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const float4 x = *kept_o(y, h, n, j);
                        o[y][j][2 * h + n] += f * x.x;
                        o[y][j + 1][2 * h + n] += f * x.y;
                        o[y][j + 2][2 * h + n] += f * x.z;
                        o[y][j + 3][2 * h + n] += f * x.w;
                    }
        }
    };

    load_k(blk);
    load_v(blk);
    for (; blk < end; blk += WARPS) {
        if (LONG && (blk - start) % (kCarryBlocks * WARPS) == 0 && blk != start) {
            if (blk - start > kCarryBlocks * WARPS)
                add_kept();
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (t == 0)
                    sh.m[warp][g + 8 * h] = m[h];
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int j = 0; j < 8; j += 4) {
                            *kept_o(y, h, n, j) = make_float4(o[y][j][2 * h + n], o[y][j + 1][2 * h + n], o[y][j + 2][2 * h + n],
                                                              o[y][j + 3][2 * h + n]);
                            o[y][j][2 * h + n] = o[y][j + 1][2 * h + n] = o[y][j + 2][2 * h + n] = o[y][j + 3][2 * h + n] = 0.0f;
                        }
            }
            __syncwarp();
        }
        float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            const uint4 qa = sh.q[g][4 * x + t], qb = sh.q[g + 8][4 * x + t];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                mma_16816<T>(s[k], qa.x, qb.x, qa.y, qb.y, kr[k][x].x, kr[k][x].y);
                mma_16816<T>(s[k], qa.z, qb.z, qa.w, qb.w, kr[k][x].z, kr[k][x].w);
            }
        }
        load_k(blk + WARPS);
        const int32_t key0 = blk * kSplitKeys + 2 * t;
        uint32_t p[2][2];   // [row half][key half]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int32_t key = key0 + (k & 1) + 8 * (k >> 1);
                x[k] = key >= c0[h] && key < c1[h] ? s[k >> 1][2 * h + (k & 1)] * c : -INFINITY;
            }
            float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > m[h]) {
                const float f = exp2_approx(m[h] - top);   // 0 from -inf
                m[h] = top;
                l[h] *= f;
#pragma unroll
                for (int y = 0; y < D / 64; ++y)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        o[y][j][2 * h] *= f;
                        o[y][j][2 * h + 1] *= f;
                    }
            }
            const float shift = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = exp2_approx(x[k] - shift);
                l[h] += x[k];
            }
            // 16 bits, as the products with V take them; l sums them as they were.
            p[h][0] = pack2<T>(x[0], x[1]);
            p[h][1] = pack2<T>(x[2], x[3]);
        }
#pragma unroll
        for (int y = 0; y < D / 64; ++y) {
            const uint32_t r[4][4] = {{vr[0][y].x, vr[0][y].y, vr[0][y].z, vr[0][y].w}, {vr[1][y].x, vr[1][y].y, vr[1][y].z, vr[1][y].w},
                                      {vr[2][y].x, vr[2][y].y, vr[2][y].z, vr[2][y].w}, {vr[3][y].x, vr[3][y].y, vr[3][y].z, vr[3][y].w}};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                mma_16816<T>(o[y][j], p[0][0], p[1][0], p[0][1], p[1][1], __byte_perm(r[0][j / 2], r[1][j / 2], sel),
                             __byte_perm(r[2][j / 2], r[3][j / 2], sel));
            }
        }
        load_v(blk + WARPS);
    }

    if (LONG && blk - start > kCarryBlocks * WARPS) {
        add_kept();
        __syncwarp();   // sh.m is written anew
    }

    // Join the warps: row sums over the quad, then every warp brings its O to the CTA's maximum.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) {
            sh.m[warp][g + 8 * h] = m[h];
            sh.l[warp][g + 8 * h] = l[h];
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t r = g + 8 * h;
        float top = sh.m[0][r];
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
            top = fmaxf(top, sh.m[w][r]);
        const float base = top == -INFINITY ? 0.0f : top, f = exp2_approx(m[h] - base);
        if (warp == 0 && t == 0) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                sum += sh.l[w][r] * exp2_approx(sh.m[w][r] - base);
            sh.cta_m[r] = top;
            sh.cta_l[r] = sum;
        }
#pragma unroll
        for (int y = 0; y < D / 64; ++y)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4*>(&sh.o[warp][r][64 * y + 16 * t + 8 * n + j]) =
                        make_float4(o[y][j][2 * h + n] * f, o[y][j + 1][2 * h + n] * f, o[y][j + 2][2 * h + n] * f,
                                    o[y][j + 3][2 * h + n] * f);
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < kSplitRows * D; i += THREADS) {
        float sum = sh.o[0][i / D][i % D];
#pragma unroll
        for (int w = 1; w < WARPS; ++w)
            sum += sh.o[w][i / D][i % D];
        sh.o[0][i / D][i % D] = sum;
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();

    if constexpr (Parts::any)
        await_last_launch();   // which wrote them

    // Join the CTAs: each writes its share of the rows' element pairs.
    for (int32_t i = rank * THREADS + threadIdx.x; i < kSplitRows * (D / 2); i += ranks * THREADS) {
        const int32_t r = i / (D / 2), d = 2 * (i % (D / 2));
        if (!exists(r))
            break;   // rows come in order
        float top = -INFINITY;
        for (int32_t k = 0; k < ranks; ++k)
            top = fmaxf(top, *cluster.map_shared_rank(&sh.cta_m[r], k));
        int32_t k0, k1;
        a.kept(off + row_of(r), L, k0, k1);
        const bool live = k0 < k1;
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f, x = 0.0f, y = 0.0f;
        for (int32_t k = 0; k < ranks && live; ++k) {
            const float f = exp2_approx(*cluster.map_shared_rank(&sh.cta_m[r], k) - base);
            const float2 e = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&sh.o[0][r][d], k));
            sum += f * *cluster.map_shared_rank(&sh.cta_l[r], k);
            x += f * e.x;
            y += f * e.y;
        }
        if constexpr (Parts::any)
            if (live)
                parts.template add<D>(b, hk, tile * kSplitRows + r, d, top, sum, x, y);
        const float inv = live ? 1.0f / sum : 0.0f;
        *reinterpret_cast<uint32_t*>(a.o.row<T>(b, head_of(r), row_of(r)) + d) = live ? pack2<T>(x * inv, y * inv) : 0u;
        if (a.lse && d == 0)
            a.lse[(static_cast<int64_t>(b) * a.Hq + head_of(r)) * a.Sq + row_of(r)] =
                live ? top * 0.6931471805599453f + logf(sum) : -INFINITY;
    }
    if (ranks > 1)
        cluster.sync();   // the others may still be reading this CTA's shared memory
}

// CTAs that share a unit's keys: until there are about four to a multiprocessor, but
// every warp of four is left two blocks of keys.
inline int split_ranks(int64_t units, int64_t keys, int nsm)
{
    int ranks = 1;
    while (ranks < kSplitMaxCluster && units * ranks < 4 * nsm && ranks * int64_t(16) * kSplitKeys <= keys)
        ranks *= 2;
    return ranks;
}

inline int64_t split_units(const AttentionArgs& a)
{
    return static_cast<int64_t>(a.B) * a.Hkv * ((static_cast<int64_t>(a.group) * a.Sq + kSplitRows - 1) / kSplitRows);
}

// Whether to split: always where the rows of a key/value head fill one tile, so that
// the keys are read once; otherwise where its CTAs (64 keys in 1 to 2.3 us, three to a
// multiprocessor) take less time than those of the tensor-memory kernel (128 keys in 1
// to 1.15 us), which walk over all keys by themselves (128 rows of one head at head
// dim 64, 256 at 128). Microseconds, measured (bf16, keys at least half filled; split /
// tensor-memory kernel):
//   32 / 8 heads d 128, 8192 keys, 1 sequence:   8 tokens 23 / 77, 32: 47 / 77, 48: 70 / 77, 64: 103 / 77
//   the same, 32768 keys:  32 tokens 155 / 288, 64: 344 / 289
//   the same, 4096 keys:   4 sequences, 8 tokens 26 / 42, 16: 53 / 42;  16 sequences, 8: 83 / 121, 16: 143 / 123
//   8 / 8 heads d 128, 2000 keys, 100 tokens, 2 sequences: 34 / 24
//   16 / 16 heads d 64, 4096 keys, 32 tokens:    1 sequence 12 / 37, 8: 47 / 39
//   8 / 8 heads d 64, 33 of 33 rows, 32 sequences: 13 / 7;  200 rows, 4096 keys, 1 sequence: 31 / 37
//   4 / 1 heads d 64, 8071 keys, 212 tokens, 1 sequence: 24 / 69;  2 / 1 heads d 128, 7381 keys, 316 tokens, 2: 42 / 80
//   4 / 1 heads d 128, 3162 keys, 791 tokens, 3 sequences: 102 / 39
constexpr int64_t kSplitMaxRows = 4096;   // of a key/value head: more are never better split

// Keys that the rows of a call keep at most.
inline int32_t split_keys(const AttentionArgs& a)
{
    return a.mask_kind == GTMS_MASK_SLIDING_WINDOW && a.window + a.Sq < a.Skv ? a.window + a.Sq : a.Skv;
}

template <int D>
bool prefer_split(const AttentionArgs& a)
{
    const int64_t rows = static_cast<int64_t>(a.group) * a.Sq;
    if (rows <= kSplitRows)
        return true;
    const int nsm = device_sms();
    if (rows > kSplitMaxRows || nsm <= 0)
        return false;
    const int64_t keys = split_keys(a);
    const int64_t units = split_units(a), ranks = split_ranks(units, keys, nsm);
    const double turns = static_cast<double>(units * ranks) / (3 * nsm);   // of three CTAs to a multiprocessor
    const double block = turns > 1.0 ? (D == 64 ? 1.3 : 2.3) : (D == 64 ? 1.0 : 1.8);
    const double split = (turns > 1.0 ? turns : 1.0) * (6.0 + block * static_cast<double>((keys + ranks * 64 - 1) / (ranks * 64)));
    const double items = static_cast<double>(a.B) * a.Hq * ((a.Sq + FwdTile<D>::rows - 1) / FwdTile<D>::rows);
    const double loads = items / (static_cast<double>(nsm) * FwdTile<D>::ctas);
    const double whole = (loads > 1.0 ? loads : 1.0) * (5.0 + (D == 64 ? 1.0 : 1.15) * static_cast<double>((keys + 127) / 128));
    return split < whole;
}

template <int WARPS>
struct SplitConfig {
    template <int D>
    static constexpr int smem = static_cast<int>(sizeof(SplitShared<D, WARPS>));
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};

    // beside_last: may start while the last launch still runs (see await_last_launch).
    SplitConfig(int64_t ctas, int ranks, int bytes, cudaStream_t st, bool beside_last = false)
    {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        cfg.blockDim = dim3(32 * WARPS);
        cfg.dynamicSmemBytes = bytes;
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = beside_last ? 2 : 1;
    }
};

// Clusters of `ranks` CTAs that the current device runs at once: fewer
// than its multiprocessors would hold, since a cluster keeps to one part of the chip,
// and not the same on every chip. Asked once per device and process; 0 where it cannot be.
template <typename T, int D, int WARPS>
int clusters_at_once(int ranks)
{
    static std::atomic<int> known[64][32];   // plus one; 0: not asked yet
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    if (dev < 64 && (n = known[dev][ranks].load(std::memory_order_relaxed)) > 0)
        return n - 1;
    constexpr int smem = SplitConfig<WARPS>::template smem<D>;
    const SplitConfig<WARPS> cfg(ranks, ranks, smem, nullptr);
    if (allow_smem<gtms_attention_split_kernel<T, D, WARPS, false>, true>(smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, gtms_attention_split_kernel<T, D, WARPS, false>, &cfg.cfg) != cudaSuccess) {
        cudaGetLastError();   // no such clusters here
        n = 0;
    }
    if (dev < 64)
        known[dev][ranks].store(n + 1, std::memory_order_relaxed);
    return n;
}

// Few units over many keys leave most of the chip's memory pipes idle with clusters of
// 8: larger ones, if they all run at once, from this many keys on (two blocks to each
// of 8 warps of 16 CTAs). bf16, one token, key/value heads of four query heads each:
//   eight warps to a CTA, head dim 128: 8 heads of 32768 keys 46 us with clusters of 8,
//     36 of 12 (54 of 16, which do not all run at once); 13 of 8192 18.0, 17.2 of 10;
//     1 of 16384 24, 16 of 16; head dim 64: 4 of 16384 16.3, 11.4, of 4200 8.0, 7.4
//   four warps, head dim 128, 8192 keys: 16 heads 27.5, 22.1 of 16; 28 heads 30.0, 28.1
//     of 12; 38 heads 36.1, 32.9 of 10; head dim 64: 16 heads 18.1, 14.2
constexpr int64_t kSplitLargeKeys = 4096;

// Somewhat smaller ones, where the clusters of 8 would need a second turn and these do
// not: 64 heads of 8192 keys, head dim 128, 65.4 -> 49.0 us (41.1, 40.5 where the lengths
// spread from 819 on), 80 heads 71.8 -> 57.1 (48.2, 45.7); head dim 64, 64 heads 40.7 ->
// 28.7. Below 5 spread lengths lose more than equal ones win (128 heads, 8 -> 3: 107.8,
// 87.5; 69.7, 77.8).
constexpr int kSplitSmaller[] = {6, 5};

template <typename T, int D, int WARPS, bool LONG, typename Parts>
cudaError_t launch_attention_split_k(const AttentionArgs& a, int64_t ctas, int ranks, cudaStream_t st, const Parts& parts)
{
    constexpr int smem = SplitConfig<WARPS>::template smem<D>;
    const cudaError_t e = allow_smem<gtms_attention_split_kernel<T, D, WARPS, LONG, Parts>, true>(smem);
    if (e != cudaSuccess)
        return e;
    SplitConfig<WARPS> cfg(ctas, ranks, smem, st, Parts::any);
    const int32_t tiles = static_cast<int32_t>((static_cast<int64_t>(a.group) * a.Sq + kSplitRows - 1) / kSplitRows);
    const int32_t ordered = WARPS == 4 && ctas > 3 * device_sms() && a.B > 1 && a.B <= kSplitOrdered;
    return cudaLaunchKernelEx(&cfg.cfg, gtms_attention_split_kernel<T, D, WARPS, LONG, Parts>, a, tiles, ordered, parts);
}

template <typename T, int D, int WARPS, typename Parts>
cudaError_t launch_attention_split_w(const AttentionArgs& a, int64_t ctas, int ranks, cudaStream_t st, const Parts& parts)
{
    // A warp takes every WARPS-th of its CTA's blocks, of which the keys can make one more than an even share.
    const bool is_long = split_keys(a) / (ranks * WARPS) + 2 * kSplitKeys > kCarryTerms<T>;
    return is_long ? launch_attention_split_k<T, D, WARPS, true>(a, ctas, ranks, st, parts)
                   : launch_attention_split_k<T, D, WARPS, false>(a, ctas, ranks, st, parts);
}

// The clusters go by the keys that the rows keep, not by the cache: under a sliding
// window the CTAs without keys would only make more turns of it (one token over 16384
// keys, window 256: 128 key/value heads of 128, clusters of 8 24.1 us, of 2 10.5; 64:
// 18.5, 7.8). Where all clusters run at once a window's warps are left with one block of
// keys instead of two (8 heads of 128, window 256: 7.8 us with clusters of 2, 6.9 of 4,
// 7.1 of 8; 32 heads 8.4, 7.5, 7.7).
template <typename T, int D, typename Parts = NoParts>
cudaError_t launch_attention_split(const AttentionArgs& a, cudaStream_t st, const Parts& parts = Parts())
{
    const int nsm = device_sms();
    if (nsm <= 0)
        return cudaErrorUnknown;
    const int64_t units = split_units(a), keys = split_keys(a);
    int ranks = split_ranks(units, keys, nsm);
    if (keys < a.Skv) {
        const int more = split_ranks(units, 2 * keys, nsm);
        if (units <= clusters_at_once<T, D, 4>(more))
            ranks = more;
    }
    if (units * ranks > INT32_MAX)
        return cudaErrorNotSupported;
    const bool large = keys >= kSplitLargeKeys;
    for (int r : kSplitLarge)
        if (large && units <= clusters_at_once<T, D, 8>(r))
            return launch_attention_split_w<T, D, 8>(a, units * r, r, st, parts);
    if (units <= clusters_at_once<T, D, 8>(ranks))
        return launch_attention_split_w<T, D, 8>(a, units * ranks, ranks, st, parts);
    for (int r : kSplitLarge)
        if (large && units <= clusters_at_once<T, D, 4>(r))
            return launch_attention_split_w<T, D, 4>(a, units * r, r, st, parts);
    if (ranks == kSplitMaxCluster && units > clusters_at_once<T, D, 4>(ranks))
        for (int r : kSplitSmaller)
            if (units <= clusters_at_once<T, D, 4>(r))
                return launch_attention_split_w<T, D, 4>(a, units * r, r, st, parts);
    return launch_attention_split_w<T, D, 4>(a, units * ranks, ranks, st, parts);
}

}  // namespace gtms
