// gtms_key_weights_tc.cuh -- the weight that each key of a cache received, on the tensor
// cores: many query rows, or some rows over many keys.
//
//   w_c = sum over the query heads of a key/value head and rows i with c in K(i) of
//         exp(scale q_i . k_c - lse_i)
//
// The transposed product S = K Q^T has a key to a row, so that the thread that owns a
// row of S in tensor memory sums its exponentials by itself: no maximum, no exchange,
// nothing written back. Two tiles of 128 keys stay in shared memory while the column
// tiles of the query rows that keep any of them stream past.
// The rows of the heads that share the keys are packed side by side (a 5-D map: element,
// head, row, key/value head, batch), so that one new token fills as many columns as it
// has heads, and a window's or a causal mask's kept columns of a key are one range.
// Roles:
//   deal (1 warp)    the work items (see ItemSlot);
//   load (1 warp)    TMA: the key tiles into one ring, the column tiles into another;
//   shift (1 warp)   -lse of the columns, in base 2, -infinity for those that do not count;
//   MMA (1 warp)     S of each key tile, held twice, so that the next column tile's
//                    products run while this one's exponentials do;
//   sum (16 warps)   four to a key tile and half of its columns; the halves meet once a block.
// Where few items make the grid (short caches of few heads), their rows are cut into
// parts, whose sums a second launch adds in order.
// What bounds it: the hand-offs of a column tile, about 2100 cycles, beside 1024 of its products
// and as many of its exponentials (tensor cores and special-function units 51 % busy each):
// [4,32/8,4096,128] bf16, causal, lengths 2500 to 4096, 179 us, 1030 TFLOP/s of kept pairs;
// timed on copies that leave them out, 154 without the exponentials, 119 without products and
// loads of queries either. Few rows over many keys: one read of the keys and the items'
// starts: the last 32 rows of 8 sequences over 16384 keys, 47 us, 4.5 TB/s.
#pragma once

#include "gtms_attention_tc.cuh"
#include "gtms_caches.h"

namespace gtms {

template <int D>
struct KeyTile {
    static constexpr int W = 2, keys = W * kTile;                          // key tiles and keys of a work item
    static constexpr int NK = D == 64 ? 6 : 3, ST = D == 64 ? 4 : 3;       // stages of the rings of key and column tiles
    static constexpr int sum_warps = 16, mma_warp = 16, load_warp = 17, shift_warp = 18, deal_warp = 19, threads = 640;
    static constexpr uint32_t bytes = kTile * D * 2, box = kTile * 128;    // a 128-row tile, 64 columns of it
    static constexpr uint32_t off_q = NK * bytes;
    static constexpr uint32_t smem = off_q + ST * bytes + 1024;            // slack to align the base
    static constexpr int tmem = 512;                                       // two S of each key tile
    static_assert(smem <= 226 * 1024, "shared memory of a CTA");
};

// How query rows become columns: `heads` shared heads (all, or 128 of more) of `rows` rows to a tile.
struct KeyColumns {
    int32_t heads, rows, head_tiles;
    int32_t mb;   // of the map of q: 0 where one batch serves all (see HeadsMap)
};

inline KeyColumns key_columns(int32_t group)
{
    KeyColumns c;
    c.heads = group < kTile ? group : kTile;
    c.rows = kTile / c.heads;
    c.head_tiles = (group + c.heads - 1) / c.heads;
    c.mb = 1;
    return c;
}

// Blocks [block0, block1) of 256 keys of one key/value head, and a part of the rows
// that keep any of them (parts only of single blocks).
struct KeyItem {
    int32_t b, hk, off, L, block0, block1, part;

    __device__ __forceinline__ void set(const AttentionArgs& a, uint32_t item, uint32_t heads, int32_t per, int32_t parts)
    {
        const int32_t bg = static_cast<int32_t>(item % heads), rest = static_cast<int32_t>(item / heads);
        const int32_t blocks = (a.Skv + 2 * kTile - 1) / (2 * kTile);
        part = rest % parts;
        block0 = rest / parts * per;
        block1 = block0 + per < blocks ? block0 + per : blocks;
        b = bg / a.Hkv;
        hk = bg - b * a.Hkv;
        off = a.offset(b);
        L = a.length(b);
    }
};

// What an item has to do for one block: rows [i0, i1) keep any of its keys; this part
// takes their column tiles from row i, head j on, `tiles` of them.
struct KeyRange {
    int32_t i0, i1, i, j, tiles;

    __device__ __forceinline__ KeyRange(const AttentionArgs& a, const KeyColumns& col, const KeyItem& it, int32_t block,
                                        int32_t parts)
    {
        const int32_t key0 = block * (2 * kTile), last = (key0 + 2 * kTile < it.L ? key0 + 2 * kTile : it.L) - 1;
        i0 = it.off < 0 ? -it.off : 0;
        i1 = it.L - it.off < a.Sq ? it.L - it.off : a.Sq;
        if (a.mask_kind != GTMS_MASK_LENGTH && key0 - it.off > i0)
            i0 = key0 - it.off;
        if (a.mask_kind == GTMS_MASK_SLIDING_WINDOW && last + a.window - it.off < i1)
            i1 = last + a.window - it.off;
        i = i0;
        j = tiles = 0;
        if (key0 >= it.L || i0 >= i1)
            return;
        const int32_t all = (i1 - i0 + col.rows - 1) / col.rows * col.head_tiles;
        if (parts == 1) {
            tiles = all;
            return;
        }
        const int32_t per = (all + parts - 1) / parts, t0 = it.part * per < all ? it.part * per : all;
        tiles = t0 + per < all ? per : all - t0;
        i = i0 + t0 / col.head_tiles * col.rows;
        j = t0 % col.head_tiles * col.heads;
    }
    __device__ __forceinline__ void next(const KeyColumns& col)
    {
        j += col.heads;
        if (j >= col.heads * col.head_tiles) {
            j = 0;
            i += col.rows;
        }
    }
};

template <int D>
struct KeyShared {
    using TL = KeyTile<D>;
    uint64_t kfull[TL::NK], kempty[TL::NK], qfull[TL::ST], qempty[TL::ST];
    // S and the shifts are held twice, and one barrier a key tile says that both have come.
    uint64_t sfull[2][TL::W], sempty[2][TL::W], hempty[2], rfull[TL::W], rempty[TL::W], mma_done;
    ItemSlot<KeyItem> items;
    __align__(16) float shift[2][kTile];
    float half[TL::W][kTile];
    uint32_t tmem_slot;
    int flag;
};

template <typename T, int D>
__global__ void __launch_bounds__(KeyTile<D>::threads, 1)
gtms_key_weights_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ HeadsMap mk,
                        const __grid_constant__ KeyWeightsArgs kw, const KeyColumns col, uint32_t heads, int32_t per,
                        int32_t parts, uint64_t wait_ns)
{
    using TL = KeyTile<D>;
    constexpr int W = TL::W, NK = TL::NK, ST = TL::ST;
    const AttentionArgs& a = kw.a;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ KeyShared<D> sh;
    const int warp = warp_value(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t raw = tc::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const GiveUp up{&sh.flag, a.status, wait_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < NK; ++s) {
            tc::mbar_init(&sh.kfull[s], 1);
            tc::mbar_init(&sh.kempty[s], 1);
        }
        for (int s = 0; s < ST; ++s) {
            tc::mbar_init(&sh.qfull[s], 1);
            tc::mbar_init(&sh.qempty[s], 1);
        }
        for (int w = 0; w < W; ++w) {
            for (int k = 0; k < 2; ++k) {
                tc::mbar_init(&sh.sfull[k][w], 2);
                tc::mbar_init(&sh.sempty[k][w], 8);
            }
            tc::mbar_init(&sh.hempty[w], TL::sum_warps);   // W == 2
            tc::mbar_init(&sh.rfull[w], 4);
            tc::mbar_init(&sh.rempty[w], 4);
        }
        tc::mbar_init(&sh.mma_done, 1);
        init_items(sh.items, TL::sum_warps + 3);   // load, shift, MMA and sum warps
        sh.flag = 0;
    }
    // Columns that no row fills stay zero for good: the copies do not reach them.
    const int32_t filled = col.heads * col.rows;
    for (int32_t i = threadIdx.x; i < ST * (D / 64) * (kTile - filled) * 8; i += TL::threads) {
        const int32_t blk = i / ((kTile - filled) * 8), at = i % ((kTile - filled) * 8);
        *reinterpret_cast<uint4*>(smem + TL::off_q + blk * TL::box + filled * 128 + at * 16) = make_uint4(0, 0, 0, 0);
    }
    tc::fence_smem_for_async();
    if (warp == TL::mma_warp) {
        __syncwarp();
        tc::tmem_alloc<TL::tmem>(&sh.tmem_slot);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = warp_value(sh.tmem_slot);

    if (warp == TL::deal_warp) {
        deal_items(sh.items, up, lane, [&](int32_t index, uint32_t& steps) {
            KeyItem it;
            it.set(a, index, heads, per, parts);
            steps = 0;
            for (int32_t k = it.block0; k < it.block1; ++k)
                steps += KeyRange(a, col, it, k, parts).tiles;
            return it;
        });
    } else if (warp == TL::load_warp) {
        uint32_t nk = 0, nq = 0, taken = 0;
        KeyItem it;
        bool ok = true;
        while (!kAttnNoLoads && take_item(sh.items, up, lane, taken, it, ok)) {
            for (int32_t k = it.block0; k < it.block1 && ok; ++k) {
                KeyRange r(a, col, it, k, parts);
                for (int w = 0; w < W && r.tiles > 0 && ok; ++w) {
                    const uint32_t s = nk % NK;
                    ok = item_wait(sh.items, up, &sh.kempty[s], ((nk / NK) & 1u) ^ 1u);   // held for a whole item
                    if (!ok)
                        break;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(&sh.kfull[s], TL::bytes);
                        load_tile<D, kTile>(base + s * TL::bytes, mk, (k * W + w) * kTile, it.hk, it.b, &sh.kfull[s]);
                    }
                    ++nk;
                }
                for (int32_t t = 0; t < r.tiles && ok; ++t, r.next(col)) {
                    const uint32_t s = nq % ST;
                    ok = up.warp_wait(&sh.qempty[s], ((nq / ST) & 1u) ^ 1u);
                    if (!ok)
                        break;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(&sh.qfull[s], filled * D * 2);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tc::tma_load_5d(base + TL::off_q + s * TL::bytes + x * TL::box, &mq, x * 64, r.j, r.i, it.hk,
                                            it.b * col.mb, &sh.qfull[s]);
                    }
                    ++nq;
                }
            }
        }
        if (!ok) {   // let the copies already issued land before the CTA can exit
            for (uint32_t k = 0; k < static_cast<uint32_t>(NK) && k < nk; ++k)
                tc::mbar_wait(&sh.kfull[(nk - 1 - k) % NK], ((nk - 1 - k) / NK) & 1u, kAttnDrainWaitNs);
            for (uint32_t k = 0; k < static_cast<uint32_t>(ST) && k < nq; ++k)
                tc::mbar_wait(&sh.qfull[(nq - 1 - k) % ST], ((nq - 1 - k) / ST) & 1u, kAttnDrainWaitNs);
        }
    } else if (warp == TL::shift_warp) {
        // This lane's four columns of a tile, as row and head in it.
        int32_t ci[4], cj[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            ci[k] = (32 * k + lane) / col.heads;
            cj[k] = (32 * k + lane) % col.heads;
        }
        uint32_t n = 0, taken = 0;
        KeyItem it;
        bool ok = true;
        while (take_item(sh.items, up, lane, taken, it, ok)) {
            const float* lse = a.lse + (static_cast<int64_t>(it.b) * a.Hq + it.hk * a.group) * a.Sq;
            for (int32_t k = it.block0; k < it.block1 && ok; ++k) {
                KeyRange r(a, col, it, k, parts);
                for (int32_t t = 0; t < r.tiles; ++t, ++n, r.next(col)) {
                    float x[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const bool counts = ci[y] < col.rows && r.i + ci[y] < r.i1 && r.j + cj[y] < a.group;
                        x[y] = counts ? __ldg(lse + static_cast<int64_t>(r.j + cj[y]) * a.Sq + r.i + ci[y]) : -INFINITY;
                    }
                    const uint32_t buf = n & 1u;
                    ok = up.warp_wait(&sh.hempty[buf], ((n >> 1) & 1u) ^ 1u);
                    if (!ok)
                        break;
#pragma unroll
                    for (int y = 0; y < 4; ++y)   // a row that kept nothing gives nothing
                        sh.shift[buf][32 * y + lane] = x[y] == -INFINITY ? -INFINITY : -x[y] * kLog2e;
                    __syncwarp();
                    if (lane < W)
                        tc::mbar_arrive(&sh.sfull[buf][lane]);
                }
            }
        }
    } else if (warp == TL::mma_warp) {
        uint32_t nk = 0, nq = 0, taken = 0;
        KeyItem it;
        bool ok = true;
        while (take_item(sh.items, up, lane, taken, it, ok)) {
            for (int32_t k = it.block0; k < it.block1 && ok; ++k) {
                const int32_t tiles = warp_value(KeyRange(a, col, it, k, parts).tiles);
                for (int32_t t = 0; t < tiles && ok; ++t, ++nq) {
                    const uint32_t sq = nq % ST, buf = nq & 1u;
                    ok = up.warp_wait(&sh.qfull[sq], (nq / ST) & 1u);
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint32_t sk = (nk + w) % NK;
                        if (t == 0)
                            ok = ok && up.warp_wait(&sh.kfull[sk], ((nk + w) / NK) & 1u);
                        ok = ok && up.warp_wait(&sh.sempty[buf][w], ((nq >> 1) & 1u) ^ 1u);
                        if (!ok)
                            break;
                        tc::fence_after_sync();
                        mma_abt<T, D, kTile>(tmem + (buf * W + w) * kTile, base + sk * TL::bytes, base + TL::off_q + sq * TL::bytes);
                        tc::commit_warp(&sh.sfull[buf][w]);
                        if (t == tiles - 1)
                            tc::commit_warp(&sh.kempty[sk]);
                    }
                    if (ok)
                        tc::commit_warp(&sh.qempty[sq]);
                }
                nk += tiles > 0 ? W : 0;
            }
        }
        // Nothing may be in flight when the tensor memory is freed.
        tc::commit_warp(&sh.mma_done);
        tc::mbar_wait(&sh.mma_done, 0, kAttnDrainWaitNs);
    } else {
        const int w = (warp >> 2) & 1, half = warp >> 3, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // 32 tensor-memory lanes per warp, lane in bits 16..
        const float c = a.scale * kLog2e;
        const uint32_t ts = tmem + lanes + w * kTile + half * 64;
        uint32_t n = 0, nr = 0, taken = 0;
        KeyItem it;
        bool ok = true;
        while (take_item(sh.items, up, lane, taken, it, ok)) {
            for (int32_t block = it.block0; block < it.block1 && ok; ++block) {
                KeyRange r(a, col, it, block, parts);
                const int32_t first = (block * W + w) * kTile, key = first + row;
                const int32_t last = (first + kTile < it.L ? first + kTile : it.L) - 1;   // the tile's last live key
                // Rows [k0, k1) keep this key; tiles from row [whole0, whole1] keep every live key of this tile with every row.
                int32_t k0 = r.i0, k1 = r.i1, whole0 = r.i0, whole1 = r.i1 - col.rows;
                if (a.mask_kind != GTMS_MASK_LENGTH) {
                    k0 = key - it.off > k0 ? key - it.off : k0;
                    whole0 = last - it.off;
                }
                if (a.mask_kind == GTMS_MASK_SLIDING_WINDOW) {
                    k1 = key + a.window - it.off < k1 ? key + a.window - it.off : k1;
                    whole1 = first + a.window - it.off - col.rows < whole1 ? first + a.window - it.off - col.rows : whole1;
                }
                const bool any = r.tiles > 0;
                float sum = 0.0f;
                for (int32_t t = 0; t < r.tiles; ++t, ++n, r.next(col)) {
                    const uint32_t buf = n & 1u;
                    ok = item_wait(sh.items, up, &sh.sfull[buf][w], (n >> 1) & 1u);
                    if (!ok)
                        break;
                    tc::fence_after_sync();
                    float x[64];
                    tc::tmem_ld64(ts + buf * (W * kTile), x);
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive(&sh.sempty[buf][w]);
                    // The exponents, all of them before the first exponential.
                    const float4* shift = reinterpret_cast<const float4*>(&sh.shift[buf][half * 64]);
                    const float2 c2 = make_float2(c, c);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float4 h = shift[k];
                        const float2 e = __ffma2_rn(make_float2(x[4 * k], x[4 * k + 1]), c2, make_float2(h.x, h.y));
                        const float2 f = __ffma2_rn(make_float2(x[4 * k + 2], x[4 * k + 3]), c2, make_float2(h.z, h.w));
                        x[4 * k] = e.x;
                        x[4 * k + 1] = e.y;
                        x[4 * k + 2] = f.x;
                        x[4 * k + 3] = f.y;
                    }
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive(&sh.hempty[buf]);
                    float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    if (__builtin_expect(r.i >= whole0 && r.i <= whole1 && r.j + col.heads <= a.group, 1)) {
#pragma unroll
                        for (int k = 0; k < 64; k += 4) {
                            acc[0] = __fadd2_rn(acc[0], make_float2(exp2_approx(x[k]), exp2_approx(x[k + 1])));
                            acc[1] = __fadd2_rn(acc[1], make_float2(exp2_approx(x[k + 2]), exp2_approx(x[k + 3])));
                        }
                    } else {
                        // Rows [k0, k1) keep this key: columns [n0, n1) of this half, rows of the tile times heads.
                        const int32_t n0 = min(max(k0 - r.i, 0), kTile) * col.heads - half * 64;
                        int32_t n1 = min(max(k1 - r.i, 0), kTile) * col.heads;
                        n1 = (col.head_tiles > 1 && n1 > a.group - r.j ? a.group - r.j : n1) - half * 64;
#pragma unroll
                        for (int k = 0; k < 64; k += 32) {
                            const uint32_t keep = bits_below(n1 - k) & ~bits_below(n0 - k);
                            if (__any_sync(0xffffffffu, keep != 0)) {   // a narrow window's keys see few of the rows
#pragma unroll
                                for (int y = 0; y < 32; ++y) {
                                    const float e = exp2_approx(x[k + y]);
                                    acc[y & 1].x += keep & (1u << y) ? e : 0.0f;
                                }
                            }
                        }
                    }
                    sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                }
                if (!ok)
                    break;
                // The halves of a tile's columns meet.
                if (any) {
                    if (half == 1) {
                        ok = up.warp_wait(&sh.rempty[w], (nr & 1u) ^ 1u);
                        if (!ok)
                            break;
                        sh.half[w][row] = sum;
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(&sh.rfull[w]);
                    } else {
                        ok = up.warp_wait(&sh.rfull[w], nr & 1u);
                        if (!ok)
                            break;
                        sum += sh.half[w][row];
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(&sh.rempty[w]);
                    }
                    ++nr;
                }
                if (half == 0 && key < a.Skv) {
                    const int64_t at = (static_cast<int64_t>(it.b) * a.Hkv + it.hk) * a.Skv + key;
                    if (parts > 1) {
                        if (key < it.L)
                            kw.parts[it.part * (static_cast<int64_t>(a.B) * a.Hkv * a.Skv) + at] = sum;
                    } else if (key < it.L) {
                        kw.weights[at] = kw.accumulate ? kw.weights[at] + sum : sum;
                    } else if (!kw.accumulate) {
                        kw.weights[at] = 0.0f;
                    }
                }
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == TL::mma_warp) {
        __syncwarp();
        tc::tmem_free<TL::tmem>(tmem);
    }
}

// The parts' sums, in order.
inline constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) gtms_key_weights_join_kernel(const KeyWeightsArgs kw, int32_t parts)
{
    const AttentionArgs& a = kw.a;
    const int64_t all = static_cast<int64_t>(a.B) * a.Hkv * a.Skv, at = blockIdx.x * static_cast<int64_t>(kSumThreads) + threadIdx.x;
    await_last_launch();
    if (at >= all)
        return;
    const int64_t bg = at / a.Skv;
    const int32_t key = static_cast<int32_t>(at - bg * a.Skv), L = a.length(static_cast<int32_t>(bg / a.Hkv));
    if (key >= L) {
        if (!kw.accumulate)
            kw.weights[at] = 0.0f;
        return;
    }
    float sum = 0.0f;
    for (int32_t p = 0; p < parts; ++p)
        sum += kw.parts[p * all + at];
    kw.weights[at] = kw.accumulate ? kw.weights[at] + sum : sum;
}

// How the work is cut: an item of many column tiles into parts of its rows, so that
// whoever is done first finds something left; blocks of few column tiles put together,
// so that keys stream in without a pause between items.
struct KeyPlan {
    int32_t per;     // blocks of 256 keys of an item
    int32_t parts;   // of its rows
};

constexpr int64_t kLongTiles = 8192;

inline KeyPlan key_plan(const AttentionArgs& a)
{
    const KeyColumns col = key_columns(a.group);
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hkv, blocks = (static_cast<int64_t>(a.Skv) + 2 * kTile - 1) / (2 * kTile);
    // Column tiles of a block at most: a window leaves a key few rows.
    const int64_t reach = a.mask_kind == GTMS_MASK_SLIDING_WINDOW && a.window + 2 * kTile < a.Sq ? a.window + 2 * kTile : a.Sq;
    const int64_t tiles = (reach + col.rows - 1) / col.rows * col.head_tiles;
    KeyPlan p{1, 1};
    // Items. Five to a multiprocessor (2, 3, 5, 8: [4,32/8,4096,128] 200, 200, 179, 176 us, the last 32 rows over 16384
    // keys 57, 49, 46, 48, [4,16/2,1816,64] 38, 31, 28, 31, [1,16/4,4266,64] 46, 43, 41, 46).
    const int64_t want = 5 * kChipSms;
    if (heads * blocks < want) {
        const int64_t parts = (want + heads * blocks - 1) / (heads * blocks);
        p.parts = static_cast<int32_t>(parts < tiles / 4 ? parts : tiles / 4);
        p.parts = p.parts > 1 ? p.parts : 1;
    } else if (tiles < 16) {
        int64_t per = 16 / tiles;
        per = per < heads * blocks / want ? per : heads * blocks / want;
        p.per = per > 1 ? static_cast<int32_t>(per) : 1;
    }
    // Long sums in parts too: one of 8192 tiles' sums, a million rows, drops 2^-11 of itself at most.
    const int64_t least = (tiles + kLongTiles - 1) / kLongTiles;
    p.parts = p.parts > least ? p.parts : static_cast<int32_t>(least);
    return p;
}

template <typename T, int D>
cudaError_t launch_key_weights_tc(const KeyWeightsArgs& kw, cudaStream_t st, uint64_t wait_ns = kAttnWaitNs)
{
    using TL = KeyTile<D>;
    const AttentionArgs& a = kw.a;
    const TensorMapEncodeFn enc = tensor_map_encoder();
    if (!bind_context() || !enc)
        return cudaErrorUnknown;
    HeadsMap mk;
    if (!encode_heads<T>(mk, a.k, a.B, a.Hkv, a.Skv, D, kTile))
        return cudaErrorInvalidValue;
    KeyColumns col = key_columns(a.group);
    col.mb = a.B > 1 && a.q.sb != 0;
    // A stride that is never stepped over still has to be a legal one.
    const cuuint64_t any = D * 2;
    CUtensorMap mq;
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.group), static_cast<cuuint64_t>(a.Sq),
                                static_cast<cuuint64_t>(a.Hkv), static_cast<cuuint64_t>(col.mb ? a.B : 1)};
    const cuuint64_t strides[4] = {a.group > 1 ? static_cast<cuuint64_t>(a.q.sh) * 2 : any, a.Sq > 1 ? static_cast<cuuint64_t>(a.q.ss) * 2 : any,
                                   a.Hkv > 1 ? static_cast<cuuint64_t>(a.q.sh) * a.group * 2 : any,
                                   col.mb ? static_cast<cuuint64_t>(a.q.sb) * 2 : any};
    const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(col.heads), static_cast<cuuint32_t>(col.rows), 1, 1}, estr[5] = {1, 1, 1, 1, 1};
    if (enc(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, a.q.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hkv;
    const KeyPlan plan = key_plan(a);
    const int64_t blocks = (static_cast<int64_t>(a.Skv) + TL::keys - 1) / TL::keys;
    const int64_t items = heads * ((blocks + plan.per - 1) / plan.per) * plan.parts;
    if (items > INT32_MAX)
        return cudaErrorNotSupported;
    constexpr auto* kern = gtms_key_weights_kernel<T, D>;
    constexpr int smem = static_cast<int>(TL::smem);
    cudaError_t e = allow_smem<kern>(smem);
    if (e == cudaSuccess)
        e = launch_kernel(kern, static_cast<unsigned>(items), TL::threads, smem, st, mq, mk, kw, col, static_cast<uint32_t>(heads),
                          plan.per, plan.parts, wait_ns);
    if (e != cudaSuccess || plan.parts == 1)
        return e;
    const int64_t ctas = (heads * a.Skv + kSumThreads - 1) / kSumThreads;
    return launch_beside_last(true, gtms_key_weights_join_kernel, static_cast<unsigned>(ctas), kSumThreads, 0, st, kw, plan.parts);
}

}  // namespace gtms
