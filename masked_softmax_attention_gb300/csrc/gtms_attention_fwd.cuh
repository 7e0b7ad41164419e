// gtms_attention_fwd.cuh -- attention forward on the tensor cores.
//
//   s_ic = scale q_i . k_c,  o_i = sum_c exp(s_ic - m_i) v_c / l_i,
//   l_i = sum_c exp(s_ic - m_i),  lse_i = m_i + log l_i   over the kept c.
//
// A CTA works on one or two tiles of 128 query rows (see FwdTile) and walks over the
// 128-key tiles that hold kept entries, last first (so that the tiles a causal mask
// cuts come first and the maximum settles early). Scores, probabilities and the
// output accumulators stay in tensor memory: S of each query tile (128 fp32
// columns; P, rounded to 16 bits, is written over the first half of it), then O
// (head_dim fp32 columns each).
// Roles:
//   deal (1 warp)     the work items (see ItemSlot);
//   load (1 warp)     TMA: the query tiles, then K and V tiles into one ring;
//   MMA (1 warp)      S_w = Q_w K^T and O_w += P_w V with P_w read from tensor
//                     memory. The two tiles alternate, so one's products run while
//                     the other's softmax does;
//   softmax (4 warps a tile) a thread owns one row: it reads its 128 scores, so the
//                     maximum and the sum need no exchange, writes P back, and at
//                     the end divides O and stores it.
// The running maximum is only raised, and O and l rescaled, when a tile exceeds it
// by more than 12 in log2 units: p stays below 2^12, which fp16, bf16 and fp32
// hold as well as numbers below 1, and almost no tile but a row's first does. The
// thread that owns the row rescales: S_w of a tile completes after every earlier
// product into O_w, so no other hand-off is needed.
// What bounds it: at head dim 128 the tensor cores, 66 % busy on a full-length
// case of 32 heads (a softmax thread's chain of scores, maximum, exponentials and
// hand-over and the two products it waits for take 2400 cycles a tile, and the two
// tiles' chains overlap): [4,32/8,4096,128] bf16 249 us in a short run of calls, 1480
// TFLOP/s, 272 us after seconds of work, at lower clocks. At 64 the
// softmax warps' instructions, 43 % of the issue slots, and their fetching: what
// made their loop shorter made it faster (masks as 32-bit words 267 -> 258 us, no
// second copy of the exponentials 251 -> 245 and 247 -> 237 us; two MMA warps,
// whose code evicts theirs, cost 70 %): [32,16,2048,64] 237 and 247 us.
#pragma once

#include "gtms_attention_tc.cuh"

namespace gtms {

constexpr float kRaiseLog2 = 12.0f;

// Query tiles (W) of a CTA and CTAs of a multiprocessor: two tiles work side by side
// on each. At head dim 128 they share a CTA, and so the keys and values in shared
// memory, which their tiles fill, as their scores and outputs fill the tensor
// memory. At 64 there is room for two CTAs of one tile, which run into each
// other's starts and ends of items and have an MMA warp each ([32,16,2048,64] bf16:
// 252 us with two tiles to a CTA, 264 with four tiles and keys by 64, 248 so;
// 24 heads of 333 rows: 9.4 -> 8.4 us).
template <int D>
struct FwdTile {
    static constexpr int W = D == 64 ? 1 : 2, ctas = 2 / W, tmem = 512 / ctas;
    // Parts in which P is handed over: halves at head dim 128, where the tensor cores bound the kernel and the first
    // half's product starts early (252 -> 245 us); at 64 the hand-over costs more than it gives (237 -> 235).
    static constexpr int parts = W;
    static constexpr int rows = W * kTile;                                 // query rows of one work item
    static constexpr int mma_warp = 4 * W, load_warp = mma_warp + 1, deal_warp = mma_warp + 2;   // after the softmax warps
    static constexpr int threads = 32 * (4 * W + 4);                       // one warp idle: register shares go by warpgroup
    // Registers a thread at launch, shared out so that a softmax thread holds its row of 128 scores.
    static constexpr int regs = W == 1 ? 128 : 168, softmax_regs = W == 1 ? 192 : 208, other_regs = W == 1 ? 64 : 88;
    static_assert(W * softmax_regs + other_regs <= (W + 1) * regs, "register shares of one block");
    static constexpr int stages = 4;                                       // of the ring of K and V tiles
    static constexpr uint32_t bytes = kTile * D * 2, box = kTile * 128;    // a 128-row tile, 64 columns of it
    static constexpr uint32_t t_o = W * kTile;                             // tensor memory: S (and P), then O
    static_assert(t_o + W * D <= tmem, "tensor memory");
    static constexpr uint32_t stage = 4096;                                // per softmax warp: 32 rows x 64 columns of results
    static constexpr uint32_t off_ring = W * bytes, off_out = off_ring + stages * bytes;
    static constexpr uint32_t smem = off_out + 4 * W * stage + 1024;       // slack to align the base
};

// Work item: W query tiles of one head, costliest row blocks first.
template <int W>
struct FwdItem {
    int32_t b, h, i0, off, L;
    int32_t lo[W], hi[W];       // key tiles [lo, hi) of each query tile
    int32_t full0[W], full1[W]; // columns [full0, full1) that every live row of the tile keeps

    __device__ __forceinline__ void set(const AttentionArgs& a, uint32_t item, uint32_t heads, int32_t blocks)
    {
        const int32_t blk = blocks - 1 - static_cast<int32_t>(item / heads);
        const int32_t bh = static_cast<int32_t>(item % heads);
        b = bh / a.Hq;
        h = bh - b * a.Hq;
        i0 = blk * W * kTile;
        off = a.offset(b);
        L = a.length(b);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int32_t i = i0 + w * kTile;
            const int32_t last = i + kTile < a.Sq ? i + kTile : a.Sq;
            const int32_t ra = off + i > 0 ? off + i : 0, rb = (off + last < L ? off + last : L) - 1;
            lo[w] = hi[w] = 0;
            full0[w] = full1[w] = 0;
            if (ra <= rb) {
                int32_t a0, a1, b0, b1;
                a.kept(ra, L, a0, a1);
                a.kept(rb, L, b0, b1);
                lo[w] = a0 / kTile;
                hi[w] = (b1 + kTile - 1) / kTile;
                full0[w] = b0;
                full1[w] = a1;
            }
        }
    }
    __device__ __forceinline__ int32_t top() const
    {
        int32_t t = 0;
#pragma unroll
        for (int w = 0; w < W; ++w)
            t = hi[w] > t ? hi[w] : t;
        return t;
    }
    __device__ __forceinline__ int32_t bottom() const
    {
        int32_t t = INT32_MAX;
#pragma unroll
        for (int w = 0; w < W; ++w)
            t = hi[w] > 0 && lo[w] < t ? lo[w] : t;
        return t;
    }
    __device__ __forceinline__ uint32_t steps(const AttentionArgs&) const { return top() > 0 ? top() - bottom() : 0; }
    __device__ __forceinline__ bool has(int w, int32_t t) const { return t >= lo[w] && t < hi[w]; }
};

template <int W>
struct FwdShared {
    uint64_t qfull[W], qempty[W];
    uint64_t kvfull[4], kvempty[4], vraw;
    uint64_t sfull[W], pready[W][2], ofull[W], oempty[W];
    ItemSlot<FwdItem<W>> items;
    uint64_t mma_done;
    uint32_t tmem_slot;
    int flag;
};

template <typename T, int D, bool LONG>
__global__ void __launch_bounds__(FwdTile<D>::threads, FwdTile<D>::ctas)
gtms_attention_fwd_kernel(const __grid_constant__ HeadsMap mq, const __grid_constant__ HeadsMap mk,
                          const __grid_constant__ HeadsMap mv, const __grid_constant__ AttentionArgs a, uint32_t heads,
                          int32_t blocks, uint64_t wait_ns)
{
    using TL = FwdTile<D>;
    constexpr int ST = TL::stages, W = TL::W, carry_tiles = kCarryTerms<T> / kTile;
    using Item = FwdItem<W>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ FwdShared<W> sh;
    const int warp = warp_value(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t raw = tc::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const GiveUp up{&sh.flag, a.status, wait_ns};

    if (threadIdx.x == 0) {
        for (int w = 0; w < W; ++w) {
            tc::mbar_init(&sh.qfull[w], 1);
            tc::mbar_init(&sh.qempty[w], 1);
            tc::mbar_init(&sh.sfull[w], 1);
            for (int k = 0; k < 2; ++k)
                tc::mbar_init(&sh.pready[w][k], 4);
            tc::mbar_init(&sh.ofull[w], 1);
            tc::mbar_init(&sh.oempty[w], 4);
        }
        for (int s = 0; s < ST; ++s) {
            tc::mbar_init(&sh.kvfull[s], 1);
            tc::mbar_init(&sh.kvempty[s], 1);
        }
        tc::mbar_init(&sh.vraw, 1);
        tc::mbar_init(&sh.mma_done, 1);
        init_items(sh.items, 4 * W + 2);   // load, MMA and softmax warps
        sh.flag = 0;
    }
    if (warp == TL::mma_warp) {
        __syncwarp();
        tc::tmem_alloc<TL::tmem>(&sh.tmem_slot);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = warp_value(sh.tmem_slot);

    if (warp >= TL::mma_warp) {
        tc::regs_lower<TL::other_regs>();
        if (warp == TL::deal_warp) {
            deal_items(sh.items, up, lane, a, [&](int32_t index) {
                Item it;
                it.set(a, index, heads, blocks);
                return it;
            });
        } else if (warp == TL::load_warp) {
            uint32_t g = 0, asked = 0, odd = 0, nraw = 0, taken = 0;   // bits w: queries loaded at all, an odd number of times
            Item it;
            bool ok = true;
            while (!kAttnNoLoads && take_item(sh.items, up, lane, taken, it, ok)) {
                const int32_t hk = it.h / a.group;
                auto tile = [&](const HeadsMap& m, int32_t t, bool tail) {
                    const uint32_t s = g % ST;
                    ok = up.warp_wait(&sh.kvempty[s], ((g / ST) & 1u) ^ 1u);
                    if (!ok)
                        return;
                    const uint32_t dst = TL::off_ring + s * TL::bytes;
                    uint64_t* bar = tail ? &sh.vraw : &sh.kvfull[s];
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(bar, TL::bytes);
                        load_tile<D, kTile>(base + dst, m, t * kTile, hk, it.b, bar);
                    }
                    if (tail) {
                        // Keys behind the length may hold anything, and 0 x NaN is NaN: zero their rows of V.
                        ok = up.warp_wait(&sh.vraw, nraw & 1u);
                        ++nraw;
                        if (!ok)
                            return;
                        zero_tile_rows<D, kTile>(smem + dst, it.L - t * kTile, kTile, lane);
                        tc::fence_smem_for_async();
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(&sh.kvfull[s]);
                    }
                    ++g;
                };
                auto queries = [&](int w) {
                    ok = up.warp_wait(&sh.qempty[w], ((odd >> w) & 1u) ^ 1u);
                    if (!ok)
                        return;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(&sh.qfull[w], TL::bytes);
                        load_tile<D, kTile>(base + w * TL::bytes, mq, it.i0 + w * kTile, it.h, it.b, &sh.qfull[w]);
                    }
                    odd ^= 1u << w;
                    asked |= 1u << w;
                };
                uint32_t loaded = 0;
                for (int32_t t = it.top() - 1; t >= it.bottom() && ok; --t) {
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        if (ok && !(loaded & (1u << w)) && it.has(w, t)) {
                            loaded |= 1u << w;
                            queries(w);
                        }
                    if (ok)
                        tile(mk, t, false);
                    if (ok)
                        tile(mv, t, (t + 1) * kTile > it.L && it.L < a.Skv);
                }
            }
            if (!ok) {   // let the copies already issued land before the CTA can exit
                for (uint32_t k = 0; k < static_cast<uint32_t>(ST) && k < g; ++k)
                    tc::mbar_wait(&sh.kvfull[(g - 1 - k) % ST], ((g - 1 - k) / ST) & 1u, kAttnDrainWaitNs);
                for (int w = 0; w < W; ++w)
                    if (asked & (1u << w))
                        tc::mbar_wait(&sh.qfull[w], ((odd >> w) & 1u) ^ 1u, kAttnDrainWaitNs);
                if (nraw)
                    tc::mbar_wait(&sh.vraw, (nraw - 1) & 1u, kAttnDrainWaitNs);
            }
        } else if (warp == TL::mma_warp) {
            constexpr uint32_t idesc_o = tc::idesc_f16<T>(kTile, D) | tc::kIdescBMnMajor;
            // n counts key tiles; bits w: parities of the queries, the hand-overs of P and the outputs of tile w.
            uint32_t n = 0, nq = 0, np = 0, no = 0, taken = 0;
            Item it;
            bool ok = true;
            while (take_item(sh.items, up, lane, taken, it, ok)) {
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    it.lo[w] = warp_value(it.lo[w]);
                    it.hi[w] = warp_value(it.hi[w]);
                }
                const int32_t top = it.top(), bottom = it.bottom();
                if (top == 0)
                    continue;
                // S_w of tile t, whose K is ring entry 2 n' (its arrival has been waited for).
                auto scores = [&](int w, int32_t t, uint32_t tile_n) {
                    if (t == it.hi[w] - 1) {
                        ok = up.warp_wait(&sh.qfull[w], (nq >> w) & 1u);
                        nq ^= 1u << w;
                        if (!ok)
                            return;
                        tc::fence_after_sync();
                    }
                    const uint32_t q0 = base + w * TL::bytes, k0 = base + TL::off_ring + ((2 * tile_n) % ST) * TL::bytes;
                    mma_abt<T, D, kTile>(tmem + w * kTile, q0, k0);
                    tc::commit_warp(&sh.sfull[w]);
                    if (t == it.lo[w])
                        tc::commit_warp(&sh.qempty[w]);
                };
                auto output = [&](int w, int32_t t) {
                    const bool first = t == it.hi[w] - 1;
                    const uint32_t v0 = base + TL::off_ring + ((2 * n + 1) % ST) * TL::bytes;
#pragma unroll
                    for (int part = 0; part < TL::parts; ++part) {
                        ok = up.warp_wait(&sh.pready[w][part], (np >> w) & 1u);
                        if (ok && first && part == 0)
                            ok = up.warp_wait(&sh.oempty[w], ((no >> w) & 1u) ^ 1u);
                        if (!ok)
                            return;
                        tc::fence_after_sync();
#pragma unroll
                        for (int ks = part * (8 / TL::parts); ks < (part + 1) * (8 / TL::parts); ++ks)
                            tc::mma_f16_ts_warp(tmem + TL::t_o + w * D, tmem + w * kTile + ks * 8,
                                                tc::smem_desc_sw128_mn(v0 + ks * 2048, TL::box), idesc_o, !first || ks > 0);
                    }
                    np ^= 1u << w;
                    if (t == it.lo[w]) {
                        tc::commit_warp(&sh.ofull[w]);
                        no ^= 1u << w;
                    }
                };
                auto arrived = [&](uint32_t e) {
                    ok = up.warp_wait(&sh.kvfull[e % ST], (e / ST) & 1u);
                    tc::fence_after_sync();
                };
                arrived(2 * n);
#pragma unroll
                for (int w = 0; w < W; ++w)
                    if (ok && it.has(w, top - 1))
                        scores(w, top - 1, n);
                if (!ok)
                    break;
                tc::commit_warp(&sh.kvempty[(2 * n) % ST]);
                for (int32_t t = top - 1; t >= bottom && ok; --t, ++n) {
                    // What the loads bring is waited for first: the hand-overs of P are the ones that matter.
                    arrived(2 * n + 1);
                    if (ok && t > bottom)
                        arrived(2 * n + 2);
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        if (ok && it.has(w, t))
                            output(w, t);
                        if (ok && it.has(w, t - 1))
                            scores(w, t - 1, n + 1);
                    }
                    if (ok) {
                        tc::commit_warp(&sh.kvempty[(2 * n + 1) % ST]);
                        if (t > bottom)
                            tc::commit_warp(&sh.kvempty[(2 * n + 2) % ST]);
                    }
                }
            }
            // Nothing may be in flight when the tensor memory is freed.
            tc::commit_warp(&sh.mma_done);
            tc::mbar_wait(&sh.mma_done, 0, kAttnDrainWaitNs);
        }
    } else {
        tc::regs_raise<TL::softmax_regs>();
        const int w = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // 32 tensor-memory lanes per warp, lane in bits 16..
        const uint32_t ts = tmem + lanes + w * kTile, to = tmem + lanes + TL::t_o + w * D;
        // exp(scale x) = exp2(c x) with c > 0: a negative scale flips the scores, a zero one clears them.
        const float c = a.scale == 0.0f ? kLog2e : fabsf(a.scale) * kLog2e;
        const float pre = a.scale > 0.0f ? 1.0f : (a.scale < 0.0f ? -1.0f : 0.0f);
        uint32_t ns = 0, no = 0, taken = 0;
        bool ok = true;
        int32_t b = 0, h = 0, i = 0, c0 = 0, c1 = 0, lo = 0, hi = 0, full0 = 0, full1 = 0;
        auto read = [&](const Item& it) {
            b = it.b;
            h = it.h;
            i = it.i0 + w * kTile + (warp & 3) * 32 + lane;
            a.kept(it.off + i, it.L, c0, c1);
            lo = it.lo[w];
            hi = it.hi[w];
            full0 = it.full0[w];
            full1 = it.full1[w];
        };
        while (take_item(sh.items, up, lane, taken, ok, read)) {
            const bool live = c0 < c1 && i < a.Sq;
            float m = -INFINITY, l = 0.0f;
            float m_carried = -INFINITY, l_carried = 0.0f;   // of the part of O that the row of o carries, in units of l
            auto carried = [&] { return l_carried > 0.0f ? l_carried * exp2_approx((m_carried - m) * c) : 0.0f; };
            for (int32_t t = hi - 1; t >= lo; --t) {
                // The first scores may have to wait while the other tile has a whole item to itself.
                ok = item_wait(sh.items, up, &sh.sfull[w], ns & 1u);
                ++ns;
                if (!ok)
                    break;
                tc::fence_after_sync();
                if (LONG && (hi - 1 - t) % carry_tiles == 0 && t != hi - 1) {
                    // The products into O are done, up to the last tile's (see above).
                    carry_accumulator<T, D>(to, live ? a.o.row<T>(b, h, i) : nullptr, carried(), l, l > 0.0f ? 1.0f / l : 0.0f);
                    m_carried = m;
                    l_carried = l;
                }
                float s[kTile];
                tc::tmem_ld128(ts, s);
                if (__builtin_expect(pre != 1.0f, 0)) {
#pragma unroll
                    for (int j = 0; j < kTile; ++j)
                        s[j] *= pre;
                }
                if (__builtin_expect((t + 1) * kTile > full1 || t * kTile < full0, 0)) {
                    const int32_t k0 = c0 - t * kTile, k1 = c1 - t * kTile;
#pragma unroll
                    for (int k = 0; k < kTile; k += 32) {
                        const uint32_t keep = bits_below(k1 - k) & ~bits_below(k0 - k);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            s[k + j] = keep & (1u << j) ? s[k + j] : -INFINITY;
                    }
                }
                float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int j = 4; j < kTile; j += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = j + 4 + k < kTile ? max3(x[k], s[j + k], s[(j + 4 + k) % kTile]) : fmaxf(x[k], s[j + k]);
                const float top = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                // 32 probabilities from column k on: exp2(c s - c m), summed in fp32, and rounded to 16 bits, the type of
                // V, with which alone the tensor cores multiply them at full rate (o is off by 1.3 to 1.5 roundings of its
                // own type instead of 1).
                auto exponentiate = [&](int k, float shift, uint32_t(&r)[16]) {
                    const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float2 e = __ffma2_rn(make_float2(s[k + 2 * j], s[k + 2 * j + 1]), c2, shift2);
                        e = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                        sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                        r[j] = pack2<T>(e.x, e.y);
                    }
                };
                const bool opening = t == hi - 1;   // nothing to rescale yet
                const bool raise = (top - m) * c > kRaiseLog2;   // a row's first kept tile: infinity
                auto raised = [&] {
                    const float f = raise ? exp2_approx((m - top) * c) : 1.0f;
                    m = raise ? top : m;
                    l *= f;
                    if (!opening) {
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            float o[16];
                            uint32_t r[16];
                            tc::tmem_ld16(to + k, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                r[j] = __float_as_uint(o[j] * f);
                            tc::tmem_st16(to + k, r);
                        }
                    }
                };
                if (__builtin_expect(__any_sync(0xffffffffu, raise), 0))
                    raised();
                const float shift = m == -INFINITY ? 0.0f : -m * c;
                auto hand_over = [&](uint64_t* bar) {
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive(bar);
                };
                uint32_t r0[16], r1[16];
                exponentiate(0, shift, r0);
                exponentiate(32, shift, r1);
                tc::tmem_st16(ts, r0);
                tc::tmem_st16(ts + 16, r1);
                if (TL::parts == 2)
                    hand_over(&sh.pready[w][0]);
                exponentiate(64, shift, r0);
                tc::tmem_st16(ts + 32, r0);
                exponentiate(96, shift, r1);
                tc::tmem_st16(ts + 48, r1);
                hand_over(&sh.pready[w][TL::parts - 1]);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (!ok)
                break;
            T* out = i < a.Sq ? a.o.row<T>(b, h, i) : nullptr;
            uint8_t* stage = smem + TL::off_out + warp * TL::stage;
            const float inv = live ? 1.0f / l : 0.0f;
            const bool any = hi > lo;
            if (any) {
                ok = up.warp_wait(&sh.ofull[w], no & 1u);
                ++no;
                if (!ok)
                    break;
                tc::fence_after_sync();
            }
#pragma unroll 1
            for (int k = 0; k < D; k += 64) {
                uint32_t r[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    r[j] = 0;
                if (any) {
                    float o[64];
                    tc::tmem_ld64(to + k, o);
                    if (LONG && hi - lo > carry_tiles && live)
                        add_carried(o, out + k, carried());
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        r[j] = live ? pack2<T>(o[2 * j] * inv, o[2 * j + 1] * inv) : 0u;
                }
                store_rows<64>(stage, lane, r, out ? out + k : nullptr);
            }
            if (any) {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&sh.oempty[w]);
            }
            if (a.lse && i < a.Sq)
                a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Sq + i] =
                    live ? (a.scale == 0.0f ? m : m * fabsf(a.scale)) + logf(l) : -INFINITY;
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

template <typename T, int D>
cudaError_t launch_attention_fwd_tc(const AttentionArgs& a, cudaStream_t st, uint64_t wait_ns = kAttnWaitNs)
{
    using TL = FwdTile<D>;
    if (!bind_context())
        return cudaErrorUnknown;
    // Without keys no tile is loaded, and q stands in for k and v in the maps.
    const bool keys = a.Skv > 0;
    HeadsMap mq, mk, mv;
    if (!encode_heads<T>(mq, a.q, a.B, a.Hq, a.Sq, D, kTile) ||
        !encode_heads<T>(mk, keys ? a.k : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile) ||
        !encode_heads<T>(mv, keys ? a.v : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile))
        return cudaErrorInvalidValue;
    // One CTA per item; the running ones take over the others' (see ItemSlot).
    const int32_t blocks = (a.Sq + TL::rows - 1) / TL::rows;
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hq;
    auto launch = [&](auto is_long) {
        constexpr auto* kern = gtms_attention_fwd_kernel<T, D, is_long()>;
        constexpr int smem = static_cast<int>(TL::smem);
        const cudaError_t e = allow_smem<kern>(smem);
        return e != cudaSuccess ? e
                                : launch_kernel(kern, static_cast<unsigned>(heads * blocks), TL::threads, smem, st, mq, mk, mv, a,
                                                static_cast<uint32_t>(heads), blocks, wait_ns);
    };
    return kept_at_most(a, a.Skv) > kCarryTerms<T> ? launch(std::true_type()) : launch(std::false_type());
}

}  // namespace gtms
