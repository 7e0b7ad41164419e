// gtms_attention_fwd.cuh -- attention forward on the tensor cores.
//
//   s_ic = scale q_i . k_c,  o_i = sum_c exp(s_ic - m_i) v_c / l_i,
//   l_i = sum_c exp(s_ic - m_i),  lse_i = m_i + log l_i   over the kept c.
//
// One persistent CTA per SM works on 256 query rows at a time, as two tiles of
// 128, and walks over the 128-key tiles that hold kept entries, last first (so
// that the tiles a causal mask cuts come first and the maximum settles early).
// Scores, probabilities and both output accumulators stay in tensor memory:
//   columns 0..255    S of tile 0 and 1 (fp32); P, rounded to 16 bits, is written
//                     over the first half of its own S;
//   columns 256..511  O of tile 0 and 1 (fp32, head_dim columns each).
// Roles:
//   load (1 warp)     TMA: the query tiles, then K and V tiles into one ring;
//   MMA (1 warp)      S_w = Q_w K^T and O_w += P_w V with P_w read from tensor
//                     memory. The two tiles alternate, so one's products run while
//                     the other's softmax does;
//   softmax (2 x 4 warps) a thread owns one row: it reads its 128 scores, so the
//                     maximum and the sum need no exchange, writes P back, and at
//                     the end divides O and stores it.
// The running maximum is only raised, and O and l rescaled, when it would grow by
// more than 8 in log2 units: p stays below 2^8, which 16-bit and fp32 hold as
// well, and the rescaling of O leaves the loop for almost every tile. The thread
// that owns the row rescales: S_w of a tile completes after every earlier product
// into O_w, so no other hand-off is needed.
#pragma once

#include "gtms_attention_tc.cuh"

namespace gtms {

constexpr int kFwdRows = 2 * kTile;                 // query rows of one work item
constexpr int kFwdMmaWarp = 8, kFwdLoadWarp = 9;    // warps 0..7 are the softmax warps
constexpr int kFwdThreads = 32 * 12;                // two warps idle: register shares go by warpgroup
// 168 registers a thread at launch (three warps to each SM quarter), shared out as
// 208 for a softmax thread, which holds a row of 128 scores, and 88 for the rest.
constexpr int kFwdRegs = 168, kFwdSoftmaxRegs = 208, kFwdOtherRegs = 88;
static_assert(2 * kFwdSoftmaxRegs + kFwdOtherRegs <= 3 * kFwdRegs, "register shares of one block");
constexpr float kRescaleLog2 = 8.0f;

template <int D>
struct FwdTile {
    static constexpr int stages = D == 64 ? 8 : 5;
    static constexpr uint32_t bytes = kTile * D * 2;          // one 128-row tile
    static constexpr uint32_t box = kTile * 128;              // one swizzled 64-column box of it
    static constexpr uint32_t off_ring = 2 * bytes;
    static constexpr uint32_t smem = (2 + stages) * bytes + 1024;   // + slack to align the base
};

struct FwdShared {
    uint64_t qfull[2], qempty[2];
    uint64_t kvfull[8], kvempty[8], vraw;
    uint64_t sfull[2], pready[2], ofull[2], oempty[2];
    uint64_t mma_done;
    uint32_t tmem_slot;
    int flag;
};

// Work item: 256 rows of one head, costliest row blocks first (a whole warp calls).
struct FwdItem {
    int32_t b, h, i0, off, L;
    int32_t lo[2], hi[2];       // key tiles [lo, hi) of each query tile
    int32_t full0[2], full1[2]; // columns [full0, full1) that every live row of the tile keeps

    __device__ __forceinline__ FwdItem(const AttentionArgs& a, int64_t item, int64_t heads, int32_t blocks)
    {
        const int32_t blk = blocks - 1 - static_cast<int32_t>(item / heads);
        const int32_t bh = static_cast<int32_t>(item % heads);
        b = bh / a.Hq;
        h = bh - b * a.Hq;
        i0 = blk * kFwdRows;
        off = warp_value(a.offset(b));
        L = warp_value(a.length(b));
#pragma unroll
        for (int w = 0; w < 2; ++w) {
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
    __device__ __forceinline__ int32_t top() const { return hi[0] > hi[1] ? hi[0] : hi[1]; }
    __device__ __forceinline__ int32_t bottom() const
    {
        if (hi[0] == 0)
            return lo[1];
        return hi[1] == 0 || lo[0] < lo[1] ? lo[0] : lo[1];
    }
    __device__ __forceinline__ bool has(int w, int32_t t) const { return t >= lo[w] && t < hi[w]; }
};

template <typename T, int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
gtms_attention_fwd_kernel(const __grid_constant__ HeadsMap mq, const __grid_constant__ HeadsMap mk,
                          const __grid_constant__ HeadsMap mv, const __grid_constant__ AttentionArgs a, int64_t heads,
                          int32_t blocks, uint64_t wait_ns)
{
    using TL = FwdTile<D>;
    constexpr int ST = TL::stages;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ FwdShared sh;
    const int warp = warp_value(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t raw = tc::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const GiveUp up{&sh.flag, a.status, wait_ns};
    const int64_t items = heads * blocks;

    if (threadIdx.x == 0) {
        for (int w = 0; w < 2; ++w) {
            tc::mbar_init(&sh.qfull[w], 1);
            tc::mbar_init(&sh.qempty[w], 1);
            tc::mbar_init(&sh.sfull[w], 1);
            tc::mbar_init(&sh.pready[w], 4);
            tc::mbar_init(&sh.ofull[w], 1);
            tc::mbar_init(&sh.oempty[w], 4);
        }
        for (int s = 0; s < ST; ++s) {
            tc::mbar_init(&sh.kvfull[s], 1);
            tc::mbar_init(&sh.kvempty[s], 1);
        }
        tc::mbar_init(&sh.vraw, 1);
        tc::mbar_init(&sh.mma_done, 1);
        sh.flag = 0;
    }
    if (warp == kFwdMmaWarp) {
        __syncwarp();
        tc::tmem_alloc<512>(&sh.tmem_slot);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = warp_value(sh.tmem_slot);

    if (warp >= kFwdMmaWarp) {
        tc::regs_lower<kFwdOtherRegs>();
        if (warp == kFwdLoadWarp) {
            uint32_t g = 0, nq[2] = {0, 0}, nraw = 0;
            bool ok = true;
            for (int64_t round = 0, item; ok && (item = snake_item(round)) < items; ++round) {
                const FwdItem it(a, item, heads, blocks);
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
                        zero_tile_rows<D>(smem + dst, it.L - t * kTile, kTile, lane);
                        tc::fence_smem_for_async();
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(&sh.kvfull[s]);
                    }
                    ++g;
                };
                auto queries = [&](int w) {
                    ok = up.warp_wait(&sh.qempty[w], (nq[w] & 1u) ^ 1u);
                    if (ok && lane == 0) {
                        tc::mbar_arrive_expect_tx(&sh.qfull[w], TL::bytes);
                        load_tile<D, kTile>(base + w * TL::bytes, mq, it.i0 + w * kTile, it.h, it.b, &sh.qfull[w]);
                    }
                    nq[w] += ok;
                };
                bool loaded[2] = {it.hi[0] == 0, it.hi[1] == 0};
                for (int32_t t = it.top() - 1; t >= it.bottom() && ok; --t) {
                    for (int w = 0; w < 2 && ok; ++w)
                        if (!loaded[w] && it.has(w, t)) {
                            loaded[w] = true;
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
                for (int w = 0; w < 2; ++w)
                    if (nq[w])
                        tc::mbar_wait(&sh.qfull[w], (nq[w] - 1) & 1u, kAttnDrainWaitNs);
                if (nraw)
                    tc::mbar_wait(&sh.vraw, (nraw - 1) & 1u, kAttnDrainWaitNs);
            }
        } else if (warp == kFwdMmaWarp) {
            constexpr uint32_t idesc_o = tc::idesc_f16<T>(kTile, D) | tc::kIdescBMnMajor;
            uint32_t n = 0, nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};
            bool ok = true;
            for (int64_t round = 0, item; ok && (item = snake_item(round)) < items; ++round) {
                const FwdItem it(a, item, heads, blocks);
                const int32_t top = it.top(), bottom = it.bottom();
                if (top == 0)
                    continue;
                // S_w of tile t, whose K is ring entry 2 n' (its arrival has been waited for).
                auto scores = [&](int w, int32_t t, uint32_t tile_n) {
                    if (t == it.hi[w] - 1) {
                        ok = up.warp_wait(&sh.qfull[w], nq[w] & 1u);
                        ++nq[w];
                        if (!ok)
                            return;
                        tc::fence_after_sync();
                    }
                    const uint32_t q0 = base + w * TL::bytes, k0 = base + TL::off_ring + ((2 * tile_n) % ST) * TL::bytes;
                    mma_abt<T, D>(tmem + w * kTile, q0, k0);
                    tc::commit_warp(&sh.sfull[w]);
                    if (t == it.lo[w])
                        tc::commit_warp(&sh.qempty[w]);
                };
                auto output = [&](int w, int32_t t) {
                    const bool first = t == it.hi[w] - 1;
                    ok = up.warp_wait(&sh.pready[w], np[w] & 1u);
                    ++np[w];
                    if (ok && first)
                        ok = up.warp_wait(&sh.oempty[w], (no[w] & 1u) ^ 1u);
                    if (!ok)
                        return;
                    tc::fence_after_sync();
                    const uint32_t v0 = base + TL::off_ring + ((2 * n + 1) % ST) * TL::bytes;
#pragma unroll
                    for (int ks = 0; ks < kTile / 16; ++ks)
                        tc::mma_f16_ts_warp(tmem + 2 * kTile + w * D, tmem + w * kTile + ks * 8,
                                            tc::smem_desc_sw128_mn(v0 + ks * 2048, TL::box), idesc_o, !first || ks > 0);
                    if (t == it.lo[w]) {
                        tc::commit_warp(&sh.ofull[w]);
                        ++no[w];
                    }
                };
                auto arrived = [&](uint32_t e) {
                    ok = up.warp_wait(&sh.kvfull[e % ST], (e / ST) & 1u);
                    tc::fence_after_sync();
                };
                arrived(2 * n);
#pragma unroll
                for (int w = 0; w < 2 && ok; ++w)
                    if (it.has(w, top - 1))
                        scores(w, top - 1, n);
                if (!ok)
                    break;
                tc::commit_warp(&sh.kvempty[(2 * n) % ST]);
                for (int32_t t = top - 1; t >= bottom && ok; --t, ++n) {
                    bool next = false;   // K of the next tile has arrived
                    arrived(2 * n + 1);
#pragma unroll
                    for (int w = 0; w < 2 && ok; ++w) {
                        if (it.has(w, t))
                            output(w, t);
                        if (ok && w == 1)
                            tc::commit_warp(&sh.kvempty[(2 * n + 1) % ST]);
                        if (ok && t > bottom && it.has(w, t - 1)) {
                            if (!next)
                                arrived(2 * n + 2);
                            next = true;
                            if (ok)
                                scores(w, t - 1, n + 1);
                        }
                    }
                    if (ok && next)
                        tc::commit_warp(&sh.kvempty[(2 * n + 2) % ST]);
                }
            }
            // Nothing may be in flight when the tensor memory is freed.
            tc::commit_warp(&sh.mma_done);
            tc::mbar_wait(&sh.mma_done, 0, kAttnDrainWaitNs);
        }
    } else {
        tc::regs_raise<kFwdSoftmaxRegs>();
        const int w = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // 32 tensor-memory lanes per warp, lane in bits 16..
        const uint32_t ts = tmem + lanes + w * kTile, to = tmem + lanes + 2 * kTile + w * D;
        // exp(scale x) = exp2(c x) with c > 0: a negative scale flips the scores, a zero one clears them.
        const float c = a.scale == 0.0f ? kLog2e : fabsf(a.scale) * kLog2e;
        const float pre = a.scale > 0.0f ? 1.0f : (a.scale < 0.0f ? -1.0f : 0.0f);
        uint32_t ns = 0, no = 0;
        bool ok = true;
        for (int64_t round = 0, item; ok && (item = snake_item(round)) < items; ++round) {
            const FwdItem it(a, item, heads, blocks);
            const int32_t i = it.i0 + w * kTile + (warp & 3) * 32 + lane;
            int32_t c0, c1;
            a.kept(it.off + i, it.L, c0, c1);
            const bool live = c0 < c1 && i < a.Sq;
            float m = -INFINITY, l = 0.0f;
            for (int32_t t = it.hi[w] - 1; t >= it.lo[w]; --t) {
                ok = up.warp_wait(&sh.sfull[w], ns & 1u);
                ++ns;
                if (!ok)
                    break;
                tc::fence_after_sync();
                float s[kTile];
                tc::tmem_ld128(ts, s);
                if (pre != 1.0f) {
#pragma unroll
                    for (int j = 0; j < kTile; ++j)
                        s[j] *= pre;
                }
                if (t * kTile < it.full0[w] || (t + 1) * kTile > it.full1[w]) {
                    const int32_t k0 = c0 - t * kTile, k1 = c1 - t * kTile;
#pragma unroll
                    for (int j = 0; j < kTile; ++j)
                        s[j] = j >= k0 && j < k1 ? s[j] : -INFINITY;
                }
                float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int j = 4; j < kTile; j += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = j + 4 + k < kTile ? fmaxf(fmaxf(x[k], s[j + k]), s[(j + 4 + k) % kTile]) : fmaxf(x[k], s[j + k]);
                const float top = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
                if (t == it.hi[w] - 1) {
                    m = top;
                } else {
                    const bool raise = (top - m) * c > kRescaleLog2;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? exp2_approx((m - top) * c) : 1.0f;
                        m = raise ? top : m;
                        l *= f;
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            float o[32];
                            uint32_t r[32];
                            tc::tmem_ld32(to + k, o);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                r[j] = __float_as_uint(o[j] * f);
                            tc::tmem_st32(to + k, r);
                        }
                    }
                }
                const float shift = m == -INFINITY ? 0.0f : -m * c;
                const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int k = 0; k < kTile; k += 32) {
                    uint32_t r[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float2 e = __ffma2_rn(make_float2(s[k + 2 * j], s[k + 2 * j + 1]), c2, shift2);
                        e = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                        sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                        r[j] = pack2<T>(e.x, e.y);
                    }
                    tc::tmem_st16(ts + k / 2, r);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&sh.pready[w]);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (!ok)
                break;
            T* out = a.o.row<T>(it.b, it.h, i);
            const float inv = live ? 1.0f / l : 0.0f;
            if (it.hi[w] > it.lo[w]) {
                ok = up.warp_wait(&sh.ofull[w], no & 1u);
                ++no;
                if (!ok)
                    break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    tc::tmem_ld32(to + k, o);
                    if (i < a.Sq) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (live)
                                v = make_uint4(pack2<T>(o[j] * inv, o[j + 1] * inv), pack2<T>(o[j + 2] * inv, o[j + 3] * inv),
                                               pack2<T>(o[j + 4] * inv, o[j + 5] * inv), pack2<T>(o[j + 6] * inv, o[j + 7] * inv));
                            *reinterpret_cast<uint4*>(out + k + j) = v;
                        }
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(&sh.oempty[w]);
            } else if (i < a.Sq) {
                for (int k = 0; k < D; k += 8)
                    *reinterpret_cast<uint4*>(out + k) = make_uint4(0, 0, 0, 0);
            }
            if (a.lse && i < a.Sq)
                a.lse[(static_cast<int64_t>(it.b) * a.Hq + it.h) * a.Sq + i] =
                    live ? (a.scale == 0.0f ? m : m * fabsf(a.scale)) + logf(l) : -INFINITY;
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kFwdMmaWarp) {
        __syncwarp();
        tc::tmem_free<512>(tmem);
    }
}

template <typename T, int D>
cudaError_t launch_attention_fwd_tc(const AttentionArgs& a, cudaStream_t st, uint64_t wait_ns = kAttnWaitNs)
{
    if (!bind_context())
        return cudaErrorUnknown;
    // Without keys no tile is loaded, and q stands in for k and v in the maps.
    const bool keys = a.Skv > 0;
    HeadsMap mq, mk, mv;
    if (!encode_heads<T>(mq, a.q, a.B, a.Hq, a.Sq, D, kTile) ||
        !encode_heads<T>(mk, keys ? a.k : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile) ||
        !encode_heads<T>(mv, keys ? a.v : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, kTile))
        return cudaErrorInvalidValue;
    auto* kern = gtms_attention_fwd_kernel<T, D>;
    constexpr int smem = static_cast<int>(FwdTile<D>::smem);
    const cudaError_t e = allow_smem<gtms_attention_fwd_kernel<T, D>>(smem);
    if (e != cudaSuccess)
        return e;
    const int32_t blocks = (a.Sq + kFwdRows - 1) / kFwdRows;
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hq, items = heads * blocks;
    const int nsm = device_sms();
    if (nsm <= 0)
        return cudaErrorUnknown;
    return launch_kernel(kern, static_cast<unsigned>(items < nsm ? items : nsm), kFwdThreads, smem, st, mq, mk, mv, a, heads,
                         blocks, wait_ns);
}

}  // namespace gtms
