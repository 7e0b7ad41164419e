// gtms_attention_bwd.cuh -- attention's backward pass on the tensor cores.
//
//   p_ic = exp(s_ic - lse_i),  ds_ic = p_ic (do_i . v_c - D_i),  D_i = do_i . o_i
//   dv_c = sum_i p_ic do_i,  dk_c = scale sum_i ds_ic q_i,  dq_i = scale sum_c ds_ic k_c
//
// Three launches. The first forms, per query row, D and lse in base 2, so that
// the others never read o (bound by memory: one read of o and do). The second
// owns 128 keys at a time and sums dk and dv over the query tiles, and the heads,
// that keep them; the third owns 128 queries and sums dq over key tiles. Scores
// and dP are formed in both: 7 products of 128 x 128 x d per tile pair instead of
// the 5 that one pass with dq summed by atomics would take. In exchange nothing
// but the results goes through memory, no order of sums depends on timing, and
// each accumulator stays in tensor memory.
// Beside fp32 sums there are two roundings to 16 bits: p and ds, once each, for their
// products, and o, from which D is formed, by the forward. Against 64 bits they make an
// error (norms) of 1.4 to 1.65 times that of one rounding of the gradients, the more of
// it from D the fewer keys a row keeps; an exact D would take two more products.
// The launches overlap: the second starts as the first drains and the third, which
// needs only the first, as the second runs out of items ([2,32/8,4096,128] bf16: 564
// us one after the other, 528 so; [1,12/4,2611,128] fp16, window 256: 48, 38).
#pragma once

#include "gtms_attention_tc.cuh"

namespace gtms {

// Both kernels own 128 rows of one side and walk over the other side in inner tiles.
// At head dim 128 the tensor cores bound them: inner tiles of 128, two warpgroups
// on a tile's columns, one CTA per SM with all of the tensor memory. At 64 the
// products take half as long and the element-wise chain of a tile (read the scores,
// exponentiate, hand over, read dP, form dS, hand over) bounds them: inner tiles of
// 64, one warpgroup, and two CTAs per SM, whose chains fill each other's gaps
// ([32,16,2048,64] bf16: 809 us with one CTA per SM, 128 x 128 tiles and four
// warpgroups on them, 713 so).
template <int D>
struct BwdShape {
    static constexpr int inner = D == 64 ? 64 : 128, groups = inner / 64, ctas = D == 64 ? 2 : 1;
    static constexpr int warps = 4 * groups, cols = 64;                     // element-wise warps; columns of a thread
    static constexpr int mma_warp = warps, load_warp = warps + 1, deal_warp = warps + 2;
    static constexpr int threads = 32 * (warps + 4);
    static constexpr int regs = D == 64 ? 128 : 168, elem_regs = D == 64 ? 176 : 208, other_regs = D == 64 ? 80 : 88;
    static_assert(groups * elem_regs + other_regs <= (groups + 1) * regs, "register shares of one block");
    static constexpr int tmem = 512 / ctas;
    static constexpr uint32_t stage = 2048;                                 // shared memory per element-wise warp for its results
    static constexpr uint32_t bytes = kTile * D * 2, inner_bytes = inner * D * 2;   // a tile of the owned side, an inner tile
    static constexpr uint32_t box = inner * 128;                            // 64 columns of an inner tile
};

constexpr int kPrepThreads = 256, kPrepMaxBlocks = 1024;

// fp16 holds p and ds scaled by powers of two, so that neither the p of long rows
// nor the ds of small gradients falls out of its range: p <= 1 by 2^14, ds by the
// power of two that takes the bound 2 max|do_i| max|v_c| of its size to at most
// 2^14. bf16 has fp32's range and takes them as they are.
template <typename T>
constexpr int kPShift = std::is_same<T, __half>::value ? 14 : 0;

__device__ __forceinline__ float gradient_factor(float do_norm, float v_norm)
{
    const float bound = 2.0f * do_norm * v_norm;
    if (!(bound > 0.0f) || bound > 3e38f)
        return 1.0f;
    int e = 14 - (ilogbf(bound) + 1);
    e = e < -100 ? -100 : (e > 100 ? 100 : e);
    return exp2f(static_cast<float>(e));
}

// Per padded query row: kPShift - lse log2(e) (-inf where nothing is kept, which
// makes every p of the row zero) and -D, so that both are added. For fp16 also the
// largest norms of the live rows of do and of the live keys of v, one partial maximum
// per block.
// A block takes 128 rows of one head at a time, D / 8 lanes to a row, and has the
// loads of four rows in flight per thread.
template <typename T, int D>
__global__ void __launch_bounds__(kPrepThreads)
gtms_attention_bwd_prep_kernel(const AttentionArgs a, int64_t row_tiles, int64_t key_tiles)
{
    constexpr int LANES = D / 8, PER = kPrepThreads / LANES, N = 4;
    constexpr bool norms = std::is_same<T, __half>::value;
    let_next_launch_start();
    const int sub = threadIdx.x % LANES, first = threadIdx.x / LANES;
    float do_norm = 0.0f, v_norm = 0.0f;
    const int32_t tiles_q = a.Sq_pad / kTile, tiles_k = (a.Skv + kTile - 1) / kTile;
    for (int64_t w = blockIdx.x; w < row_tiles; w += gridDim.x) {
        const int64_t bh = w / tiles_q;
        const int32_t i0 = static_cast<int32_t>(w - bh * tiles_q) * kTile;
        const int32_t b = static_cast<int32_t>(bh / a.Hq), h = static_cast<int32_t>(bh - static_cast<int64_t>(b) * a.Hq);
        const int32_t off = a.offset(b), L = a.length(b);
        const T* px = a.dout.row<T>(b, h, i0) + 8 * sub;
        const T* py = a.o.row<T>(b, h, i0) + 8 * sub;
        for (int32_t r0 = first; r0 < kTile; r0 += N * PER) {
            uint4 x[N], y[N];
            float lse[N];
            bool live[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int32_t r = r0 + n * PER;
                int32_t c0 = 0, c1 = 0;
                if (i0 + r < a.Sq)
                    a.kept(off + i0 + r, L, c0, c1);
                live[n] = c0 < c1;
                x[n] = y[n] = make_uint4(0, 0, 0, 0);
                lse[n] = -INFINITY;
                if (live[n]) {
                    x[n] = __ldg(reinterpret_cast<const uint4*>(px + r * a.dout.ss));
                    y[n] = __ldg(reinterpret_cast<const uint4*>(py + r * a.o.ss));
                    if (sub == 0)
                        lse[n] = kPShift<T> - __ldg(a.lse + bh * a.Sq + i0 + r) * kLog2e;
                }
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const T* xe = reinterpret_cast<const T*>(&x[n]);
                const T* ye = reinterpret_cast<const T*>(&y[n]);
                float dot = 0.0f, sq = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float f = static_cast<float>(xe[k]);
                    dot += f * static_cast<float>(ye[k]);
                    sq += f * f;
                }
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) {
                    dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    if (norms)
                        sq += __shfl_xor_sync(0xffffffffu, sq, o);
                }
                do_norm = fmaxf(do_norm, sq);
                if (sub == 0) {
                    const int64_t at = bh * a.Sq_pad + i0 + r0 + n * PER;
                    a.delta[at] = -dot;
                    a.lse2[at] = lse[n];
                }
            }
        }
    }
    if constexpr (norms) {
        for (int64_t w = blockIdx.x; w < key_tiles; w += gridDim.x) {
            const int64_t bg = w / tiles_k;
            const int32_t c0 = static_cast<int32_t>(w - bg * tiles_k) * kTile, b = static_cast<int32_t>(bg / a.Hkv);
            const int32_t L = a.length(b);
            const T* pv = a.v.row<T>(b, bg - static_cast<int64_t>(b) * a.Hkv, c0) + 8 * sub;
            for (int32_t r0 = first; r0 < kTile; r0 += N * PER) {
                uint4 x[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int32_t r = r0 + n * PER;
                    x[n] = c0 + r < L ? __ldg(reinterpret_cast<const uint4*>(pv + r * a.v.ss)) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const T* xe = reinterpret_cast<const T*>(&x[n]);
                    float sq = 0.0f;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        sq += static_cast<float>(xe[k]) * static_cast<float>(xe[k]);
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1)
                        sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    v_norm = fmaxf(v_norm, sq);
                }
            }
        }
        __shared__ float part[2][kPrepThreads / 32];
        do_norm = team_max<32>(do_norm, nullptr);
        v_norm = team_max<32>(v_norm, nullptr);
        if ((threadIdx.x & 31) == 0) {
            part[0][threadIdx.x >> 5] = do_norm;
            part[1][threadIdx.x >> 5] = v_norm;
        }
        __syncthreads();
        if (threadIdx.x < 2) {
            float m = 0.0f;
            for (int k = 0; k < kPrepThreads / 32; ++k)
                m = fmaxf(m, part[threadIdx.x][k]);
            a.norms[threadIdx.x * kPrepMaxBlocks + blockIdx.x] = sqrtf(m);
        }
    }
}

// The factor of ds, from the partial maxima (every thread of the block calls).
template <typename T>
__device__ __forceinline__ float block_gradient_factor(const AttentionArgs& a, float* shared2)
{
    if constexpr (!std::is_same<T, __half>::value)
        return 1.0f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < 2) {
        float m = 0.0f;
        for (int k = lane; k < a.norm_blocks; k += 32)
            m = fmaxf(m, __ldcg(a.norms + warp * kPrepMaxBlocks + k));
        m = team_max<32>(m, nullptr);
        if (lane == 0)
            shared2[warp] = m;
    }
    __syncthreads();
    return gradient_factor(shared2[0], shared2[1]);
}

// Zeroes what stands outside [k0, k1).
__device__ __forceinline__ void keep_range(float (&v)[64], int32_t k0, int32_t k1)
{
#pragma unroll
    for (int k = 0; k < 64; k += 32) {
        const uint32_t keep = bits_below(k1 - k) & ~bits_below(k0 - k);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            v[k + j] = keep & (1u << j) ? v[k + j] : 0.0f;
    }
}

// What a long sum of gradients that comes out scaled by f is carried by (see
// kCarryTerms): units of 1 / f, and none where f leaves no such unit.
struct Carried {
    float unit, per_unit;

    __device__ __forceinline__ explicit Carried(float f)
    {
        const bool usable = fabsf(f) >= 1e-30f && fabsf(f) <= 1e30f;
        per_unit = usable ? f : 0.0f;
        unit = usable ? 1.0f / f : 0.0f;
    }
};

// A warp's 32 rows x COLS columns of an accumulator at `acc` (zeros where there is
// none) and, where carried, of what `out` carries, scaled by f; the lanes' rows that are
// not live are zero. A zero comes out as +0.0.
template <typename T, int COLS>
__device__ __forceinline__ void write_rows(uint8_t* stage, int lane, uint32_t acc, bool any, bool live, float f, T* out,
                                           bool carried)
{
#pragma unroll 1
    for (int k = 0; k < COLS; k += 32) {
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            r[j] = 0;
        if (any) {
            float o[32];
            tc::tmem_ld32(acc + k, o);
            if (carried && live && out)
                add_carried(o, out + k, Carried(f).unit);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                r[j] = live ? pack2<T>(o[2 * j] * f + 0.0f, o[2 * j + 1] * f + 0.0f) : 0u;
        }
        store_rows<32>(stage, lane, r, out ? out + k : nullptr);
    }
}

// ---------------------------------------------------------------------------
// dk, dv. Scores are formed transposed, S^T = K Q^T and dP^T = V dO^T, so that P^T
// and dS^T are in tensor memory as the A operands of dV += P^T dO and
// dK += dS^T Q. Tensor memory: S^T, dP^T (P^T and dS^T, 16 bits, over them, each
// warpgroup's part over its own scores), dV, dK (head_dim columns each). While the
// element-wise warps form dS of one query tile the tensor cores run dV of that
// tile and S of the next, and while they form P of the next, dK and dP.
// ---------------------------------------------------------------------------
template <int D>
struct DkvTile {
    using SH = BwdShape<D>;
    static constexpr int stages = D == 64 ? 4 : 2;
    static constexpr uint32_t off_k = 0, off_v = SH::bytes, off_q = 2 * SH::bytes, off_do = off_q + stages * SH::inner_bytes;
    static constexpr uint32_t off_rows = off_do + stages * SH::inner_bytes;   // per stage: lse2 and D of the inner rows
    static constexpr uint32_t rows_bytes = 2 * SH::inner * 4;
    static constexpr uint32_t off_out = off_rows + stages * rows_bytes;
    static constexpr uint32_t smem = off_out + SH::warps * SH::stage + 1024;   // slack to align the base
    // Tensor memory columns.
    static constexpr uint32_t t_s = 0, t_dp = SH::inner, t_dv = 2 * SH::inner, t_dk = t_dv + D;
    static_assert(t_dk + D <= SH::tmem, "tensor memory");
    // First column of the 16-bit operand's columns k on: each warpgroup's part over its own scores.
    static constexpr uint32_t packed(int k) { return k / SH::cols * SH::cols + k % SH::cols / 2; }
};

struct DkvItem {
    int32_t b, g, j, off, L, lo, hi;   // key tile j of head g; inner query tiles [lo, hi)

    __device__ __forceinline__ void set(const AttentionArgs& a, uint32_t item, uint32_t heads, int32_t inner)
    {
        // Under a causal mask the first key tiles are kept by the most rows.
        j = static_cast<int32_t>(item / heads);
        const int32_t bg = static_cast<int32_t>(item % heads);
        b = bg / a.Hkv;
        g = bg - b * a.Hkv;
        off = a.offset(b);
        L = a.length(b);
        lo = hi = 0;
        const int32_t ca = j * kTile, cb = (ca + kTile < L ? ca + kTile : L) - 1;   // live keys
        if (ca > cb)
            return;
        int32_t ra = a.mask_kind == GTMS_MASK_LENGTH ? 0 : ca, rb = L - 1;
        if (a.mask_kind == GTMS_MASK_SLIDING_WINDOW && cb + a.window - 1 < rb)
            rb = cb + a.window - 1;
        int32_t ia = ra - off, ib = rb - off;
        ia = ia > 0 ? ia : 0;
        ib = ib < a.Sq - 1 ? ib : a.Sq - 1;
        if (ia <= ib) {
            lo = ia / inner;
            hi = ib / inner + 1;
        }
    }
    __device__ __forceinline__ uint32_t steps(const AttentionArgs& a) const
    {
        return static_cast<uint32_t>(hi - lo) * static_cast<uint32_t>(a.group);
    }
};

struct DkvShared {
    uint64_t kfull, kempty, vfull, vempty;
    uint64_t qfull[4], qempty[4], dofull[4], doempty[4], raw;
    uint64_t sfull, pready, dpfull, dsready, accfull, accempty, mma_done;
    ItemSlot<DkvItem> items;
    uint32_t tmem_slot;
    int flag;
    float norm[2];
};

template <typename T, int D, bool LONG>
__global__ void __launch_bounds__(BwdShape<D>::threads, BwdShape<D>::ctas)
gtms_attention_dkv_kernel(const __grid_constant__ HeadsMap mq, const __grid_constant__ HeadsMap mk,
                          const __grid_constant__ HeadsMap mv, const __grid_constant__ HeadsMap mdo,
                          const __grid_constant__ AttentionArgs a, uint32_t heads, uint64_t wait_ns)
{
    using TL = DkvTile<D>;
    using SH = BwdShape<D>;
    constexpr int ST = TL::stages, carry_tiles = kCarryTerms<T> / SH::inner;   // inner tiles of a part of a long sum
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ DkvShared sh;
    const int warp = warp_value(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t raw = tc::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const GiveUp up{&sh.flag, a.status, wait_ns};

    if (threadIdx.x == 0) {
        uint64_t* const one[] = {&sh.kfull, &sh.kempty, &sh.vfull, &sh.vempty, &sh.raw, &sh.sfull, &sh.dpfull, &sh.accfull,
                                 &sh.mma_done};
        for (uint64_t* m : one)
            tc::mbar_init(m, 1);
        for (int s = 0; s < ST; ++s)
            for (uint64_t* m : {&sh.qfull[s], &sh.qempty[s], &sh.dofull[s], &sh.doempty[s]})
                tc::mbar_init(m, 1);
        tc::mbar_init(&sh.pready, SH::warps);
        tc::mbar_init(&sh.dsready, SH::warps);
        tc::mbar_init(&sh.accempty, SH::warps);
        init_items(sh.items, SH::warps + 2);   // load, MMA and element-wise warps
        sh.flag = 0;
    }
    if (warp == SH::mma_warp) {
        __syncwarp();
        tc::tmem_alloc<SH::tmem>(&sh.tmem_slot);
    }
    await_last_launch();       // the row statistics stand in memory
    let_next_launch_start();   // dq needs them, and nothing of this launch
    const float factor = block_gradient_factor<T>(a, sh.norm);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = warp_value(sh.tmem_slot), t_s = tmem + TL::t_s, t_dp = tmem + TL::t_dp, t_dv = tmem + TL::t_dv,
                   t_dk = tmem + TL::t_dk;

    if (warp >= SH::mma_warp) {
        tc::regs_lower<SH::other_regs>();
        if (warp == SH::deal_warp) {
            deal_items(sh.items, up, lane, a, [&](int32_t index) {
                DkvItem it;
                it.set(a, index, heads, SH::inner);
                return it;
            });
        } else if (warp == SH::load_warp) {
            uint32_t gq = 0, nk = 0, nraw = 0;
            uint32_t taken = 0;
            DkvItem it;
            uint32_t issued_q = 0, issued_do = 0, issued_k = 0, issued_v = 0;
            bool ok = true;
            while (!kAttnNoLoads && take_item(sh.items, up, lane, taken, it, ok)) {
                if (it.lo == it.hi)
                    continue;
                // An inner tile of queries or output gradients; rows that keep nothing may hold
                // anything, and 0 x NaN is NaN: they are zeroed before the tensor cores see them.
                auto rows = [&](const HeadsMap& m, uint32_t dst, int32_t i, int32_t h, uint64_t* full, uint32_t extra,
                                uint32_t rows_dst, int64_t at) {
                    const int32_t i0 = i * SH::inner;
                    const int32_t n = a.Sq - i0 < SH::inner ? a.Sq - i0 : SH::inner;
                    const int32_t za = -it.off - i0 > 0 ? -it.off - i0 : 0;
                    const int32_t zb = it.L - it.off - i0 < n ? it.L - it.off - i0 : n;
                    const bool patch = za > 0 || zb < n;
                    uint64_t* bar = patch ? &sh.raw : full;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(bar, SH::inner_bytes + extra);
                        load_tile<D, SH::inner>(base + dst, m, i0, h, it.b, bar);
                        if (extra) {
                            tc::bulk_load_1d(base + rows_dst, a.lse2 + at, extra / 2, bar);
                            tc::bulk_load_1d(base + rows_dst + extra / 2, a.delta + at, extra / 2, bar);
                        }
                    }
                    if (patch) {
                        ok = up.warp_wait(&sh.raw, nraw & 1u);
                        ++nraw;
                        if (!ok)
                            return;
                        zero_tile_rows<D, SH::inner>(smem + dst, 0, za, lane);
                        zero_tile_rows<D, SH::inner>(smem + dst, zb, n, lane);
                        tc::fence_smem_for_async();
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(full);
                    }
                };
                bool first = true;
                for (int32_t h = it.g * a.group; h < (it.g + 1) * a.group && ok; ++h)
                    for (int32_t i = it.lo; i < it.hi && ok; ++i) {
                        const uint32_t s = gq % ST, ph = ((gq / ST) & 1u) ^ 1u;
                        const int64_t at = (static_cast<int64_t>(it.b) * a.Hq + h) * a.Sq_pad + i * SH::inner;
                        if (first) {
                            ok = up.warp_wait(&sh.kempty, (nk & 1u) ^ 1u);
                            if (!ok)
                                break;
                            if (lane == 0) {
                                tc::mbar_arrive_expect_tx(&sh.kfull, SH::bytes);
                                load_tile<D, kTile, SH::inner>(base + TL::off_k, mk, it.j * kTile, it.g, it.b, &sh.kfull);
                            }
                            issued_k = nk + 1;
                        }
                        ok = up.warp_wait(&sh.qempty[s], ph);
                        if (!ok)
                            break;
                        rows(mq, TL::off_q + s * SH::inner_bytes, i, h, &sh.qfull[s], TL::rows_bytes, TL::off_rows + s * TL::rows_bytes, at);
                        if (!ok)
                            break;
                        issued_q = gq + 1;
                        if (first) {
                            ok = up.warp_wait(&sh.vempty, (nk & 1u) ^ 1u);
                            if (!ok)
                                break;
                            if (lane == 0) {
                                tc::mbar_arrive_expect_tx(&sh.vfull, SH::bytes);
                                load_tile<D, kTile, SH::inner>(base + TL::off_v, mv, it.j * kTile, it.g, it.b, &sh.vfull);
                            }
                            issued_v = nk + 1;
                            first = false;
                        }
                        ok = up.warp_wait(&sh.doempty[s], ph);
                        if (!ok)
                            break;
                        rows(mdo, TL::off_do + s * SH::inner_bytes, i, h, &sh.dofull[s], 0, 0, 0);
                        if (!ok)
                            break;
                        issued_do = gq + 1;
                        ++gq;
                    }
                ++nk;
            }
            if (!ok) {   // let the copies already issued land before the CTA can exit
                for (uint32_t k = 0; k < static_cast<uint32_t>(ST); ++k) {
                    if (k < issued_q)
                        tc::mbar_wait(&sh.qfull[(issued_q - 1 - k) % ST], ((issued_q - 1 - k) / ST) & 1u, kAttnDrainWaitNs);
                    if (k < issued_do)
                        tc::mbar_wait(&sh.dofull[(issued_do - 1 - k) % ST], ((issued_do - 1 - k) / ST) & 1u, kAttnDrainWaitNs);
                }
                if (issued_k)
                    tc::mbar_wait(&sh.kfull, (issued_k - 1) & 1u, kAttnDrainWaitNs);
                if (issued_v)
                    tc::mbar_wait(&sh.vfull, (issued_v - 1) & 1u, kAttnDrainWaitNs);
                if (nraw)
                    tc::mbar_wait(&sh.raw, (nraw - 1) & 1u, kAttnDrainWaitNs);
            }
        } else if (warp == SH::mma_warp) {
            constexpr uint32_t idesc_acc = tc::idesc_f16<T>(kTile, D) | tc::kIdescBMnMajor;
            uint32_t gq = 0, gt = 0, nk = 0, taken = 0;   // query tiles, element-wise hand-offs, items
            DkvItem it;
            bool ok = true;
            // acc += A B, A 16 bits in tensor memory and B a tile of rows.
            auto accumulate = [&](uint32_t acc, uint32_t t_a, uint32_t rows, bool more) {
#pragma unroll
                for (int ks = 0; ks < SH::inner / 16; ++ks)
                    tc::mma_f16_ts_warp(acc, t_a + TL::packed(16 * ks), tc::smem_desc_sw128_mn(rows + ks * 2048, SH::box), idesc_acc,
                                        more || ks > 0);
            };
            while (take_item(sh.items, up, lane, taken, it, ok)) {
                const int32_t n = warp_value((it.hi - it.lo) * a.group);
                if (n == 0)
                    continue;
                auto scores = [&](uint32_t q) {
                    ok = up.warp_wait(&sh.qfull[q % ST], (q / ST) & 1u);
                    if (!ok)
                        return;
                    tc::fence_after_sync();
                    mma_abt<T, D, SH::inner>(t_s, base + TL::off_k, base + TL::off_q + (q % ST) * SH::inner_bytes);
                    tc::commit_warp(&sh.sfull);
                };
                auto products = [&](uint32_t q) {
                    ok = up.warp_wait(&sh.dofull[q % ST], (q / ST) & 1u);
                    if (!ok)
                        return;
                    tc::fence_after_sync();
                    mma_abt<T, D, SH::inner>(t_dp, base + TL::off_v, base + TL::off_do + (q % ST) * SH::inner_bytes);
                    tc::commit_warp(&sh.dpfull);
                };
                ok = up.warp_wait(&sh.kfull, nk & 1u);
                if (ok)
                    scores(gq);
                if (ok && n == 1)
                    tc::commit_warp(&sh.kempty);
                if (ok)
                    ok = up.warp_wait(&sh.vfull, nk & 1u);
                if (ok)
                    products(gq);
                if (ok && n == 1)
                    tc::commit_warp(&sh.vempty);
                for (int32_t k = 0; k < n && ok; ++k, ++gq, ++gt) {
                    const bool next = k + 1 < n, last_next = k + 2 == n;
                    auto next_scores = [&] {
                        scores(gq + 1);
                        if (ok && last_next)
                            tc::commit_warp(&sh.kempty);
                    };
                    auto next_products = [&] {
                        products(gq + 1);
                        if (ok && last_next)
                            tc::commit_warp(&sh.vempty);
                    };
                    ok = ok && up.warp_wait(&sh.pready, gt & 1u);
                    if (ok && k == 0)
                        ok = up.warp_wait(&sh.accempty, (nk & 1u) ^ 1u);
                    if (!ok)
                        break;
                    tc::fence_after_sync();
                    accumulate(t_dv, t_s, base + TL::off_do + (gq % ST) * SH::inner_bytes, k > 0);
                    tc::commit_warp(&sh.doempty[gq % ST]);
                    if (next)   // P has gone: its columns take the next scores
                        next_scores();
                    ok = ok && up.warp_wait(&sh.dsready, gt & 1u);
                    if (!ok)
                        break;
                    tc::fence_after_sync();
                    accumulate(t_dk, t_dp, base + TL::off_q + (gq % ST) * SH::inner_bytes, k > 0);
                    tc::commit_warp(&sh.qempty[gq % ST]);
                    if (next)
                        next_products();
                }
                if (ok)
                    tc::commit_warp(&sh.accfull);
                ++nk;
            }
            tc::commit_warp(&sh.mma_done);   // nothing may be in flight when the tensor memory is freed
            tc::mbar_wait(&sh.mma_done, 0, kAttnDrainWaitNs);
        }
    } else {
        tc::regs_raise<SH::elem_regs>();
        const int part = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t my_s = t_s + lanes + part * SH::cols, my_dp = t_dp + lanes + part * SH::cols;
        const float c = a.scale * kLog2e;
        const float2 c2 = make_float2(c, c);
        const float fk = factor * exp2f(static_cast<float>(-kPShift<T>));
        uint32_t gt = 0, nk = 0, taken = 0;
        DkvItem it;
        bool ok = true;
        auto arrive = [&](uint64_t* bar) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(bar);
        };
        while (take_item(sh.items, up, lane, taken, it, ok)) {
            const int32_t key = it.j * kTile + row;
            const bool any = it.lo != it.hi;
            const uint32_t first = gt;
            for (int32_t h = 0; h < (any ? a.group : 0) && ok; ++h)
                for (int32_t i = it.lo; i < it.hi; ++i, ++gt) {
                    const uint32_t s = gt % ST;
                    if (LONG && (gt - first) % carry_tiles == 0 && gt != first) {
                        // dP of this tile says that the products into dK are done, and with them those into dV.
                        ok = up.warp_wait(&sh.dpfull, gt & 1u);
                        if (!ok)
                            break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int which = 0; which < 2; ++which)
                            if (SH::groups == 1 || part == which) {
                                const Carried c(which ? a.scale / factor : exp2f(static_cast<float>(-kPShift<T>)));
                                carry_accumulator<T, D>((which ? t_dk : t_dv) + lanes,
                                                        key < a.Skv ? (which ? a.dk : a.dv).row<T>(it.b, it.g, key) : nullptr,
                                                        gt - first > carry_tiles ? c.unit : 0.0f, c.unit, c.per_unit);
                            }
                    }
                    // S says that the queries' tile has arrived, and the rows' lse2 and D with it on the same barrier.
                    ok = up.warp_wait(&sh.sfull, gt & 1u);
                    if (!ok)
                        break;
                    tc::fence_after_sync();
                    const float* lse2 = reinterpret_cast<const float*>(smem + TL::off_rows + s * TL::rows_bytes) + part * SH::cols;
                    const float* delta = lse2 + SH::inner;
                    float p[SH::cols];
                    tc::tmem_ld64(my_s, p);
                    const bool multiplied = up.ask(&sh.dpfull, gt & 1u);
#pragma unroll
                    for (int j = 0; j < SH::cols; j += 4) {
                        const float4 e = *reinterpret_cast<const float4*>(lse2 + j);
                        const float2 x = __ffma2_rn(make_float2(p[j], p[j + 1]), c2, make_float2(e.x, e.y));
                        const float2 y = __ffma2_rn(make_float2(p[j + 2], p[j + 3]), c2, make_float2(e.z, e.w));
                        p[j] = exp2_approx(x.x);
                        p[j + 1] = exp2_approx(x.y);
                        p[j + 2] = exp2_approx(y.x);
                        p[j + 3] = exp2_approx(y.y);
                    }
                    const int32_t r0 = it.off + i * SH::inner;   // the tile's first position
                    if (__builtin_expect(a.mask_kind != GTMS_MASK_LENGTH &&
                                             (r0 < it.j * kTile + kTile - 1 ||
                                              (a.mask_kind == GTMS_MASK_SLIDING_WINDOW &&
                                               r0 + SH::inner - 1 >= it.j * kTile + a.window)), 0)) {
                        const int32_t k0 = key - r0 - part * SH::cols;
                        const int32_t k1 = a.mask_kind == GTMS_MASK_SLIDING_WINDOW ? k0 + a.window : SH::cols;
                        keep_range(p, k0, k1);
                    }
                    uint32_t r[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        r[j] = pack2<T>(p[2 * j], p[2 * j + 1]);
                    tc::tmem_st32(my_s, r);
                    tc::tmem_wait_st();
                    arrive(&sh.pready);
                    ok = up.warp_wait(&sh.dpfull, gt & 1u, multiplied);
                    if (!ok)
                        break;
                    tc::fence_after_sync();
                    float ds[SH::cols];
                    tc::tmem_ld64(my_dp, ds);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const int at = 2 * j;
                        const float4 e = *reinterpret_cast<const float4*>(delta + at);
                        float2 x = __fadd2_rn(make_float2(ds[at], ds[at + 1]), make_float2(e.x, e.y));
                        float2 y = __fadd2_rn(make_float2(ds[at + 2], ds[at + 3]), make_float2(e.z, e.w));
                        if (kPShift<T> != 0) {
                            x = __fmul2_rn(x, make_float2(fk, fk));
                            y = __fmul2_rn(y, make_float2(fk, fk));
                        }
                        x = __fmul2_rn(x, make_float2(p[at], p[at + 1]));
                        y = __fmul2_rn(y, make_float2(p[at + 2], p[at + 3]));
                        r[j] = pack2<T>(x.x, x.y);
                        r[j + 1] = pack2<T>(y.x, y.y);
                    }
                    tc::tmem_st32(my_dp, r);
                    tc::tmem_wait_st();
                    arrive(&sh.dsready);
                }
            if (!ok)
                break;
            if (any) {
                ok = up.warp_wait(&sh.accfull, nk & 1u);
                ++nk;
                if (!ok)
                    break;
                tc::fence_after_sync();
            }
            // A row each of dV and of dK: two warpgroups take one of them each.
#pragma unroll
            for (int which = 0; which < 2; ++which)
                if (SH::groups == 1 || part == which) {
                    T* out = key < a.Skv ? (which ? a.dk : a.dv).row<T>(it.b, it.g, key) : nullptr;
                    write_rows<T, D>(smem + TL::off_out + warp * SH::stage, lane, (which ? t_dk : t_dv) + lanes, any,
                                     key < it.L, which ? a.scale / factor : exp2f(static_cast<float>(-kPShift<T>)), out,
                                     LONG && gt - first > carry_tiles);
                }
            if (any)
                arrive(&sh.accempty);
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == SH::mma_warp) {
        __syncwarp();
        tc::tmem_free<SH::tmem>(tmem);
    }
}

// ---------------------------------------------------------------------------
// dq. S = Q K^T, dP = dO V^T (128 columns of tensor memory each), dS (16 bits,
// twice) and dQ. P never leaves the registers, so S and dP of the next key tile are
// formed as soon as this one's have been read, and dQ of this one as soon as dS is
// written.
// ---------------------------------------------------------------------------
template <int D>
struct DqTile {
    using SH = BwdShape<D>;
    static constexpr int k_stages = D == 64 ? 4 : 3, v_stages = D == 64 ? 3 : 1;
    static constexpr uint32_t off_q = 0, off_do = SH::bytes, off_k = 2 * SH::bytes, off_v = off_k + k_stages * SH::inner_bytes;
    static constexpr uint32_t off_out = off_v + v_stages * SH::inner_bytes;
    static constexpr uint32_t smem = off_out + SH::warps * SH::stage + 1024;   // slack to align the base
    // Tensor memory columns; dS twice.
    static constexpr uint32_t t_s = 0, t_dp = SH::inner, t_ds = 2 * SH::inner, t_dq = 3 * SH::inner;
    static_assert(t_dq + D <= SH::tmem, "tensor memory");
};

struct DqItem {
    int32_t b, h, i0, off, L, lo, hi, full0, full1;

    __device__ __forceinline__ void set(const AttentionArgs& a, uint32_t item, uint32_t heads, int32_t blocks, int32_t inner)
    {
        const int32_t bh = static_cast<int32_t>(item % heads);
        i0 = (blocks - 1 - static_cast<int32_t>(item / heads)) * kTile;
        b = bh / a.Hq;
        h = bh - b * a.Hq;
        off = a.offset(b);
        L = a.length(b);
        const int32_t last = i0 + kTile < a.Sq ? i0 + kTile : a.Sq;
        const int32_t ra = off + i0 > 0 ? off + i0 : 0, rb = (off + last < L ? off + last : L) - 1;
        lo = hi = full0 = full1 = 0;
        if (ra <= rb) {
            int32_t a0, a1, b0, b1;
            a.kept(ra, L, a0, a1);
            a.kept(rb, L, b0, b1);
            lo = a0 / inner;
            hi = (b1 + inner - 1) / inner;
            full0 = b0;
            full1 = a1;
        }
    }
    __device__ __forceinline__ uint32_t steps(const AttentionArgs&) const { return hi - lo; }
};

struct DqShared {
    uint64_t qfull, qempty, dofull, doempty;
    uint64_t kfull[4], kempty[4], vfull[3], vempty[3], raw;
    uint64_t sfull, sread, dpfull, dpread, accfull, accempty, mma_done;
    // One for each copy of dS: S and dP of the next tile are formed before the MMA warp waits for this one's dS,
    // so that a late MMA warp can find dS of both written. On one barrier that is two phases, which a parity bit
    // does not tell from none.
    uint64_t dsready[2];
    ItemSlot<DqItem> items;
    uint32_t tmem_slot;
    int flag;
    float norm[2];
};

template <typename T, int D, bool LONG>
__global__ void __launch_bounds__(BwdShape<D>::threads, BwdShape<D>::ctas)
gtms_attention_dq_kernel(const __grid_constant__ HeadsMap mq, const __grid_constant__ HeadsMap mk,
                         const __grid_constant__ HeadsMap mv, const __grid_constant__ HeadsMap mdo,
                         const __grid_constant__ AttentionArgs a, uint32_t heads, int32_t blocks, uint64_t wait_ns)
{
    using TL = DqTile<D>;
    using SH = BwdShape<D>;
    constexpr int KS = TL::k_stages, VS = TL::v_stages, carry_tiles = kCarryTerms<T> / SH::inner;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ DqShared sh;
    const int warp = warp_value(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t raw = tc::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const GiveUp up{&sh.flag, a.status, wait_ns};

    if (threadIdx.x == 0) {
        for (uint64_t* m : {&sh.qfull, &sh.qempty, &sh.dofull, &sh.doempty, &sh.raw, &sh.sfull, &sh.dpfull, &sh.accfull,
                            &sh.mma_done})
            tc::mbar_init(m, 1);
        for (int s = 0; s < KS; ++s) {
            tc::mbar_init(&sh.kfull[s], 1);
            tc::mbar_init(&sh.kempty[s], 1);
        }
        for (int s = 0; s < VS; ++s) {
            tc::mbar_init(&sh.vfull[s], 1);
            tc::mbar_init(&sh.vempty[s], 1);
        }
        tc::mbar_init(&sh.sread, SH::warps);
        tc::mbar_init(&sh.dpread, SH::warps);
        tc::mbar_init(&sh.dsready[0], SH::warps);
        tc::mbar_init(&sh.dsready[1], SH::warps);
        tc::mbar_init(&sh.accempty, SH::warps);
        init_items(sh.items, SH::warps + 2);   // load, MMA and element-wise warps
        sh.flag = 0;
    }
    if (warp == SH::mma_warp) {
        __syncwarp();
        tc::tmem_alloc<SH::tmem>(&sh.tmem_slot);
    }
    const float factor = block_gradient_factor<T>(a, sh.norm);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = warp_value(sh.tmem_slot), t_s = tmem + TL::t_s, t_dp = tmem + TL::t_dp, t_ds = tmem + TL::t_ds,
                   t_dq = tmem + TL::t_dq;

    if (warp >= SH::mma_warp) {
        tc::regs_lower<SH::other_regs>();
        if (warp == SH::deal_warp) {
            deal_items(sh.items, up, lane, a, [&](int32_t index) {
                DqItem it;
                it.set(a, index, heads, blocks, SH::inner);
                return it;
            });
        } else if (warp == SH::load_warp) {
            uint32_t gk = 0, gv = 0, nq = 0, ndo = 0, nraw = 0, taken = 0;
            DqItem it;
            bool ok = true;
            while (!kAttnNoLoads && take_item(sh.items, up, lane, taken, it, ok)) {
                if (it.lo == it.hi)
                    continue;
                const int32_t hk = it.h / a.group;
                auto queries = [&](const HeadsMap& m, uint32_t dst, uint64_t* full, uint64_t* empty, uint32_t& count) {
                    ok = up.warp_wait(empty, (count & 1u) ^ 1u);
                    if (!ok)
                        return;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(full, SH::bytes);
                        load_tile<D, kTile, SH::inner>(base + dst, m, it.i0, it.h, it.b, full);
                    }
                    ++count;
                };
                auto keys = [&](const HeadsMap& m, uint32_t dst, int32_t t, uint64_t* full, uint64_t* empty, uint32_t phase,
                                bool tail) {
                    ok = up.warp_wait(empty, phase ^ 1u);
                    if (!ok)
                        return;
                    uint64_t* bar = tail ? &sh.raw : full;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(bar, SH::inner_bytes);
                        load_tile<D, SH::inner>(base + dst, m, t * SH::inner, hk, it.b, bar);
                    }
                    if (tail) {   // keys behind the length meet a zero ds in dQ: they must be numbers
                        ok = up.warp_wait(&sh.raw, nraw & 1u);
                        ++nraw;
                        if (!ok)
                            return;
                        zero_tile_rows<D, SH::inner>(smem + dst, it.L - t * SH::inner, SH::inner, lane);
                        tc::fence_smem_for_async();
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(full);
                    }
                };
                for (int32_t t = it.lo; t < it.hi && ok; ++t) {
                    if (t == it.lo)
                        queries(mq, TL::off_q, &sh.qfull, &sh.qempty, nq);
                    if (ok) {
                        keys(mk, TL::off_k + (gk % KS) * SH::inner_bytes, t, &sh.kfull[gk % KS], &sh.kempty[gk % KS], (gk / KS) & 1u,
                             (t + 1) * SH::inner > it.L && it.L < a.Skv);
                        gk += ok;
                    }
                    if (ok && t == it.lo)
                        queries(mdo, TL::off_do, &sh.dofull, &sh.doempty, ndo);
                    if (ok) {
                        keys(mv, TL::off_v + (gv % VS) * SH::inner_bytes, t, &sh.vfull[gv % VS], &sh.vempty[gv % VS], (gv / VS) & 1u, false);
                        gv += ok;
                    }
                }
            }
            if (!ok) {   // let the copies already issued land before the CTA can exit
                for (uint32_t k = 0; k < static_cast<uint32_t>(KS) && k < gk; ++k)
                    tc::mbar_wait(&sh.kfull[(gk - 1 - k) % KS], ((gk - 1 - k) / KS) & 1u, kAttnDrainWaitNs);
                for (uint32_t k = 0; k < static_cast<uint32_t>(VS) && k < gv; ++k)
                    tc::mbar_wait(&sh.vfull[(gv - 1 - k) % VS], ((gv - 1 - k) / VS) & 1u, kAttnDrainWaitNs);
                if (nq)
                    tc::mbar_wait(&sh.qfull, (nq - 1) & 1u, kAttnDrainWaitNs);
                if (ndo)
                    tc::mbar_wait(&sh.dofull, (ndo - 1) & 1u, kAttnDrainWaitNs);
                if (nraw)
                    tc::mbar_wait(&sh.raw, (nraw - 1) & 1u, kAttnDrainWaitNs);
            }
        } else if (warp == SH::mma_warp) {
            constexpr uint32_t idesc_acc = tc::idesc_f16<T>(kTile, D) | tc::kIdescBMnMajor;
            uint32_t g = 0, ni = 0, taken = 0;   // key tiles, items
            DqItem it;
            bool ok = true;
            while (take_item(sh.items, up, lane, taken, it, ok)) {
                const int32_t n = warp_value(it.hi - it.lo);
                if (n == 0)
                    continue;
                auto scores = [&](uint32_t k, bool last) {
                    ok = up.warp_wait(&sh.kfull[k % KS], (k / KS) & 1u);
                    if (!ok)
                        return;
                    tc::fence_after_sync();
                    mma_abt<T, D, SH::inner>(t_s, base + TL::off_q, base + TL::off_k + (k % KS) * SH::inner_bytes);
                    tc::commit_warp(&sh.sfull);
                    if (last)
                        tc::commit_warp(&sh.qempty);
                };
                auto products = [&](uint32_t k, bool last) {
                    ok = up.warp_wait(&sh.vfull[k % VS], (k / VS) & 1u);
                    if (!ok)
                        return;
                    tc::fence_after_sync();
                    mma_abt<T, D, SH::inner>(t_dp, base + TL::off_do, base + TL::off_v + (k % VS) * SH::inner_bytes);
                    tc::commit_warp(&sh.dpfull);
                    tc::commit_warp(&sh.vempty[k % VS]);
                    if (last)
                        tc::commit_warp(&sh.doempty);
                };
                ok = up.warp_wait(&sh.qfull, ni & 1u);
                if (ok)
                    scores(g, n == 1);
                if (ok)
                    ok = up.warp_wait(&sh.dofull, ni & 1u);
                if (ok)
                    products(g, n == 1);
                for (int32_t k = 0; k < n && ok; ++k, ++g) {
                    if (k + 1 < n) {
                        ok = up.warp_wait(&sh.sread, g & 1u);
                        if (ok)
                            scores(g + 1, k + 2 == n);
                        ok = ok && up.warp_wait(&sh.dpread, g & 1u);
                        if (ok)
                            products(g + 1, k + 2 == n);
                    }
                    ok = ok && up.warp_wait(&sh.dsready[g & 1u], (g >> 1) & 1u);
                    if (ok && k == 0)
                        ok = up.warp_wait(&sh.accempty, (ni & 1u) ^ 1u);
                    if (!ok)
                        break;
                    tc::fence_after_sync();
                    const uint32_t k0 = base + TL::off_k + (g % KS) * SH::inner_bytes, ds = t_ds + (g & 1u) * (SH::inner / 2);
#pragma unroll
                    for (int ks = 0; ks < SH::inner / 16; ++ks)
                        tc::mma_f16_ts_warp(t_dq, ds + ks * 8, tc::smem_desc_sw128_mn(k0 + ks * 2048, SH::box), idesc_acc,
                                            k > 0 || ks > 0);
                    tc::commit_warp(&sh.kempty[g % KS]);
                }
                if (ok)
                    tc::commit_warp(&sh.accfull);
                ++ni;
            }
            tc::commit_warp(&sh.mma_done);   // nothing may be in flight when the tensor memory is freed
            tc::mbar_wait(&sh.mma_done, 0, kAttnDrainWaitNs);
        }
    } else {
        tc::regs_raise<SH::elem_regs>();
        const int part = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t my_s = t_s + lanes + part * SH::cols, my_dp = t_dp + lanes + part * SH::cols;
        const uint32_t my_ds = t_ds + lanes + part * (SH::cols / 2);
        const float c = a.scale * kLog2e;
        const float2 c2 = make_float2(c, c);
        const float fk = factor * exp2f(static_cast<float>(-kPShift<T>));
        uint32_t g = 0, ni = 0, taken = 0;
        DqItem it;
        bool ok = true;
        auto arrive = [&](uint64_t* bar) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(bar);
        };
        while (take_item(sh.items, up, lane, taken, it, ok)) {
            const int32_t i = it.i0 + row;
            int32_t c0, c1;
            a.kept(it.off + i, it.L, c0, c1);
            const bool live = c0 < c1 && i < a.Sq;
            const int64_t at = (static_cast<int64_t>(it.b) * a.Hq + it.h) * a.Sq_pad + i;
            const float neg_lse = __ldg(a.lse2 + at), neg_delta = __ldg(a.delta + at);
            const float2 lse2 = make_float2(neg_lse, neg_lse), delta2 = make_float2(neg_delta, neg_delta);
            constexpr int cols = D / SH::groups;
            T* out = i < a.Sq ? a.dq.row<T>(it.b, it.h, i) + part * cols : nullptr;
            bool scored = false;
            for (int32_t t = it.lo; t < it.hi; ++t, ++g) {
                if (LONG && (t - it.lo) % carry_tiles == 0 && t != it.lo) {
                    ok = up.warp_wait(&sh.kempty[(g - 1) % KS], ((g - 1) / KS) & 1u);   // the products into dQ are done
                    if (!ok)
                        break;
                    tc::fence_after_sync();
                    const Carried c(a.scale / factor);
                    carry_accumulator<T, cols>(t_dq + lanes + part * cols, out, t - it.lo > carry_tiles ? c.unit : 0.0f, c.unit,
                                               c.per_unit);
                }
                ok = up.warp_wait(&sh.sfull, g & 1u, scored);
                if (!ok)
                    break;
                tc::fence_after_sync();
                float p[SH::cols];
                tc::tmem_ld64(my_s, p);
                arrive(&sh.sread);
                const bool multiplied = up.ask(&sh.dpfull, g & 1u);
#pragma unroll
                for (int j = 0; j < SH::cols; j += 2) {
                    const float2 x = __ffma2_rn(make_float2(p[j], p[j + 1]), c2, lse2);
                    p[j] = exp2_approx(x.x);
                    p[j + 1] = exp2_approx(x.y);
                }
                ok = up.warp_wait(&sh.dpfull, g & 1u, multiplied);
                if (!ok)
                    break;
                tc::fence_after_sync();
                float ds[SH::cols];
                tc::tmem_ld64(my_dp, ds);
                arrive(&sh.dpread);
                // The columns of dS are free once dQ of the tile before last is done, which its keys' release says too.
                const bool released = g < 2 || up.ask(&sh.kempty[(g - 2) % KS], ((g - 2) / KS) & 1u);
#pragma unroll
                for (int j = 0; j < SH::cols; j += 2) {
                    float2 x = __fadd2_rn(make_float2(ds[j], ds[j + 1]), delta2);
                    if (kPShift<T> != 0)
                        x = __fmul2_rn(x, make_float2(fk, fk));
                    x = __fmul2_rn(x, make_float2(p[j], p[j + 1]));
                    ds[j] = x.x;
                    ds[j + 1] = x.y;
                }
                if (__builtin_expect(t * SH::inner < it.full0 || (t + 1) * SH::inner > it.full1, 0))
                    keep_range(ds, c0 - t * SH::inner - part * SH::cols, c1 - t * SH::inner - part * SH::cols);
                ok = up.warp_wait(&sh.kempty[(g - 2) % KS], ((g - 2) / KS) & 1u, released);
                if (!ok)
                    break;
                uint32_t r[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    r[j] = pack2<T>(ds[2 * j], ds[2 * j + 1]);
                tc::tmem_st32(my_ds + (g & 1u) * (SH::inner / 2), r);
                scored = t + 1 < it.hi && up.ask(&sh.sfull, (g + 1) & 1u);
                tc::tmem_wait_st();
                arrive(&sh.dsready[g & 1u]);
            }
            if (!ok)
                break;
            const bool any = it.lo != it.hi;
            if (any) {
                ok = up.warp_wait(&sh.accfull, ni & 1u);
                ++ni;
                if (!ok)
                    break;
                tc::fence_after_sync();
            }
            write_rows<T, cols>(smem + TL::off_out + warp * SH::stage, lane, t_dq + lanes + part * cols, any, live,
                                a.scale / factor, out, LONG && it.hi - it.lo > carry_tiles);
            if (any)
                arrive(&sh.accempty);
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == SH::mma_warp) {
        __syncwarp();
        tc::tmem_free<SH::tmem>(tmem);
    }
    await_last_launch();   // so that the end of this launch is that of the one before it too
}

template <typename T, int D>
cudaError_t launch_attention_bwd_tc(const AttentionArgs& args, cudaStream_t st, uint64_t wait_ns = kAttnWaitNs)
{
    using SH = BwdShape<D>;
    AttentionArgs a = args;
    if (!bind_context())
        return cudaErrorUnknown;
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hq, kv_heads = static_cast<int64_t>(a.B) * a.Hkv;
    // Where one side has no rows its tensors may be null: nothing of them is loaded, and the other side's
    // stand in for them in the maps.
    const bool rows = a.Sq > 0, keys = a.Skv > 0;
    HeadsMap mq, mk, mv, mdo;
    if (!encode_heads<T>(mq, rows ? a.q : a.k, a.B, a.Hq, rows ? a.Sq : 1, D, SH::inner) ||
        !encode_heads<T>(mdo, rows ? a.dout : a.k, a.B, a.Hq, rows ? a.Sq : 1, D, SH::inner) ||
        !encode_heads<T>(mk, keys ? a.k : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, SH::inner) ||
        !encode_heads<T>(mv, keys ? a.v : a.q, a.B, a.Hkv, keys ? a.Skv : 1, D, SH::inner))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    {
        constexpr bool norms = std::is_same<T, __half>::value;
        const int64_t n = heads * (a.Sq_pad / kTile), m = norms ? kv_heads * ((a.Skv + kTile - 1) / kTile) : 0;
        int64_t blocks = n > m ? n : m;
        if (norms && blocks > kPrepMaxBlocks)
            blocks = kPrepMaxBlocks;   // one partial maximum each
        a.norm_blocks = static_cast<int32_t>(blocks);
        if (blocks > 0)
            e = launch_kernel(gtms_attention_bwd_prep_kernel<T, D>, static_cast<unsigned>(blocks), kPrepThreads, 0, st, a, n, m);
    }
    // One CTA per item; the running ones take over the others' (see ItemSlot).
    auto launch_dkv = [&](auto is_long) {
        constexpr auto* kern = gtms_attention_dkv_kernel<T, D, is_long()>;
        constexpr int smem = static_cast<int>(DkvTile<D>::smem);
        const cudaError_t allowed = allow_smem<kern>(smem);
        return allowed != cudaSuccess
                   ? allowed
                   : launch_beside_last(a.norm_blocks > 0, kern, static_cast<unsigned>(kv_heads * ((a.Skv + kTile - 1) / kTile)),
                                        BwdShape<D>::threads, smem, st, mq, mk, mv, mdo, a, static_cast<uint32_t>(kv_heads), wait_ns);
    };
    auto launch_dq = [&](auto is_long) {
        constexpr auto* kern = gtms_attention_dq_kernel<T, D, is_long()>;
        constexpr int smem = static_cast<int>(DqTile<D>::smem);
        const int32_t blocks = a.Sq_pad / kTile;
        const cudaError_t allowed = allow_smem<kern>(smem);
        return allowed != cudaSuccess ? allowed
                                      : launch_beside_last(keys, kern, static_cast<unsigned>(heads * blocks), BwdShape<D>::threads, smem,
                                                           st, mq, mk, mv, mdo, a, static_cast<uint32_t>(heads), blocks, wait_ns);
    };
    if (e == cudaSuccess && keys)
        e = kept_at_most(a, a.Sq) * a.group > kCarryTerms<T> ? launch_dkv(std::true_type()) : launch_dkv(std::false_type());
    if (e == cudaSuccess && rows)
        e = kept_at_most(a, a.Skv) > kCarryTerms<T> ? launch_dq(std::true_type()) : launch_dq(std::false_type());
    return e;
}

}  // namespace gtms
