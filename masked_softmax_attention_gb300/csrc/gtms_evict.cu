// gtms_evict.cu -- eviction from a key/value cache by the weight its keys received.
//
// Of a sequence's n > keep entries stay the first `first`, the last `recent` and, of
// those between, the keep - first - recent of highest weight (ties to the lowest
// index), in the order in which they stood. Two launches, the second's start under the
// first's end:
//   select  finds them: the weight of the last one that stays by three histograms of the
//           weights' order-preserving bits, then each entry's place by counting those
//           before it. No atomics on results, so the same inputs give the same cache; a
//           cluster of CTAs shares a long row.
//   gather  (or move, in place) takes rows of k and v, weights and positions. What bounds
//           the call: the kept rows are read once and written once (a weight is 4 of its
//           4 + 4 D bytes).
// Timed here, on the device, rows of 256 bytes: HALF, 32 sequences of 7000 to 16384 entries, 8
// heads, of which 8192 stay: 345 us, 6.3 TB/s, the selection's share some 20; and QUARTER, one
// sequence of 131072, 8 heads, of which 32768 stay: 63 us, of them 18 (64 CTAs; a cluster's
// sums of 2048 bins, two barriers each, come to 2.7 us of each histogram). The figures
// below are those of this code with the one thing changed.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "gtms_attention_tc.cuh"
#include "gtms_caches.h"

namespace gtms {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32, kSelectCluster = 8;
// Where a CTA of select has its weights: in registers, in shared memory, or, longer
// shares, in memory, which every pass reads anew. In shared memory instead of registers
// HALF takes 352 us and QUARTER 66, two such CTAs to a multiprocessor 412 and 71 (they leave
// little first-level cache for gather's loads); in memory instead of shared memory 8 heads of
// 262144, 16384 stay, 66 instead of 52.
constexpr int kSelectKeys = 16, kSelectHeld = kSelectKeys * kSelectThreads, kSelectStaged = 40960;
enum class Keys { held, staged, memory };
// Bins of a histogram (11, 11 and 10 bits), and its copies, by lane: neighbouring weights
// share their exponents, and lanes that count into one place wait for each other.
constexpr int kBins = 2048, kCopies = 4;
static_assert(kBins == 2 * kSelectThreads && kSelectWarps == 32, "two bins to a thread, a warp's count to a lane");

struct SelectShared {
    __align__(16) uint32_t hist[kBins][kCopies];
    __align__(16) uint32_t theirs[kBins];           // the ranks' counts of the bins that this one sums
    uint32_t sums[kBins / 2], groups[kBins / 64];   // their sums, and those of 32 bins
    uint32_t warp_sum[kSelectWarps];
    uint32_t digit, above, in;                // found: the digit, entries above it, entries of it
    uint32_t gt[kSelectWarps], eq[kSelectWarps];
    uint32_t cta_gt, cta_eq;
};

// Bits that order as the weights do: NaN above all, -0 and +0 alike.
__device__ __forceinline__ uint32_t ordered(float w)
{
    const uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return 0xffffffffu;
    if ((u & 0x7fffffffu) == 0)
        return 0x80000000u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <Keys WHERE>
__global__ void __launch_bounds__(kSelectThreads, 1)
gtms_evict_select_kernel(const EvictArgs a)
{
    extern __shared__ __align__(16) uint4 raw[];
    SelectShared& sh = *reinterpret_cast<SelectShared*>(raw);
    uint32_t* keys = reinterpret_cast<uint32_t*>(&sh + 1);   // this CTA's share, ordered
    let_next_launch_start();   // it waits for what this one writes
    const cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t bh = blockIdx.x / ranks;
    const int32_t b = static_cast<int32_t>(bh / a.H), n = a.length(b);
    if (threadIdx.x == 0 && rank == 0 && bh == static_cast<int64_t>(b) * a.H)
        a.lens_out[b] = n < a.keep ? n : a.keep;
    if (n <= a.keep)
        return;   // all stay: the whole cluster leaves
    const float* w = a.weights + bh * a.S;
    int32_t* kept = a.kept + bh * a.keep;

    // The entries at the ends stay.
    const int32_t lo = a.first, hi = n - a.recent;
    for (int32_t i = rank * kSelectThreads + threadIdx.x; i < a.first; i += ranks * kSelectThreads)
        kept[i] = i;
    for (int32_t i = rank * kSelectThreads + threadIdx.x; i < a.recent; i += ranks * kSelectThreads)
        kept[a.keep - a.recent + i] = hi + i;
    uint32_t need = static_cast<uint32_t>(a.keep - a.first - a.recent);
    if (need == 0)
        return;

    if (ranks > 1)
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");   // no rank writes to one that has not started

    // Shares: contiguous, whole warps' steps, so that a CTA's and a warp's entries precede the next one's.
    const int32_t m = hi - lo, step = 32 * kSelectWarps;
    const int32_t share = static_cast<int32_t>((static_cast<int64_t>(m) + ranks - 1) / ranks + step - 1) / step * step;
    const int64_t from64 = lo + static_cast<int64_t>(rank) * share;
    const int32_t from = static_cast<int32_t>(from64 < hi ? from64 : hi), count = hi - from < share ? hi - from : share;
    const float* mine = w + from;
    const int32_t part = share / kSelectWarps;   // of a warp, a multiple of 32
    const int32_t w0 = warp * part < count ? warp * part : count, w1 = w0 + part < count ? w0 + part : count;
    uint32_t held[WHERE == Keys::held ? kSelectKeys : 1];
    // f(first entry of 32, this lane's key) in the order of the warp's entries; the key behind the last is 0, which is no
    // weight's and counts in a bin that none of them has.
    auto in_order = [&](auto&& f) {
        if constexpr (WHERE == Keys::held) {
#pragma unroll
            for (int g = 0; g < kSelectKeys; g += 4)
                if (w0 + g * 32 < w1)
#pragma unroll
                    for (int j = g; j < g + 4; ++j)
                        f(w0 + j * 32, held[j]);
        } else {
            for (int32_t i = w0; i < w1; i += 32)
                f(i, i + lane >= w1 ? 0u : WHERE == Keys::staged ? keys[i + lane] : ordered(__ldg(mine + i + lane)));
        }
    };
    auto any_order = [&](auto&& f) {
        if constexpr (WHERE == Keys::held) {
            in_order([&](int32_t, uint32_t k) { f(k); });
        } else {
#pragma unroll 4
            for (int32_t i = threadIdx.x; i < count; i += kSelectThreads)
                f(WHERE == Keys::staged ? keys[i] : ordered(__ldg(mine + i)));
        }
    };
    if constexpr (WHERE == Keys::held) {
#pragma unroll
        for (int j = 0; j < kSelectKeys; ++j)
            held[j] = w0 + j * 32 + lane < w1 ? __float_as_uint(__ldg(mine + w0 + j * 32 + lane)) : 0;
    }
    if (WHERE == Keys::staged)
#pragma unroll 8
        for (int32_t i = threadIdx.x; i < count; i += kSelectThreads)
            keys[i] = ordered(__ldg(mine + i));
#pragma unroll
    for (int k = 0; k < 2; ++k)
        *reinterpret_cast<uint4*>(sh.hist[threadIdx.x + k * kSelectThreads]) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if constexpr (WHERE == Keys::held) {
#pragma unroll
        for (int g = 0; g < kSelectKeys; g += 4)
            if (w0 + g * 32 < w1)
#pragma unroll
                for (int j = g; j < g + 4; ++j)
                    held[j] = w0 + j * 32 + lane < w1 ? ordered(__uint_as_float(held[j])) : 0u;
    }

    uint32_t prefix = 0, mask = 0;
    bool tied = false;   // some of those that equal the last that stays go
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const uint32_t digits = pass < 2 ? kBins - 1u : kBins / 2 - 1u;
        any_order([&](uint32_t k) {
            if ((k & mask) == prefix)
                atomicAdd(&sh.hist[(k >> shift) & digits][lane % kCopies], 1u);   // counts: their order does not matter
        });
        __syncthreads();
        // Thread t has bins 2047 - 2 t and 2046 - 2 t: the highest first. Read, they are empty for the next pass.
        const int bin = kBins - 2 - 2 * static_cast<int>(threadIdx.x);
        uint4 *bx = reinterpret_cast<uint4*>(sh.hist[bin]), *by = reinterpret_cast<uint4*>(sh.hist[bin + 1]);
        const uint4 x = *bx, y = *by;
        *bx = *by = make_uint4(0, 0, 0, 0);
        const uint32_t low = x.x + x.y + x.z + x.w, high = y.x + y.y + y.z + y.w;
        if (ranks == 1) {
            // Entries in the bins above this thread's.
            uint32_t up = low + high;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t z = __shfl_up_sync(0xffffffffu, up, o);
                up += lane >= o ? z : 0;
            }
            if (lane == 31)
                sh.warp_sum[warp] = up;
            __syncthreads();
            const uint32_t below_me = lane < warp ? sh.warp_sum[lane] : 0;
            const uint32_t above = up - low - high + __reduce_add_sync(0xffffffffu, below_me);
            if (above < need && need <= above + low + high) {   // one thread's bins hold the need-th largest
                const bool first = need <= above + high;
                sh.digit = first ? bin + 1 : bin;
                sh.above = first ? above : above + high;
                sh.in = first ? high : low;
            }
        } else {
            // A rank sums kBins / ranks bins over the cluster: every rank hands it its counts (all ranks reading all bins of
            // all others: 7000 to 9000 cycles, this 5100).
            const int slice = kBins / static_cast<int>(ranks);
            if (pass == 0)
                asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
            *reinterpret_cast<uint2*>(cluster.map_shared_rank(&sh.theirs[rank * slice + bin % slice], bin / slice)) = make_uint2(low, high);
            cluster.sync();
            if (static_cast<int>(threadIdx.x) < slice) {
                uint32_t sum = 0;
#pragma unroll
                for (uint32_t r = 0; r < kSelectCluster; ++r)
                    sum += r < ranks ? sh.theirs[r * slice + threadIdx.x] : 0;
                sh.sums[threadIdx.x] = sum;
                sum = __reduce_add_sync(0xffffffffu, sum);
                if (lane == 0)
                    sh.groups[warp] = sum;
            }
            cluster.sync();
            if (warp == 0) {
                // The group of 32 bins that holds the need-th largest, highest first, and then the bin.
                const int per = slice / 32, g = kBins / 32 - 2 - 2 * lane;   // this lane's groups: g + 1 and g
                const uint32_t g1 = *cluster.map_shared_rank(&sh.groups[(g + 1) % per], (g + 1) / per);
                const uint32_t g0 = *cluster.map_shared_rank(&sh.groups[g % per], g / per);
                uint32_t up = g0 + g1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t z = __shfl_up_sync(0xffffffffu, up, o);
                    up += lane >= o ? z : 0;
                }
                uint32_t above = up - g0 - g1;
                const int src = __ffs(__ballot_sync(0xffffffffu, need <= up)) - 1;   // the first lane that reaches it
                const bool first = need <= above + g1;
                const int group = __shfl_sync(0xffffffffu, first ? g + 1 : g, src);
                above = __shfl_sync(0xffffffffu, first ? above : above + g1, src);
                const int mine_bin = group * 32 + 31 - lane;
                const uint32_t c = *cluster.map_shared_rank(&sh.sums[mine_bin % slice], mine_bin / slice);
                up = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t z = __shfl_up_sync(0xffffffffu, up, o);
                    up += lane >= o ? z : 0;
                }
                if (lane == __ffs(__ballot_sync(0xffffffffu, need <= above + up)) - 1) {
                    sh.digit = mine_bin;
                    sh.above = above + up - c;
                    sh.in = c;
                }
            }
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        mask |= digits << shift;
        need -= sh.above;
        tied = sh.in > need;
    }
    // Those above `prefix` stay, and the first `need` that equal it.

    // Places: what the CTAs, warps and lanes before have.
    uint32_t gt = 0, eq = 0;
    in_order([&](int32_t, uint32_t k) {
        gt += k > prefix;
        eq += k == prefix;
    });
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sh.gt[warp] = gt;
        sh.eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t g = __reduce_add_sync(0xffffffffu, sh.gt[lane]), e = __reduce_add_sync(0xffffffffu, sh.eq[lane]);
        if (lane == 0) {
            sh.cta_gt = g;
            sh.cta_eq = e;
        }
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    gt = eq = 0;
    {   // those of the CTAs before, and of this one's warps before
        const bool before = lane < static_cast<int>(rank);
        const uint32_t g = before ? *cluster.map_shared_rank(&sh.cta_gt, lane) : 0, e = before ? *cluster.map_shared_rank(&sh.cta_eq, lane) : 0;
        gt = __reduce_add_sync(0xffffffffu, g + (lane < warp ? sh.gt[lane] : 0));
        eq = __reduce_add_sync(0xffffffffu, e + (lane < warp ? sh.eq[lane] : 0));
    }
    int32_t* to = kept + a.first;
    const uint32_t below = (1u << lane) - 1u;
    if (!tied) {   // no count of those that equal it (with it HALF 347 us, QUARTER 64)
        const uint32_t at_least = prefix - 1;
        uint32_t before = gt + (eq < need ? eq : need);
        in_order([&](int32_t i, uint32_t k) {   // the whole warp
            const uint32_t g = __ballot_sync(0xffffffffu, k > at_least);
            if (k > at_least)
                to[before + __popc(g & below)] = from + i + lane;
            before += __popc(g);
        });
    } else {
        in_order([&](int32_t i, uint32_t k) {   // the whole warp
            const uint32_t g = __ballot_sync(0xffffffffu, k > prefix), e = __ballot_sync(0xffffffffu, k == prefix);
            const uint32_t eq_before = eq + __popc(e & below);
            if (k > prefix || (k == prefix && eq_before < need))
                to[gt + __popc(g & below) + (eq_before < need ? eq_before : need)] = from + i + lane;
            gt += __popc(g);
            eq += __popc(e);
        });
    }
    if (ranks > 1)
        cluster.sync();   // the others may still be reading this CTA's counts
}

constexpr int kGatherThreads = 256, kGatherUnroll = 2;

// Rows go elsewhere: a CTA moves its part of one (batch, head)'s rows of k and v, and of
// weights and positions. Neighbouring threads take the 16-byte units of a row; a thread
// has its unit of two rows of both in flight (of four, with fewer CTAs for their
// registers: HALF 363 us, QUARTER 67; of one: 351 and 63; six or eight CTAs by a limit on
// registers: 354 and 65, 385 and 71).
__global__ void __launch_bounds__(kGatherThreads)
gtms_evict_gather_kernel(const EvictArgs a, int32_t parts, int32_t rows)
{
    const int64_t bh = blockIdx.x / parts;
    const int32_t part = static_cast<int32_t>(blockIdx.x % parts);
    const int32_t b = static_cast<int32_t>(bh / a.H), h = static_cast<int32_t>(bh - static_cast<int64_t>(b) * a.H);
    const int32_t n = a.length(b), stay = n < a.keep ? n : a.keep;
    const int32_t j0 = part * rows, j1 = stay - j0 < rows ? stay : j0 + rows;
    await_last_launch();   // which wrote `kept`; every CTA waits, so that this launch ends after that one
    if (j0 >= j1)
        return;
    const int32_t* kept = n > a.keep ? a.kept + bh * a.keep : nullptr;
    const int32_t unit = threadIdx.x % a.units, mine = threadIdx.x / a.units, turn = kGatherThreads / a.units;
    const uint4 *ki = a.in[0].row<uint4>(b, h, 0) + unit, *vi = a.in[1].row<uint4>(b, h, 0) + unit;
    uint4 *ko = a.out[0].row<uint4>(b, h, 0) + unit, *vo = a.out[1].row<uint4>(b, h, 0) + unit;
    const bool take_k = (a.moved & 1) && mine < turn, take_v = (a.moved & 2) && mine < turn;
    for (int32_t j = j0 + mine; j < j1; j += turn * kGatherUnroll) {
        int32_t from[kGatherUnroll];
        uint4 kr[kGatherUnroll], vr[kGatherUnroll];
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int32_t x = j + u * turn;
            from[u] = x < j1 && kept ? kept[x] : x;
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const bool any = j + u * turn < j1;
            if (any && take_k)
                kr[u] = __ldcs(ki + from[u] * a.in[0].ss);
            if (any && take_v)
                vr[u] = __ldcs(vi + from[u] * a.in[1].ss);
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int32_t x = j + u * turn;
            if (x < j1 && take_k)
                __stcs(ko + x * a.out[0].ss, kr[u]);
            if (x < j1 && take_v)
                __stcs(vo + x * a.out[1].ss, vr[u]);
        }
    }
    if (a.moved & 4)
        for (int32_t j = j0 + threadIdx.x; j < j1; j += kGatherThreads) {
            const int32_t from = kept ? kept[j] : j;
            a.weights_out[bh * a.S_out + j] = a.weights[bh * a.S + from];
            if (a.positions_out)
                a.positions_out[bh * a.S_out + j] = a.positions ? a.positions[bh * a.S + from] : from;
        }
}

// Rows stay in their cache: entry j goes to row j, at or before where it stood, so a
// (batch, head)'s rows go in order, in steps: all of a step have been read (the barrier)
// before any is written, and later steps read only rows behind those that this one
// writes. A cluster's CTAs share the rows of a step; the copies of the steps that follow
// are in flight in shared memory meanwhile, and their rows' numbers are read a step before.
// In place HALF takes 318 us (the sequences of up to 8192 entries stay as they are; all of
// 16384: 357) and QUARTER 87; a CTA to a slice of every row's columns instead took about
// twice as long. A step of 32 KB a CTA, since the cluster's barrier takes a microsecond of each: of
// 16 KB, all of 16384, 378, and QUARTER 111; of 8 KB 367 and 156; two stages 411 and 97.
constexpr int kMoveStages = 3, kMoveUnroll = 8, kMoveCluster = 8;
constexpr int kMoveBytes = kMoveStages * kMoveUnroll * kGatherThreads * 16;

// Weights and positions in place, or one of them: all of a step have been read before
// any is written, as above.
__device__ __forceinline__ void move_labels(const EvictArgs& a, int64_t bh, const int32_t* kept, int32_t stay, int32_t rank, int32_t ranks)
{
    constexpr int N = 8, STEP = N * kGatherThreads;
    const cg::cluster_group cluster = cg::this_cluster();
    for (int32_t s = 0; s < stay; s += STEP * ranks) {
        const int32_t j0 = s + rank * STEP;
        float w[N];
        int32_t p[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int32_t i = u * kGatherThreads + threadIdx.x;
            p[u] = i < stay - j0 ? (kept ? kept[j0 + i] : j0 + i) : 0;
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const bool any = u * kGatherThreads + static_cast<int32_t>(threadIdx.x) < stay - j0;
            w[u] = any ? a.weights[bh * a.S + p[u]] : 0.f;
            p[u] = any && a.positions ? a.positions[bh * a.S + p[u]] : p[u];
        }
        cluster.sync();
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int32_t i = u * kGatherThreads + threadIdx.x;
            if (i < stay - j0) {
                a.weights_out[bh * a.S_out + j0 + i] = w[u];
                if (a.positions_out)
                    a.positions_out[bh * a.S_out + j0 + i] = p[u];
            }
        }
    }
}

// blockIdx.y: k, v, and the weights and positions; blockIdx.x: CTAs of a cluster, heads.
__global__ void __launch_bounds__(kGatherThreads)
gtms_evict_move_kernel(const EvictArgs a)
{
    extern __shared__ __align__(16) uint4 raw[];   // kMoveStages x kMoveUnroll x threads
    const cg::cluster_group cluster = cg::this_cluster();
    const int32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int which = blockIdx.y;
    const int64_t bh = blockIdx.x / ranks;
    const int32_t b = static_cast<int32_t>(bh / a.H), h = static_cast<int32_t>(bh - static_cast<int64_t>(b) * a.H);
    const int32_t n = a.length(b);
    await_last_launch();   // as above
    if (a.moved >> which & 1)
        return;
    const int32_t* kept = n > a.keep ? a.kept + bh * a.keep : nullptr;
    if (which == 2)
        return move_labels(a, bh, kept, n < a.keep ? n : a.keep, rank, ranks);
    if (!kept)
        return;   // everything stands where it is to stand
    // The first entries that stay are where they belong: kept[j] - j never falls.
    int32_t lo = 0, hi = a.keep;
    while (lo < hi) {
        const int32_t mid = (lo + hi) / 2;
        if (kept[mid] > mid)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int32_t turn = kGatherThreads / a.units, row = threadIdx.x / a.units, rows = turn * kMoveUnroll;
    const int32_t end = row < turn ? a.keep : 0;   // of this thread
    const int32_t steps = (a.keep - lo + rows * ranks - 1) / (rows * ranks), first = lo + rank * rows + row;
    uint4* base = a.in[which].row<uint4>(b, h, 0) + threadIdx.x % a.units;
    const int64_t ss = a.in[which].ss;
    auto place = [&](int32_t s, int u) { return first + s * rows * ranks + u * turn; };
    auto stage = [&](int32_t s, int u) { return raw + (s % kMoveStages * kMoveUnroll + u) * kGatherThreads + threadIdx.x; };
    int32_t from[kMoveUnroll];   // of the step that `load` copies next
    auto ask = [&](int32_t s) {
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            from[u] = s < steps && place(s, u) < end ? kept[place(s, u)] : -1;
    };
    auto load = [&](int32_t s) {
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (from[u] >= 0)
                tc::cp_async16(tc::smem_u32(stage(s, u)), base + from[u] * ss, 16);
        tc::cp_async_commit();
        ask(s + 1);
    };
    ask(0);
    for (int32_t s = 0; s < kMoveStages - 1; ++s)
        load(s);
    asm volatile("cp.async.wait_group %0;" :: "n"(kMoveStages - 2) : "memory");
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // copies of step 0 have landed
    for (int32_t s = 0; s < steps; ++s) {
        load(s + kMoveStages - 1);   // the stage of step s - 1, which this thread alone reads and writes
        asm volatile("cp.async.wait_group %0;" :: "n"(kMoveStages - 2) : "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // everyone's of step s
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // this thread's of step s + 1
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (place(s, u) < end)
                base[place(s, u) * ss] = *stage(s, u);
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ranks: CTAs of a cluster; beside: may start while the last launch still runs (see await_last_launch).
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, unsigned block, size_t smem, unsigned ranks, bool beside, cudaStream_t st,
                   Args... args)
{
    cudaLaunchAttribute attrs[2];
    cudaLaunchConfig_t cfg = {};
    if (beside) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (ranks > 1) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs].val.clusterDim.x = ranks;
        attrs[cfg.numAttrs].val.clusterDim.y = attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attrs;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <Keys WHERE>
cudaError_t launch_select(const EvictArgs& a, unsigned ranks, int32_t share, cudaStream_t st)
{
    constexpr int most = static_cast<int>(sizeof(SelectShared)) + (WHERE == Keys::staged ? kSelectStaged * 4 : 0);
    static_assert(most <= 226 * 1024, "shared memory of a CTA");
    const cudaError_t e = allow_smem<gtms_evict_select_kernel<WHERE>>(most);
    return e != cudaSuccess ? e
                            : launch(gtms_evict_select_kernel<WHERE>, dim3(static_cast<unsigned>(a.B) * a.H * ranks),
                                     kSelectThreads, sizeof(SelectShared) + (WHERE == Keys::staged ? share * 4 : 0), ranks, false,
                                     st, a);
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& args, cudaStream_t st)
{
    EvictArgs a = args;
    const int64_t heads = static_cast<int64_t>(a.B) * a.H;
    // Select: CTAs to a row as long as all run at once, 4096 weights to each at least (32 heads of 60129 weights: clusters
    // of 8, which take two turns, 63 us the call, of 4 38).
    unsigned ranks = 1;
    while (ranks < kSelectCluster && 2 * heads * ranks <= kChipSms && static_cast<int64_t>(ranks) * 8192 <= a.S)
        ranks *= 2;
    const int32_t step = 32 * kSelectWarps;
    const int32_t share = static_cast<int32_t>((static_cast<int64_t>(a.S) + ranks - 1) / ranks + step - 1) / step * step;
    cudaError_t e = share <= kSelectHeld     ? launch_select<Keys::held>(a, ranks, share, st)
                    : share <= kSelectStaged ? launch_select<Keys::staged>(a, ranks, share, st)
                                             : launch_select<Keys::memory>(a, ranks, share, st);
    if (e != cudaSuccess || a.keep == 0)
        return e;
    // Weights and positions go with whoever moves, in order where either is compacted in place.
    if (!(a.weights == a.weights_out || (a.positions && a.positions == a.positions_out)))
        a.moved |= 4;
    if (a.moved) {
        // Rows of a CTA: 4 turns of its threads (HALF 345 us; 8 turns 348, 2 turns 356, 32 turns 365), fewer until there
        // are six CTAs to a multiprocessor.
        const int32_t turn = kGatherThreads / a.units * kGatherUnroll;
        int32_t rows = 4 * turn;
        while (rows > turn && heads * ((a.keep + rows - 1) / rows) < 6 * kChipSms)
            rows /= 2;
        const int64_t parts = (a.keep + rows - 1) / rows;
        if (heads * parts > INT32_MAX)
            return cudaErrorNotSupported;
        if ((e = launch(gtms_evict_gather_kernel, dim3(static_cast<unsigned>(heads * parts)), kGatherThreads, 0, 1, true, st, a,
                        static_cast<int32_t>(parts), rows)) != cudaSuccess)
            return e;
    }
    if (a.moved != 7) {
        // CTAs of a cluster to a head's rows until there are two to a multiprocessor, each with rows for two steps at least.
        const int64_t rows = kGatherThreads / a.units * kMoveUnroll;
        unsigned ranks = 1;
        while (ranks < kMoveCluster && heads * 2 * ranks < 2 * kChipSms && 4 * ranks * rows <= a.keep)
            ranks *= 2;
        if ((e = allow_smem<gtms_evict_move_kernel>(kMoveBytes)) == cudaSuccess)
            e = launch(gtms_evict_move_kernel, dim3(static_cast<unsigned>(heads * ranks), 3), kGatherThreads, kMoveBytes, ranks, true,
                       st, a);
    }
    return e;
}

}  // namespace gtms
