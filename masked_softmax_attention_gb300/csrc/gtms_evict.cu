// gtms_evict.cu -- eviction from a key/value cache by the weight its keys received.
//
// Of a sequence's n > keep entries stay the first `first`, the last `recent` and, of
// those between, the keep - first - recent of highest weight (ties to the lowest
// index), in the order in which they stood. Two launches:
//   select  finds them: the weight of the last one that stays by four histograms of 8
//           bits of the weights' order-preserving bits, then each entry's place by
//           counting those before it. No atomics on results, so the same inputs give
//           the same cache; a cluster of CTAs shares a long row.
//   gather  moves rows of k and v, weights and positions. What bounds the call: the
//           kept rows are read once and written once (a weight is 4 of its 4 + 4 D bytes).
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "gtms_caches.h"
#include "gtms_device.h"
#include "gtms_tcgen05.cuh"

namespace gtms {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32, kSelectCluster = 8;
// Weights that a CTA holds in shared memory; of longer shares every pass reads memory anew.
constexpr int kSelectStaged = 40960;
// Copies of a histogram, one a lane: neighbouring weights share their exponents, and 32
// lanes that count into one place would wait for each other.
constexpr int kCopies = 32;

struct SelectShared {
    uint32_t hist[256][kCopies];
    uint32_t total[2][256];        // of this CTA, by the pass's parity, so that the others may still read the last one
    uint32_t sum[256];             // over the cluster
    uint32_t digit, above;         // found: the digit, entries above it
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

template <bool STAGED>
__global__ void __launch_bounds__(kSelectThreads)
gtms_evict_select_kernel(const EvictArgs a)
{
    extern __shared__ __align__(16) uint32_t keys[];   // this CTA's share, ordered
    __shared__ SelectShared sh;
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

    // Shares: contiguous, whole warps' steps, so that a CTA's and a warp's entries precede the next one's.
    const int32_t m = hi - lo, step = 32 * kSelectWarps;
    const int32_t share = static_cast<int32_t>((static_cast<int64_t>(m) + ranks - 1) / ranks + step - 1) / step * step;
    const int64_t from64 = lo + static_cast<int64_t>(rank) * share;
    const int32_t from = static_cast<int32_t>(from64 < hi ? from64 : hi), count = hi - from < share ? hi - from : share;
    const float* mine = w + from;
    auto key_at = [&](int32_t i) { return STAGED ? keys[i] : ordered(__ldg(mine + i)); };
    if (STAGED)
        for (int32_t i = threadIdx.x; i < count; i += kSelectThreads)
            keys[i] = ordered(__ldg(mine + i));

    uint32_t prefix = 0, mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int32_t i = threadIdx.x; i < 256 * kCopies; i += kSelectThreads)
            (&sh.hist[0][0])[i] = 0;
        __syncthreads();
        for (int32_t i = threadIdx.x; i < count; i += kSelectThreads) {
            const uint32_t k = key_at(i);
            if ((k & mask) == prefix)
                atomicAdd(&sh.hist[(k >> shift) & 255u][lane % kCopies], 1u);   // counts: their order does not matter
        }
        __syncthreads();
        // A warp adds up 256 / kSelectWarps bins, a lane a copy.
        for (int d = warp; d < 256; d += kSelectWarps) {
            const uint32_t t = __reduce_add_sync(0xffffffffu, sh.hist[d][lane]);
            if (lane == 0)
                sh.total[pass & 1][d] = t;
        }
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
        if (threadIdx.x < 256) {
            uint32_t t = 0;
            for (uint32_t r = 0; r < ranks; ++r)
                t += *cluster.map_shared_rank(&sh.total[pass & 1][threadIdx.x], r);
            sh.sum[threadIdx.x] = t;
        }
        __syncthreads();
        if (warp == 0) {   // the bin in which the need-th largest stands; lane 0 has the highest eight
            uint32_t t[8], mass = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                mass += t[j] = sh.sum[255 - 8 * lane - j];
            uint32_t up = mass;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
                up += lane >= o ? x : 0;
            }
            uint32_t above = up - mass;
            if (above < need && need <= up) {
                int j = 0;
#pragma unroll
                for (int x = 0; x < 7; ++x)
                    if (j == x && above + t[x] < need) {
                        above += t[x];
                        ++j;
                    }
                sh.digit = 255 - 8 * lane - j;
                sh.above = above;
            }
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        mask |= 255u << shift;
        need -= sh.above;
    }
    // Those above `prefix` stay, and the first `need` that equal it.

    // Places: what the CTAs, warps and lanes before have.
    const int32_t part = share / kSelectWarps;   // a multiple of 32
    const int32_t w0 = warp * part < count ? warp * part : count, w1 = w0 + part < count ? w0 + part : count;
    uint32_t gt = 0, eq = 0;
    for (int32_t i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = key_at(i);
        gt += k > prefix;
        eq += k == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sh.gt[warp] = gt;
        sh.eq[warp] = eq;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t g = 0, e = 0;
        for (int i = 0; i < kSelectWarps; ++i) {
            g += sh.gt[i];
            e += sh.eq[i];
        }
        sh.cta_gt = g;
        sh.cta_eq = e;
    }
    if (ranks > 1)
        cluster.sync();
    else
        __syncthreads();
    gt = eq = 0;
    for (uint32_t r = 0; r < rank; ++r) {
        gt += *cluster.map_shared_rank(&sh.cta_gt, r);
        eq += *cluster.map_shared_rank(&sh.cta_eq, r);
    }
    for (int i = 0; i < warp; ++i) {
        gt += sh.gt[i];
        eq += sh.eq[i];
    }
    int32_t* to = kept + a.first;
    const uint32_t below = (1u << lane) - 1u;
    for (int32_t i = w0; i < w1; i += 32) {   // the whole warp
        const uint32_t k = i + lane < w1 ? key_at(i + lane) : 0u;   // 0 is no weight's key
        const uint32_t g = __ballot_sync(0xffffffffu, k > prefix), e = __ballot_sync(0xffffffffu, k == prefix && i + lane < w1);
        const uint32_t eq_before = eq + __popc(e & below);
        const bool stays = k > prefix || ((e >> lane & 1u) && eq_before < need);
        if (stays)
            to[gt + __popc(g & below) + (eq_before < need ? eq_before : need)] = from + i + lane;
        gt += __popc(g);
        eq += __popc(e);
    }
    if (ranks > 1)
        cluster.sync();   // the others may still be reading this CTA's counts
}

constexpr int kGatherThreads = 256, kGatherUnroll = 4;

// Rows go elsewhere: a CTA moves its part of one (batch, head)'s rows of k (blockIdx.y
// 0) or v. Neighbouring threads take the 16-byte units of a row.
__global__ void __launch_bounds__(kGatherThreads)
gtms_evict_gather_kernel(const EvictArgs a, int32_t parts, int32_t rows)
{
    const int which = blockIdx.y;
    const int64_t bh = blockIdx.x / parts;
    const int32_t part = static_cast<int32_t>(blockIdx.x % parts);
    const int32_t b = static_cast<int32_t>(bh / a.H), h = static_cast<int32_t>(bh - static_cast<int64_t>(b) * a.H);
    const int32_t n = a.length(b), stay = n < a.keep ? n : a.keep;
    const int32_t j0 = part * rows, j1 = stay - j0 < rows ? stay : j0 + rows;
    if (j0 >= j1 || !(a.moved >> which & 1))
        return;
    const int32_t* kept = n > a.keep ? a.kept + bh * a.keep : nullptr;
    const uint8_t* in = a.in[which].row<uint8_t>(0, 0, 0);
    uint8_t* out = a.out[which].row<uint8_t>(0, 0, 0);
    const int64_t in0 = (b * a.in[which].sb + h * a.in[which].sh) * 16, out0 = (b * a.out[which].sb + h * a.out[which].sh) * 16;
    const int32_t total = (j1 - j0) * a.units;   // rows * units stays below 2^31 (see the launch)
    for (int32_t i0 = threadIdx.x; i0 < total; i0 += kGatherThreads * kGatherUnroll) {
        int32_t from[kGatherUnroll];
        uint4 v[kGatherUnroll];
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int32_t i = i0 + u * kGatherThreads;
            if (i < total)
                from[u] = kept ? kept[j0 + i / a.units] : j0 + i / a.units;
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int32_t i = i0 + u * kGatherThreads;
            if (i < total)
                v[u] = __ldcs(reinterpret_cast<const uint4*>(in + in0 + (from[u] * a.in[which].ss + i % a.units) * 16));
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int32_t i = i0 + u * kGatherThreads;
            if (i < total)
                *reinterpret_cast<uint4*>(out + out0 + ((j0 + i / a.units) * a.out[which].ss + i % a.units) * 16) = v[u];
        }
    }
}

// Rows stay in their cache: entry j goes to row j, at or before where it stood, so a
// (batch, head)'s rows go in order, in steps: all of a step have been read (the barrier)
// before any is written, and later steps read only rows behind those that this one
// writes. What runs side by side is columns: a CTA moves `width` 16-byte units of every
// row, several steps of copies in flight in shared memory.
constexpr int kMoveStages = 4, kMoveUnroll = 4;

__global__ void __launch_bounds__(kGatherThreads)
gtms_evict_move_kernel(const EvictArgs a, int32_t slices, int32_t width)
{
    extern __shared__ __align__(16) uint4 ring[];   // kMoveStages x kMoveUnroll x threads
    const int which = blockIdx.y;
    const int64_t bh = blockIdx.x / slices;
    const int32_t unit0 = static_cast<int32_t>(blockIdx.x % slices) * width;
    const int32_t b = static_cast<int32_t>(bh / a.H), h = static_cast<int32_t>(bh - static_cast<int64_t>(b) * a.H);
    const int32_t n = a.length(b);
    if (n <= a.keep || (a.moved >> which & 1))
        return;   // everything stands where it is to stand
    const int32_t* kept = a.kept + bh * a.keep;
    // The first entries that stay are where they belong: kept[j] - j never falls.
    int32_t lo = 0, hi = a.keep;
    while (lo < hi) {
        const int32_t mid = (lo + hi) / 2;
        if (kept[mid] > mid)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int32_t w = a.units - unit0 < width ? a.units - unit0 : width;
    const int32_t rows = kGatherThreads * kMoveUnroll / w;   // of a step
    const int32_t steps = (a.keep - lo + rows - 1) / rows;
    uint8_t* base = a.in[which].row<uint8_t>(0, 0, 0) + (b * a.in[which].sb + h * a.in[which].sh + unit0) * 16;
    const int64_t ss = a.in[which].ss;
    auto load = [&](int32_t s) {
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int32_t i = u * kGatherThreads + threadIdx.x, r = i / w, j = lo + s * rows + r;
            if (s < steps && r < rows && j < a.keep)
                tc::cp_async16(tc::smem_u32(ring + (s % kMoveStages) * (kMoveUnroll * kGatherThreads) + i),
                               base + (kept[j] * ss + i % w) * 16, 16);
        }
        tc::cp_async_commit();
    };
    for (int32_t s = 0; s < kMoveStages - 1; ++s)
        load(s);
    for (int32_t s = 0; s < steps; ++s) {
        load(s + kMoveStages - 1);   // the stage of step s - 1, whose thread this is for all of its units
        asm volatile("cp.async.wait_group %0;" :: "n"(kMoveStages - 1) : "memory");
        __syncthreads();   // everyone's copies of step s have landed
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int32_t i = u * kGatherThreads + threadIdx.x, r = i / w, j = lo + s * rows + r;
            if (r < rows && j < a.keep)
                *reinterpret_cast<uint4*>(base + (j * ss + i % w) * 16) =
                    ring[(s % kMoveStages) * (kMoveUnroll * kGatherThreads) + i];
        }
    }
}

// Weights and positions. In place one CTA takes a (batch, head)'s in steps, a step held
// in shared memory until all of it has been read; otherwise a CTA takes one step.
template <int THREADS, int N>
__global__ void __launch_bounds__(THREADS)
gtms_evict_labels_kernel(const EvictArgs a, int32_t parts)
{
    constexpr int STEP = THREADS * N;
    extern __shared__ __align__(16) uint4 ring[];
    float* w = reinterpret_cast<float*>(ring);
    int32_t* p = reinterpret_cast<int32_t*>(ring) + STEP;
    const int64_t bh = blockIdx.x / parts;
    const int32_t b = static_cast<int32_t>(bh / a.H);
    const int32_t n = a.length(b), stay = n < a.keep ? n : a.keep;
    const int32_t* kept = n > a.keep ? a.kept + bh * a.keep : nullptr;
    for (int64_t j0 = static_cast<int64_t>(blockIdx.x % parts) * STEP; j0 < stay; j0 += static_cast<int64_t>(parts) * STEP) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int32_t i = u * THREADS + threadIdx.x;
            if (j0 + i < stay) {
                const int32_t from = kept ? kept[j0 + i] : static_cast<int32_t>(j0 + i);
                w[i] = a.weights[bh * a.S + from];
                p[i] = a.positions ? a.positions[bh * a.S + from] : from;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int32_t i = u * THREADS + threadIdx.x;
            if (j0 + i < stay) {
                a.weights_out[bh * a.S_out + j0 + i] = w[i];
                if (a.positions_out)
                    a.positions_out[bh * a.S_out + j0 + i] = p[i];
            }
        }
        __syncthreads();
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, unsigned block, size_t smem, unsigned ranks, cudaStream_t st, Args... args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ranks;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = ranks > 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool STAGED>
cudaError_t launch_select(const EvictArgs& a, unsigned ranks, int32_t share, cudaStream_t st)
{
    const cudaError_t e = allow_smem<gtms_evict_select_kernel<STAGED>>(kSelectStaged * 4);
    return e != cudaSuccess ? e
                            : launch(gtms_evict_select_kernel<STAGED>, dim3(static_cast<unsigned>(a.B) * a.H * ranks),
                                     kSelectThreads, STAGED ? share * 4 : 0, ranks, st, a);
}

template <int THREADS, int N>
cudaError_t launch_labels(const EvictArgs& a, int64_t heads, int64_t parts, cudaStream_t st)
{
    constexpr int smem = THREADS * N * 8;
    if (heads * parts > INT32_MAX)
        return cudaErrorNotSupported;
    const cudaError_t e = allow_smem<gtms_evict_labels_kernel<THREADS, N>>(smem);
    return e != cudaSuccess ? e
                            : launch(gtms_evict_labels_kernel<THREADS, N>, dim3(static_cast<unsigned>(heads * parts)), THREADS,
                                     smem, 1, st, a, static_cast<int32_t>(parts));
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t st)
{
    const int64_t heads = static_cast<int64_t>(a.B) * a.H;
    // Select: CTAs to a row until the chip is busy, 4096 weights to each at least.
    unsigned ranks = 1;
    while (ranks < kSelectCluster && heads * ranks < kChipSms && static_cast<int64_t>(ranks) * 8192 <= a.S)
        ranks *= 2;
    const int32_t step = 32 * kSelectWarps;
    const int32_t share = static_cast<int32_t>((static_cast<int64_t>(a.S) + ranks - 1) / ranks + step - 1) / step * step;
    cudaError_t e = share <= kSelectStaged ? launch_select<true>(a, ranks, share, st) : launch_select<false>(a, ranks, share, st);
    if (e != cudaSuccess || a.keep == 0)
        return e;
    const int32_t stay = a.keep;
    if (a.moved) {
        // Rows of a CTA: 16 turns of its threads, fewer until there are eight CTAs to a multiprocessor.
        int32_t rows = (16 * kGatherThreads * kGatherUnroll + a.units - 1) / a.units;
        while (rows > 16 && heads * 2 * ((stay + rows - 1) / rows) < 8 * kChipSms)
            rows /= 2;
        const int64_t parts = (stay + rows - 1) / rows;
        if (heads * parts > INT32_MAX)
            return cudaErrorNotSupported;
        if ((e = launch(gtms_evict_gather_kernel, dim3(static_cast<unsigned>(heads * parts), 2), kGatherThreads, 0, 1, st, a,
                        static_cast<int32_t>(parts), rows)) != cudaSuccess)
            return e;
    }
    if (a.moved != 3) {
        // Columns of a CTA: whole rows, or slices of 32 bytes at least until there are two CTAs to a multiprocessor.
        int32_t width = a.units;
        while (width > 2 && heads * 2 * ((a.units + width - 1) / width) < 2 * kChipSms)
            width = (width + 1) / 2;
        const int32_t slices = (a.units + width - 1) / width;
        constexpr int smem = kMoveStages * kMoveUnroll * kGatherThreads * 16;
        if ((e = allow_smem<gtms_evict_move_kernel>(smem)) != cudaSuccess ||
            (e = launch(gtms_evict_move_kernel, dim3(static_cast<unsigned>(heads * slices), 2), kGatherThreads, smem, 1, st, a,
                        slices, width)) != cudaSuccess)
            return e;
    }
    const bool in_place = a.weights == a.weights_out || (a.positions && a.positions == a.positions_out);
    return in_place ? launch_labels<1024, 8>(a, heads, 1, st) : launch_labels<256, 4>(a, heads, (stay + 1023) / 1024, st);
}

}  // namespace gtms
