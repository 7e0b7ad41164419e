// gtms_attention_tc.cuh -- what the tensor-core attention kernels share: tensor
// maps of strided heads, the give-up protocol of their waits, tile loads.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gtms_attention.h"
#include "gtms_attn_tma.cuh"
#include "gtms_device.h"
#include "gtms_tcgen05.cuh"

namespace gtms {

constexpr int kTile = 128;   // rows and columns of one score tile

// Where a test build makes chosen warps late: before every wait of theirs.
#ifndef GTMS_ATTENTION_BEFORE_WAIT
#define GTMS_ATTENTION_BEFORE_WAIT()
#endif

// A strided [B, H, S, D] tensor as a 4-D map (d, s, h, b) of 64-column boxes with
// the 128-byte swizzle. Rows past S read as zero. A broadcast dimension (stride 0)
// becomes an extent of one, and the kernels' coordinates along it are multiplied
// by 0 (mh, mb).
struct HeadsMap {
    CUtensorMap map;
    int32_t mh, mb;
};

// Makes the current device's context this thread's: the tensor-map encoder is a
// driver call, and a thread whose first CUDA call it is (autograd's, say) has none yet.
inline bool bind_context()
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

template <typename T>
inline bool encode_heads(HeadsMap& m, const HeadsRef& t, int64_t B, int64_t H, int64_t S, int64_t D, uint32_t rows)
{
    const TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc)
        return false;
    m.mh = H > 1 && t.sh != 0;
    m.mb = B > 1 && t.sb != 0;
    // A stride that is never stepped over still has to be a legal one.
    const int64_t any = D;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(m.mh ? H : 1),
                                static_cast<cuuint64_t>(m.mb ? B : 1)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(S > 1 ? t.ss : any) * 2, static_cast<cuuint64_t>(m.mh ? t.sh : any) * 2,
                                   static_cast<cuuint64_t>(m.mb ? t.sb : any) * 2};
    const cuuint32_t box[4] = {64, rows, 1, 1}, estr[4] = {1, 1, 1, 1};
    return enc(&m.map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, t.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows row0 .. row0 + ROWS - 1 of head (h, b), as 64-column blocks of ROWS x 128
// bytes; the map's boxes are BOX rows high.
template <int D, int ROWS, int BOX = ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const HeadsMap& m, int32_t row0, int32_t h, int32_t b, uint64_t* bar)
{
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
#pragma unroll
        for (int y = 0; y < ROWS; y += BOX)
            tc::tma_load_4d(dst + (x * ROWS + y) * 128, &m.map, x * 64, row0 + y, h * m.mh, b * m.mb, bar);
}

// Every wait of these kernels is bounded (limit_ns, or for a whole item that much for
// each of its tiles, see item_wait): one that runs out raises the flag and
// the caller's status word, and every other role leaves its loop at the next wait
// that does not succeed at once.
struct GiveUp {
    int* flag;
    int32_t* status;
    uint64_t limit_ns;

    __device__ __forceinline__ bool raised() const { return *reinterpret_cast<const volatile int*>(flag) != 0; }
    __device__ __forceinline__ void raise() const
    {
        *reinterpret_cast<volatile int*>(flag) = 1;
        if (status)
            atomicOr(status, GTMS_ERR_TIMEOUT);
    }
    // With a limit of 4 (*tiles + 1) times limit_ns where `tiles` is given.
    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const volatile uint32_t* tiles = nullptr) const
    {
        GTMS_ATTENTION_BEFORE_WAIT();
        if (tc::mbar_try_wait(bar, parity))
            return true;
        const uint64_t t0 = tc::globaltimer_ns();
        for (;;) {
            if (tc::mbar_try_wait(bar, parity))
                return true;
            if (raised())
                return false;
            if (tc::globaltimer_ns() - t0 >= (tiles ? 4 * (uint64_t(*tiles) + 1) * limit_ns : limit_ns)) {
                raise();
                return false;
            }
        }
    }
    // Beside busy tensor cores shared memory answers slowly, and even a wait for a
    // phase that has long completed stalls a warp for 100 to 200 cycles. So a phase
    // that is expected to have completed is asked after ahead of the work that
    // precedes its use, and only the answer is looked at there.
    __device__ __forceinline__ bool ask(uint64_t* bar, uint32_t parity) const { return tc::mbar_test(bar, parity); }
    __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, bool asked) const
    {
        return __all_sync(0xffffffffu, asked) || warp_wait(bar, parity);
    }
    // All 32 lanes wait; the verdict is the warp's, so that warp-collective
    // instructions that follow stay converged.
    __device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    }
    // A wait that lasts as long as work on so many tiles, each with a few hand-offs.
    __device__ __forceinline__ bool warp_wait_tiles(uint64_t* bar, uint32_t parity, const volatile uint32_t* tiles) const
    {
        return __all_sync(0xffffffffu, wait(bar, parity, tiles)) != 0;
    }
};

// Launches that follow each other in a stream and may overlap: a kernel lets the next
// one start (once every CTA of its own has said so or has gone), and that one waits
// for the end of this, with all of its writes, where it needs it.
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_last_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... KArgs, typename... Args>
inline cudaError_t launch_beside_last(bool beside, void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem,
                                      cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Zeroes rows [from, to) of a swizzled tile of ROWS rows (a whole warp works).
template <int D, int ROWS>
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int32_t from, int32_t to, int lane)
{
    for (int32_t x = 0; x < D / 64; ++x)
        for (int32_t i = from * 8 + lane; i < to * 8; i += 32)   // 16-byte chunks, 8 to a row
            *reinterpret_cast<uint4*>(tile + x * ROWS * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// The value of lane 0, for the compiler a warp's one value.
__device__ __forceinline__ int warp_value(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Work items. The grid has one CTA per item, costliest first, but only as many run
// as the multiprocessors hold: each, its own item handed out, asks the hardware
// for another CTA's in its place, so that whoever is done first takes the next one
// (a static deal leaves CTAs idle when lengths differ), and its pipelines run on
// from item to item. One warp works the items out and deals them to the others
// through shared memory, one item ahead of their use, which keeps the index
// arithmetic and the loads of lengths out of their way.
template <typename Item>
struct ItemSlot {
    __align__(16) uint4 response;
    uint64_t full, empty, answered;
    uint32_t longest;   // tiles of the longest item dealt yet
    Item item;
};

template <typename Item>
__device__ __forceinline__ void init_items(ItemSlot<Item>& s, int readers)
{
    tc::mbar_init(&s.full, 1);
    tc::mbar_init(&s.empty, readers);
    tc::mbar_init(&s.answered, 1);
    s.longest = 0;
}

// Waits for an item to be dealt, for all readers to have taken it, and for its first
// results by a reader that had no rows in the one before it, last as long as a warp is
// busy with the one before. An item has as many tiles as rows or keys and shared heads
// make, so the limit goes by the longest one yet, and is read only once the wait has not
// succeeded at once; the waits inside an item, whose limit is a hand-off's, end these
// too where they run out, by the raised flag.
template <typename Item>
__device__ __forceinline__ bool item_wait(const ItemSlot<Item>& s, const GiveUp& up, uint64_t* bar, uint32_t parity)
{
    return up.warp_wait_tiles(bar, parity, &s.longest);
}

// The dealing warp: make(index, steps) is the item of a CTA index, of `steps` tiles
// that a warp walks over; an item with b < 0 ends the deal. The next item is asked
// for once every reader has taken the last. Where a role has given up, the CTAs that are
// left are taken over all the same and dropped, so that a grid that cannot make progress
// ends at once and not CTA by CTA.
template <typename Item, typename Make>
__device__ __forceinline__ void deal_items(ItemSlot<Item>& s, const GiveUp& up, int lane, Make make)
{
    int32_t index = blockIdx.x;
    bool ok = true;
    for (uint32_t n = 0; index >= 0; ++n) {
        if (n > 0) {
            ok = ok && item_wait(s, up, &s.empty, (n - 1) & 1u);
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&s.answered, 16);
                tc::next_cta_request(tc::smem_u32(&s.response), &s.answered);
            }
            __syncwarp();
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&s.answered, (n - 1) & 1u, kAttnDrainWaitNs))) {
                up.raise();
                return;
            }
            index = tc::next_cta_index(tc::smem_u32(&s.response));
            tc::fence_smem_for_async();   // the response has been read before the next one may land
            __syncwarp();
        }
        if (!ok)
            continue;
        Item it;
        it.b = -1;
        uint32_t steps = 0;
        if (index >= 0) {
            it = make(index, steps);
        }
        if (lane == 0) {
            s.item = it;
            if (steps > s.longest)
                *reinterpret_cast<volatile uint32_t*>(&s.longest) = steps;
            tc::mbar_arrive(&s.full);
        }
    }
}

// The same with make(index), whose steps(a) are the tiles.
template <typename Item, typename Make>
__device__ __forceinline__ void deal_items(ItemSlot<Item>& s, const GiveUp& up, int lane, const AttentionArgs& a, Make make)
{
    deal_items(s, up, lane, [&](int32_t index, uint32_t& steps) {
        const Item it = make(index);
        steps = it.steps(a);
        return it;
    });
}

// The next item, for a reading warp (n counts its items), handed to read() while it
// stands in shared memory; false at the end of the deal or where a role gave up.
template <typename Item, typename Read>
__device__ __forceinline__ bool take_item(ItemSlot<Item>& s, const GiveUp& up, int lane, uint32_t& n, bool& ok, Read read)
{
    ok = ok && item_wait(s, up, &s.full, n & 1u);
    if (!ok)
        return false;
    const bool more = s.item.b >= 0;
    if (more)
        read(s.item);
    __syncwarp();
    if (lane == 0)
        tc::mbar_arrive(&s.empty);
    ++n;
    return more;
}
template <typename Item>
__device__ __forceinline__ bool take_item(ItemSlot<Item>& s, const GiveUp& up, int lane, uint32_t& n, Item& it, bool& ok)
{
    return take_item(s, up, lane, n, ok, [&](const Item& x) { it = x; });
}

// A warp's 32 rows x COLS columns of results, 16 bits each, through shared memory
// (64 COLS bytes, 16-byte chunks swizzled by row) so that neighbouring lanes write
// a row's bytes together: straight from the rows' owners every store would touch
// 32 lines. `row` is the address of this lane's row's columns, null where it is
// not written.
template <int COLS>
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint32_t (&v)[COLS / 2], void* row)
{
    constexpr int CH = COLS / 8, ROWS = 32 / CH;   // chunks of a row, rows of one store
    __syncwarp();
#pragma unroll
    for (int j = 0; j < CH; ++j)
        *reinterpret_cast<uint4*>(stage + lane * (16 * CH) + ((j ^ (lane % 8 * CH / 8)) << 4)) =
            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    __syncwarp();
    const uint64_t mine = reinterpret_cast<uint64_t>(row);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int r = ROWS * k + lane / CH, j = lane % CH;
        const uint64_t to = __shfl_sync(0xffffffffu, mine, r);
        const uint4 x = *reinterpret_cast<const uint4*>(stage + r * (16 * CH) + ((j ^ (r % 8 * CH / 8)) << 4));
        if (to)
            *reinterpret_cast<uint4*>(to + 16 * j) = x;
    }
}

// S (or dP) = A B^T: K-major operands of 128 and N rows x D (a whole warp calls).
template <typename T, int D, int N>
__device__ __forceinline__ void mma_abt(uint32_t d, uint32_t a, uint32_t b)
{
    constexpr uint32_t idesc = tc::idesc_f16<T>(kTile, N);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {   // 16 columns of a swizzled 64-column block
        const uint32_t at = (ks & 3) * 32;
        tc::mma_f16_warp(d, tc::smem_desc_sw128(a + (ks >> 2) * (kTile * 128) + at, 1024),
                         tc::smem_desc_sw128(b + (ks >> 2) * (N * 128) + at, 1024), idesc, ks > 0);
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if constexpr (std::is_same_v<T, __half>)
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// Long sums. The tensor cores' fp32 accumulators cut off what does not fit instead of
// rounding it, so that every product of 16 terms can lose a unit in the last place, toward
// zero: a sum of 2^20 terms of one sign comes out 0.5 to 0.7 % short. So after every
// kCarryTerms terms the thread that owns a row of results takes the part that 16 bits
// hold out of the accumulator and carries it in the result's own place in memory, which
// nobody else reads; the rest, exact in fp32, stays in. The next part is added to it
// there, and in the end the last one. Sums of up to kCarryTerms terms stay as they are,
// short by 2e-4 at most in fp16 and 9e-4 in bf16, where half a step is 5e-4 and 4e-3.
// Kernels come with (LONG) and without the code for it: its mere presence costs the shorter
// sums of every other call 1 to 4 % (forward 271 -> 275 and 242 -> 249 us, backward 577 ->
// 581 and 712 -> 741 at [4,32/8,4096,128], [32,16,2048,64], [2,32/8,4096,128] and
// [32,16,2048,64]).
template <typename T>
constexpr int kCarryTerms = std::is_same<T, __half>::value ? 1 << 15 : 1 << 17;

// Keys that a tile of 128 rows keeps at most, and rows that keep one of a tile of 128 keys.
inline int64_t kept_at_most(const AttentionArgs& a, int32_t extent)
{
    const int32_t reach = a.window + kTile;
    return a.mask_kind == GTMS_MASK_SLIDING_WINDOW && reach < extent ? reach : extent;
}

// x += unit times what row `at` carries.
template <typename T, int N>
__device__ __forceinline__ void add_carried(float (&x)[N], const T* at, float unit)
{
#pragma unroll
    for (int j = 0; j < N; j += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(at + j);
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[j + k] += unit * static_cast<float>(e[k]);
    }
}

// Carries round(x / unit), finite always, and leaves the rest in x (per_unit = 1 / unit).
template <typename T, int N>
__device__ __forceinline__ void carry(float (&x)[N], T* at, float unit, float per_unit)
{
    constexpr float top = std::is_same<T, __half>::value ? 65504.0f : 3.3895313892515355e38f;
#pragma unroll
    for (int j = 0; j < N; j += 8) {
        uint4 v;
        uint32_t* r = reinterpret_cast<uint32_t*>(&v);
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            r[k] = pack2<T>(fminf(fmaxf(x[j + 2 * k] * per_unit, -top), top), fminf(fmaxf(x[j + 2 * k + 1] * per_unit, -top), top));
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[j + k] -= unit * static_cast<float>(e[k]);
        *reinterpret_cast<uint4*>(at + j) = v;
    }
}

// The same for COLS columns of an accumulator at `acc` (a whole warp calls; a lane
// without a row passes null): what row `at` carries already counts `before` each.
template <typename T, int COLS>
__device__ __forceinline__ void carry_accumulator(uint32_t acc, T* at, float before, float unit, float per_unit)
{
#pragma unroll 1
    for (int k = 0; k < COLS; k += 16) {
        float x[16];
        uint32_t r[16];
        tc::tmem_ld16(acc + k, x);
        if (at) {
            if (before != 0.0f)
                add_carried(x, at + k, before);
            carry(x, at + k, unit, per_unit);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
            r[j] = __float_as_uint(x[j]);
        tc::tmem_st16(acc + k, r);
    }
    tc::tmem_wait_st();
}

// The lowest n bits, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t bits_below(int32_t n)
{
    return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u);
}

// 2^x, off by 2^-22 of it at most, far below the rounding to 16 bits that follows; results below 2^-126 are zero
// beside a row's largest probability of 1.
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// D += A B on registers: A 16 x 16 (rows by lane / 4), B 16 x 8, fp32 sums.
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes that are read once, zero where !use (nothing is read then).
template <typename T>
__device__ __forceinline__ uint4 load_once(const T* p, bool use)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (use)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

}  // namespace gtms
