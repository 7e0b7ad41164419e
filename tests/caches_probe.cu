// Test-only library (built by tests/test_caches_timing_gpu.py, never part of libgtms): the
// key-weight and shared-prefix kernels with chosen warps late before every wait of theirs,
// and with time limits of the caller's. Hand-offs must hold whatever the warps' pace, so
// the results are those of the normal build, bit for bit. Compiled with
// GTMS_ATTN_TMA_NO_LOADS=1 as well: no copy is issued, no wait can complete, and the
// kernels must record GTMS_ERR_TIMEOUT, leave their loops and return.
#include <cstdint>

__device__ uint32_t gtms_late_warps;   // bit w: warp w of every CTA
__device__ uint32_t gtms_late_ns;

#define GTMS_ATTENTION_BEFORE_WAIT()                    \
    if ((gtms_late_warps >> (threadIdx.x >> 5)) & 1u)   \
    __nanosleep(gtms_late_ns)
#include "gtms_key_weights_tc.cuh"
#include "gtms_shared_prefix.cuh"

namespace {

gtms::HeadsRef heads(void* p, int64_t H, int64_t S, int64_t D) { return {p, H * S * D, S * D, D}; }

}  // namespace

// Contiguous bf16 tensors q, k, v, o, k_prefix, v_prefix. what: 0 key weights (into `weights`; the workspace takes
// partial sums), 1 rows of their own over a prefix, 2 packed rows (the workspace as large as the plan asks).
extern "C" __attribute__((visibility("default"))) int gtms_test_caches(
    int32_t what, void* const* tensors, float* lse, float* weights, const int32_t* seq_lens, const int32_t* q_offsets, int32_t B,
    int32_t Hq, int32_t Hkv, int32_t Sq, int32_t Skv, int32_t D, int32_t G, int32_t P, float scale, int32_t mask_kind, int32_t window,
    uint32_t late_warps, uint32_t late_ns, int32_t* status, void* workspace, void* stream, uint64_t wait_ns)
{
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    gtms::AttentionArgs a{};
    a.q = heads(tensors[0], Hq, Sq, D);
    a.k = heads(tensors[1], Hkv, Skv, D);
    a.v = heads(tensors[2], Hkv, Skv, D);
    a.o = heads(tensors[3], Hq, Sq, D);
    a.lse = lse;
    a.seq_lens = seq_lens;
    a.q_offsets = q_offsets;
    a.status = status;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.group = Hq / Hkv;
    a.Sq = Sq;
    a.Skv = Skv;
    a.mask_kind = mask_kind;
    a.window = window;
    a.scale = scale;
    gtms::PrefixArgs p{};
    p.k = heads(tensors[4], Hkv, P, D);
    p.v = heads(tensors[5], Hkv, P, D);
    p.G = G;
    p.P = P;
    p.n = G > 0 ? B / G : 0;
    cudaError_t e = cudaMemcpyToSymbolAsync(gtms_late_warps, &late_warps, 4, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(gtms_late_ns, &late_ns, 4, 0, cudaMemcpyHostToDevice, st);
    if (e != cudaSuccess)
        return static_cast<int>(e);
    auto run = [&](auto dim) {
        constexpr int d = dim();
        if (what == 0) {
            gtms::KeyWeightsArgs w{};
            w.a = a;
            w.weights = weights;
            w.parts = static_cast<float*>(workspace);
            return gtms::launch_key_weights_tc<__nv_bfloat16, d>(w, st, wait_ns);
        }
        if (what == 1)
            return gtms::launch_prefixed_whole<__nv_bfloat16, d>(a, p, st, wait_ns);
        return gtms::launch_prefix_packed<__nv_bfloat16, d>(a, p, gtms::packed_plan<d>(a, p), workspace, st, wait_ns);
    };
    return static_cast<int>(D == 64 ? run(std::integral_constant<int, 64>()) : run(std::integral_constant<int, 128>()));
}
