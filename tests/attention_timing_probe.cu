// Test-only library (built by tests/test_attention_timing_gpu.py, never part of
// libgtms): the attention kernels with chosen warps late before every wait of theirs.
// Hand-offs must hold whatever the warps' pace, so the results are those of the
// normal build, bit for bit.
#include <cstdint>

__device__ uint32_t gtms_late_warps;   // bit w: warp w of every CTA
__device__ uint32_t gtms_late_ns;

#define GTMS_ATTENTION_BEFORE_WAIT()                    \
    if ((gtms_late_warps >> (threadIdx.x >> 5)) & 1u)   \
    __nanosleep(gtms_late_ns)
#include "gtms_attention_bwd.cuh"
#include "gtms_attention_fwd.cuh"

namespace {

template <int D>
cudaError_t run(gtms::AttentionArgs a, void* workspace, cudaStream_t st, uint64_t wait_ns)
{
    if (!workspace)
        return gtms::launch_attention_fwd_tc<__nv_bfloat16, D>(a, st, wait_ns);
    gtms::attention_workspace(a, workspace);
    return gtms::launch_attention_bwd_tc<__nv_bfloat16, D>(a, st, wait_ns);
}

}  // namespace

// Contiguous bf16 tensors: q, k, v, o (forward, without a workspace), and dout, dq, dk, dv with one (backward).
// Waits run out after wait_ns.
extern "C" __attribute__((visibility("default"))) int gtms_test_attention_late(
    void* const* tensors, float* lse, const int32_t* seq_lens, const int32_t* q_offsets, int32_t B, int32_t Hq, int32_t Hkv,
    int32_t Sq, int32_t Skv, int32_t D, float scale, int32_t mask_kind, uint32_t late_warps, uint32_t late_ns, int32_t* status, void* workspace, void* stream,
    uint64_t wait_ns)
{
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    gtms::AttentionArgs a{};
    gtms::HeadsRef* const ref[8] = {&a.q, &a.k, &a.v, &a.o, &a.dout, &a.dq, &a.dk, &a.dv};
    for (int i = 0; i < 8; ++i) {
        const bool of_k = i == 1 || i == 2 || i >= 6;
        const int64_t H = of_k ? Hkv : Hq, row = D, head = (of_k ? Skv : Sq) * row;
        *ref[i] = {tensors[i], H * head, head, row};
    }
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
    a.scale = scale;
    cudaError_t e = cudaMemcpyToSymbolAsync(gtms_late_warps, &late_warps, 4, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(gtms_late_ns, &late_ns, 4, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = D == 64 ? run<64>(a, workspace, st, wait_ns) : run<128>(a, workspace, st, wait_ns);
    return static_cast<int>(e);
}
