// Test-only library (built by tests/test_attention_gpu.py, never part of libgtms):
// the attention kernels compiled with GTMS_ATTN_TMA_NO_LOADS, so their load warps
// issue no copies. No other role's wait can then complete: each runs out after
// `wait_ns` nanoseconds, and the kernels must record GTMS_ERR_TIMEOUT in the status
// word, leave their loops, free their tensor memory and return.
#define GTMS_ATTN_TMA_NO_LOADS 1
#include "gtms_attention_bwd.cuh"
#include "gtms_attention_fwd.cuh"

namespace {

template <int D>
int run(gtms::AttentionArgs a, void* workspace, void* stream, uint64_t wait_ns)
{
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!workspace)
        return static_cast<int>(gtms::launch_attention_fwd_tc<__nv_bfloat16, D>(a, st, wait_ns));
    gtms::attention_workspace(a, workspace);
    return static_cast<int>(gtms::launch_attention_bwd_tc<__nv_bfloat16, D>(a, st, wait_ns));
}

}  // namespace

// Contiguous [B, H, S, D] bf16 tensors: q, k, v, o (forward), and dout, dq, dk, dv with a workspace (backward).
extern "C" __attribute__((visibility("default"))) int gtms_test_attention_no_loads(
    void* const* tensors, float* lse, const int32_t* seq_lens, int32_t B, int32_t H, int32_t S, int32_t D, float scale,
    int32_t* status, void* workspace, void* stream, uint64_t wait_ns)
{
    gtms::AttentionArgs a{};
    gtms::HeadsRef* const ref[8] = {&a.q, &a.k, &a.v, &a.o, &a.dout, &a.dq, &a.dk, &a.dv};
    for (int i = 0; i < 8; ++i)
        *ref[i] = {tensors[i], static_cast<int64_t>(H) * S * D, static_cast<int64_t>(S) * D, D};
    a.lse = lse;
    a.seq_lens = seq_lens;
    a.status = status;
    a.B = B;
    a.Hq = a.Hkv = H;
    a.group = 1;
    a.Sq = a.Skv = S;
    a.mask_kind = GTMS_MASK_GROUPED_TRIL;
    a.scale = scale;
    return D == 64 ? run<64>(a, workspace, stream, wait_ns) : run<128>(a, workspace, stream, wait_ns);
}
