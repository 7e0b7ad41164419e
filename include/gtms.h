/*
 * gtms.h -- C ABI of libgtms: the grouped-tril masked softmax over attention
 * scores, forward and backward, as hand-written CUDA kernels for sm_103a.
 *
 * The operation ("Attention-Mask-Optimization" README, section
 * "算子行为（融合下面的计算）", operator behaviour, and its printed worked
 * example): X is a contiguous row-major [B, M, S, S] tensor of attention
 * scores (B batches, M heads, S x S scores per head). For batch b with
 * valid length L = seq_lens[b], entry (r, c) is kept iff r < L, c < L and
 * c <= r; the same mask applies to every head. The kept entries of each row
 * are passed through a softmax of scale * x ("优化ScaledMaskSoftmax算子",
 * section 4.1: the scale sits inside the exponent); every masked entry is
 * written as +0.0, and rows r >= L are all +0.0. The mask is computed from
 * (r, c, seq_lens[b]) inside the kernel and never read from memory (the
 * README's implementation idea, "实现思路"); masked inputs are never loaded.
 *
 * The backward ("ops(8): self-attention 的 CUDA 实现及优化 (下)", section 2.1,
 * Softmax 求导: dy_i/dx_j = y_i (delta_ij - y_j); section 2.2 applies the scale
 * in the softmax backward) is dx = scale * y * (dy - rowsum(dy * y)) on kept
 * entries and +0.0 on masked ones.
 *
 * Values of seq_lens outside [0, S] are clamped to that range in the kernel.
 * Arithmetic is fp32 for every IO dtype; outputs are rounded to the IO dtype
 * to nearest, ties to even.
 *
 * Ownership and threading. The caller owns every buffer. All tensor
 * pointers are addresses the current CUDA device can dereference: device
 * memory, or page-locked host memory mapped with gtms_device_pointer_of_host;
 * seq_lens is an int32[B] array in such memory. The library allocates
 * nothing, keeps no per-call state, is safe to call from several host
 * threads, and never synchronises: work is enqueued on `stream` (a
 * cudaStream_t passed as void*; NULL is the legacy default stream) and the
 * call returns at once. The host never reads seq_lens.
 *
 * Aliasing. Outputs may alias an input exactly (y == x; dx == dy or
 * dx == y): each row is read before that row is written. Partial overlap of
 * an output with any input, or of seq_lens with an output, is rejected.
 *
 * Errors are returned, never raised, trapped or printed:
 *   GTMS_OK              work enqueued (or nothing to do: B*M*S == 0).
 *   GTMS_ERR_INVALID_ARG null pointer with B*M*S > 0, B/M/S < 0, a size whose
 *                        byte count overflows, a non-finite scale, a pointer
 *                        not aligned to its element size, partial overlap.
 *   GTMS_ERR_UNSUPPORTED unknown dtype; S > GTMS_MAX_S; or S > 8192 with a row
 *                        whose byte length is not a multiple of 16 or a buffer
 *                        that is not 16-byte aligned (long rows are streamed
 *                        in 16-byte units only).
 *   GTMS_ERR_CUDA        the kernel launch failed (the status the launch call
 *                        itself returned; an error left behind by earlier,
 *                        unrelated work on the thread is not reported here).
 *   GTMS_ERR_TIMEOUT     never returned by a call, which returns before its
 *                        kernel runs: it is the code that the attention step's
 *                        kernel writes into the caller's status word when one of
 *                        its bounded internal waits ran out (see
 *                        gtms_attention_softmax_backward).
 * All argument checks run on the host before anything is enqueued; a call
 * that returns an error has enqueued nothing.
 */
#ifndef GTMS_H
#define GTMS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GTMS_VERSION 1
#define GTMS_MAX_S 65536

typedef enum { GTMS_F32 = 0, GTMS_BF16 = 1, GTMS_F16 = 2 } gtms_dtype;

/*
 * Mask families ("优化ScaledMaskSoftmax算子", section 6, lists a local window
 * mask and a length mask next to the default). Each keeps a contiguous column
 * range of a row r < L = clamp(seq_lens[b], 0, S) and nothing of rows r >= L:
 *   GTMS_MASK_GROUPED_TRIL   c <= r                (the operator above)
 *   GTMS_MASK_LENGTH         c < L                 (padded keys and queries)
 *   GTMS_MASK_SLIDING_WINDOW r - window < c <= r   (causal band, window >= 1;
 *                            the section's garbled local-window snippet is read
 *                            as this band)
 */
typedef enum {
    GTMS_MASK_GROUPED_TRIL = 0,
    GTMS_MASK_LENGTH = 1,
    GTMS_MASK_SLIDING_WINDOW = 2
} gtms_mask_kind;

typedef enum {
    GTMS_OK = 0,
    GTMS_ERR_INVALID_ARG = 1,
    GTMS_ERR_UNSUPPORTED = 2,
    GTMS_ERR_CUDA = 3,
    GTMS_ERR_TIMEOUT = 4
} gtms_status;

/*
 * Forward: y = grouped-tril masked softmax(scale * x).
 *   x        device, [B, M, S, S] of `dtype`, read-only; only the kept prefix
 *            x[b, m, r, 0 : min(r + 1, L)] of rows r < L is loaded.
 *   y        device, [B, M, S, S] of `dtype`, every element written.
 *   seq_lens device, int32[B].
 *   scale    finite float, applied inside the exponent.
 *   dtype    gtms_dtype of x and y.
 *   stream   cudaStream_t or NULL.
 */
int gtms_forward(const void* x, void* y, const int32_t* seq_lens,
                 int64_t B, int64_t M, int64_t S, float scale, int dtype, void* stream);

/*
 * Backward: dx = scale * y * (dy - rowsum(dy * y)) under the same mask.
 *   y, dy    device, [B, M, S, S] of `dtype`, read-only (y is the forward
 *            output); only the kept prefix of each live row is loaded.
 *   dx       device, [B, M, S, S] of `dtype`, every element written.
 *   Other arguments as in gtms_forward.
 */
int gtms_backward(const void* y, const void* dy, void* dx, const int32_t* seq_lens,
                  int64_t B, int64_t M, int64_t S, float scale, int dtype, void* stream);

/*
 * gtms_forward computed by the staged kernel: the block-per-row design of
 * "优化ScaledMaskSoftmax算子" (sections 2.2 and 4.2: a thread block per row,
 * the row staged in shared memory), with each live row's kept units brought
 * into shared memory by one TMA bulk copy, several rows ahead of the row being
 * reduced. Same operation, arguments and errors as gtms_forward, and the same
 * output values within the parity tolerances. On GB300 it measured slower than
 * gtms_forward (S = 2048 bf16: 5.6 against 6.4 TB/s), which stays the fast
 * path; this entry point is kept for comparison and for other parts.
 * GTMS_ERR_UNSUPPORTED beyond gtms_forward's cases: rows whose byte length is
 * not a multiple of 16 or is 32 KB or more, buffers not 16-byte aligned.
 * A copy that does not arrive within 1 s of GPU time is given up on: the row is
 * then read straight from x (same result), never waited on forever.
 */
int gtms_forward_staged(const void* x, void* y, const int32_t* seq_lens,
                        int64_t B, int64_t M, int64_t S, float scale, int dtype, void* stream);

/*
 * Device address of a page-locked host buffer (allocated with cudaHostAlloc
 * or registered with cudaHostRegister), for passing host-resident tensors
 * straight to gtms_forward / gtms_backward: the kernels then read the kept
 * inputs from, and write every output to, host memory over the host link
 * (NVLink-C2C on Grace-Blackwell), with no staging copy.
 *   host     pointer into a page-locked host allocation.
 *   device   out: the address the current device uses for it.
 * Returns GTMS_ERR_INVALID_ARG for null arguments or for memory the CUDA
 * runtime cannot map for the current device, GTMS_ERR_CUDA for other runtime
 * errors. (Where the device reads pageable host memory through the host's page
 * tables, as on Grace-Blackwell, the runtime maps pageable memory as well;
 * page-locked memory is still what the transfer rate assumes.) Host-only,
 * enqueues nothing, allocates nothing.
 */
int gtms_device_pointer_of_host(const void* host, void** device);

/*
 * gtms_forward / gtms_backward with another mask family (gtms_mask_kind).
 * `window` is the band width of GTMS_MASK_SLIDING_WINDOW (>= 1; widths >= S
 * give the grouped-tril op) and is ignored by the other kinds. An unknown kind
 * is GTMS_ERR_UNSUPPORTED, a sliding window narrower than 1
 * GTMS_ERR_INVALID_ARG; everything else is as for gtms_forward / gtms_backward
 * (gtms_forward is gtms_forward_masked with GTMS_MASK_GROUPED_TRIL).
 */
int gtms_forward_masked(const void* x, void* y, const int32_t* seq_lens, int64_t B, int64_t M, int64_t S,
                        float scale, int mask_kind, int64_t window, int dtype, void* stream);
int gtms_backward_masked(const void* y, const void* dy, void* dx, const int32_t* seq_lens, int64_t B, int64_t M,
                         int64_t S, float scale, int mask_kind, int64_t window, int dtype, void* stream);

/*
 * Masked softmax with an explicit keep mask ("优化ScaledMaskSoftmax算子",
 * sections 2.2 and 3.1: input, mask, scale; section 4.1: a row with nothing
 * kept is zero). y[b, m, r, c] = softmax over {c' : mask[b', r, c'] != 0} of
 * scale * x[b, m, r, c'] at kept entries, +0.0 elsewhere; b' = 0 when
 * mask_batches == 1, else b. The backward is dx = scale * y * (dy - rowsum(dy * y))
 * over the same kept set.
 *   mask         device uint8 [mask_batches, S, S], 8-byte aligned, read-only,
 *                shared by the M heads; nonzero = keep.
 *   mask_batches 1 or B.
 * Masked inputs are not loaded: each 16-byte unit of x (or of y and dy) is
 * read only if its mask bytes keep at least one element.
 * GTMS_ERR_INVALID_ARG also covers a null or misaligned mask, mask_batches
 * other than 1 or B, and a mask overlapping the output. GTMS_ERR_UNSUPPORTED:
 * S > 8192, rows that are not 16-byte multiples, or buffers not 16-byte aligned.
 */
int gtms_forward_explicit(const void* x, void* y, const uint8_t* mask, int64_t mask_batches, int64_t B, int64_t M,
                          int64_t S, float scale, int dtype, void* stream);
int gtms_backward_explicit(const void* y, const void* dy, void* dx, const uint8_t* mask, int64_t mask_batches,
                           int64_t B, int64_t M, int64_t S, float scale, int dtype, void* stream);

/*
 * Attention-backward step around the masked softmax, fused with its GEMM on the
 * tensor cores ("ops(8): self-attention 的 CUDA 实现及优化 (下)", section 2.1: with
 * P the softmax output, O = P V and upstream gradient dO, the backward forms
 * dP = dO V^T and then the softmax backward of dP):
 *   dS[b,m,r,c] = scale * P[b,m,r,c] * (dP[r,c] - sum_c' dP[r,c'] P[b,m,r,c'])
 * on the grouped-tril kept entries (c <= r < L), +0.0 elsewhere, with
 * dP[r,c] = sum_k dO[b,m,r,k] V[b,m,c,k] accumulated in fp32 and never
 * written to memory.
 *   p        [B,M,S,S] of `dtype` (the forward output), read-only. Masked
 *            entries are never used (NaN there does not reach ds); tiles
 *            right of the diagonal and padded row blocks are not read.
 *   dout, v  [B,M,S,head_dim] of `dtype`, read-only.
 *   ds       [B,M,S,S] of `dtype`, every element written; may equal p.
 * The four tensors are device-addressable: when all four are device memory
 * the call runs a persistent TMA-fed kernel (one CTA per SM); otherwise
 * (mapped page-locked host memory, see gtms_device_pointer_of_host) a kernel
 * that copies with cp.async and reads P only in 16-byte units that hold a
 * kept entry.
 *   seq_lens device int32[B]; scale finite.
 *   head_dim 64 or 128; dtype GTMS_BF16 or GTMS_F16; S a multiple of 8.
 *   status   NULL, or a device-addressable int32 that the kernel ORs
 *            GTMS_ERR_TIMEOUT into when one of its internal waits (a hand-off
 *            between its warps, each bounded to 1 s of GPU time) ran out; the
 *            kernel then stops early and its results are incomplete. The
 *            caller clears the word before the call and reads it after
 *            synchronising with `stream`: 0, or GTMS_ERR_TIMEOUT.
 * All pointers 16-byte aligned (status 4-byte). GTMS_ERR_UNSUPPORTED: fp32,
 * other head dims, S not a multiple of 8, S > GTMS_MAX_S. Otherwise as
 * gtms_backward.
 */
int gtms_attention_softmax_backward(const void* p, const void* dout, const void* v, void* ds, const int32_t* seq_lens,
                                    int64_t B, int64_t M, int64_t S, int64_t head_dim, float scale, int dtype,
                                    int32_t* status, void* stream);

/*
 * A [B, H, S, head_dim] tensor of `dtype` whose element (b, h, s, j) stands at
 * data + b * stride_b + h * stride_h + s * stride_s + j (strides in elements):
 * the rows of a head are contiguous vectors, and the three outer dimensions may
 * be laid out in any order (a [B, S, H, head_dim] projection, or the q, k and v
 * parts of one fused projection, need no copy). Strides are not negative; the
 * stride of a dimension of extent 1 is ignored. An input may repeat itself
 * (stride 0 over an extent above 1: one head or batch broadcast); an output's
 * elements must be distinct.
 */
typedef struct {
    void* data;
    int64_t stride_b, stride_h, stride_s;
} gtms_heads;

/*
 * Sizes and options of the attention calls. Hq is a multiple of Hkv: query head
 * h reads key/value head h / (Hq / Hkv). The mask families are those of
 * gtms_forward_masked with row i of batch b at position
 * r = q_offsets[b] + i (r = i without q_offsets) and L = clamp(seq_lens[b], 0, Skv):
 * nothing is kept of rows with r < 0 or r >= L, otherwise
 *   GTMS_MASK_GROUPED_TRIL   c <= r,
 *   GTMS_MASK_LENGTH         c < L,
 *   GTMS_MASK_SLIDING_WINDOW r - window < c <= r.
 * Whole sequences take Sq == Skv and no offsets. New tokens over a cache take
 * the cache's capacity as Skv, the live length (new tokens included) as
 * seq_lens[b] and seq_lens[b] - Sq as q_offsets[b]; one new token is Sq == 1.
 */
typedef struct {
    int64_t B, Hq, Hkv, Sq, Skv, head_dim;
    int64_t window;
    int32_t mask_kind, dtype;
    float scale;
} gtms_attention_shape;

#define GTMS_ATTENTION_MAX_S (1 << 24)

/*
 * Attention: with s_ic = scale * q_i . k_c over the kept entries c of row i,
 *   o_i = sum_c softmax(s_i)_c v_c,   lse_i = log sum_c exp(s_ic)
 * in one pass, the scores and probabilities staying on the chip. Rows that keep
 * nothing get o = +0.0 and lse = -inf.
 *   q        [B, Hq, Sq, head_dim], k, v [B, Hkv, Skv, head_dim], read-only.
 *   o        [B, Hq, Sq, head_dim], every element written.
 *   lse      fp32 [B, Hq, Sq], contiguous, or NULL.
 *   seq_lens device int32[B]; q_offsets device int32[B] or NULL.
 *   status   as in gtms_attention_softmax_backward; the limit of 1 s is that of the
 *            hand-offs of one tile, and however long the rows are, a call that
 *            makes progress is not given up.
 * k and v at c >= L and q at r >= L are never used: anything may stand there,
 * NaN too. Inside the live length a NaN or infinity in k stays in the rows that
 * keep it; one in v can also reach rows that mask it, those within 127 rows of one
 * that keeps a key of the same 128-key tile (a masked probability is an exact zero,
 * but the tile's product multiplies it).
 * Sums, maxima and accumulators are fp32; probabilities are rounded once to
 * `dtype` for the product with v, and o once on its way out. The accumulators of
 * the tensor cores cut off instead of rounding: a sum is short by up to 2e-4 of its
 * terms' size in fp16 and 9e-4 in bf16 (half a step of which is 5e-4 and 4e-3), and
 * no more however long it is: longer ones are formed in parts, between which o
 * (the backward: dq, dk, dv) holds what 16 bits take of the sum so far.
 * dtype GTMS_BF16 or GTMS_F16, head_dim 64 or 128. Data 16-byte aligned,
 * strides multiples of 8 elements, below 2^40 bytes and not below head_dim, save
 * for the strides of 0 of a broadcast batch or head. o must not overlap the inputs;
 * one that lies between another operand's elements is told apart from it where both
 * repeat with one common period (the parts of one fused projection).
 * GTMS_ERR_INVALID_ARG: null arguments, negative sizes or strides, Hq not a
 * multiple of Hkv, a non-finite scale, a window below 1 with the sliding window,
 * overlaps, an output that repeats itself, misaligned lse, seq_lens, q_offsets
 * (4 bytes). GTMS_ERR_UNSUPPORTED: other dtypes and head dims, Sq or Skv above
 * GTMS_ATTENTION_MAX_S, an unknown mask kind, data or strides not aligned as
 * above, more work than a grid holds. Nothing to do (no rows of o) is GTMS_OK.
 */
int gtms_attention_forward(const gtms_attention_shape* shape, const gtms_heads* q, const gtms_heads* k,
                           const gtms_heads* v, const gtms_heads* o, float* lse, const int32_t* seq_lens,
                           const int32_t* q_offsets, int32_t* status, void* stream);

/*
 * The gradients of gtms_attention_forward, from its inputs and results; the
 * probabilities are recomputed as p_ic = exp(s_ic - lse_i):
 *   D_i  = do_i . o_i            ds_ic = p_ic (do_i . v_c - D_i)
 *   dq_i = scale sum_c ds_ic k_c dk_c = scale sum_i ds_ic q_i   dv_c = sum_i p_ic do_i
 * with dk and dv summed over the query heads that share the key/value head.
 *   o, lse, dout      the forward's results and the gradient of o.
 *   dq, dk, dv        every element written; +0.0 where nothing is kept.
 *   workspace         device memory of at least the bytes that
 *                     gtms_attention_backward_workspace gives, 16-byte aligned;
 *                     its contents need not be set, and calls that may run at
 *                     the same time need one each.
 * The sums run in a fixed order (no atomics on the gradients): the same inputs
 * give the same bits. p and ds are rounded once to `dtype` for their products.
 * q, o, lse and dout of rows that keep nothing, and k and v at c >= L, are never
 * used; a NaN or infinity in a live row or key can reach the gradients of the rows
 * and keys that share a 128 x 128 tile with it. The three gradients must not overlap
 * each other or any input. Otherwise as gtms_attention_forward.
 */
int gtms_attention_backward(const gtms_attention_shape* shape, const gtms_heads* q, const gtms_heads* k,
                            const gtms_heads* v, const gtms_heads* o, const float* lse, const gtms_heads* dout,
                            const gtms_heads* dq, const gtms_heads* dk, const gtms_heads* dv,
                            const int32_t* seq_lens, const int32_t* q_offsets, void* workspace,
                            uint64_t workspace_bytes, int32_t* status, void* stream);

/* Bytes of workspace that gtms_attention_backward needs for this shape. Host-only, enqueues nothing. */
int gtms_attention_backward_workspace(const gtms_attention_shape* shape, uint64_t* bytes);

/*
 * Rotary positions: pair j of the first rot_dim elements of each head is turned
 * by the angle a = positions[b][s] * inv_freq[j],
 *   y1 = amplitude (x1 cos a - x2 sin a),  y2 = amplitude (x2 cos a + x1 sin a),
 * and the elements from rot_dim on are copied. The pair is (j, j + rot_dim / 2),
 * or (2j, 2j + 1) when `interleaved` is not 0. With `inverse` not 0 the angle is
 * -a: the gradient of the forward call.
 *   x, y      [B, H, S, head_dim]; y may be x itself (same data and strides).
 *   x2, y2    a second tensor of H2 heads turned by the same call (q and k), or
 *             both NULL.
 *   positions device int32 [position_batches, S], position_batches 1 or B.
 *   inv_freq  device fp32 [rot_dim / 2].
 * The angle is formed and reduced in extended precision, so positions far from
 * zero keep full fp32 accuracy. Arithmetic is fp32 for every dtype (GTMS_F32,
 * GTMS_BF16, GTMS_F16); outputs are rounded once.
 * head_dim up to 1024, rot_dim even, 0 <= rot_dim <= head_dim. Data and strides
 * need only be element-aligned; 16-byte aligned ones take the wide kernel.
 * GTMS_ERR_INVALID_ARG: null arguments, negative sizes or strides, an odd or too
 * large rot_dim, a non-finite amplitude, misaligned pointers, an output that
 * repeats itself or overlaps an input other than as its exact alias.
 * GTMS_ERR_UNSUPPORTED: an unknown dtype, head_dim above 1024, S or H + H2 above
 * GTMS_ATTENTION_MAX_S, more tokens (B * S) than a grid holds.
 */
int gtms_rotary(const gtms_heads* x, const gtms_heads* y, const gtms_heads* x2, const gtms_heads* y2, int64_t B,
                int64_t H, int64_t H2, int64_t S, int64_t head_dim, int64_t rot_dim, const int32_t* positions,
                int64_t position_batches, const float* inv_freq, int interleaved, float amplitude, int inverse,
                int dtype, void* stream);

/*
 * Inverse frequencies of gtms_rotary, into `inv_freq` (host memory, rot_dim / 2
 * floats): f_j = base^(-2j / rot_dim), then for long contexts
 *   GTMS_ROTARY_PLAIN    f_j
 *   GTMS_ROTARY_LINEAR   f_j / factor
 *   GTMS_ROTARY_BY_PARTS (1 - m) f_j / factor + m f_j with
 *                        m = clamp((turns_j - low_turns) / (high_turns - low_turns), 0, 1),
 *                        turns_j = original_length f_j / (2 pi): pairs that turn more than
 *                        high_turns times over the original length keep their frequency,
 *                        those below low_turns are stretched.
 * Computed in double and rounded once. GTMS_ERR_INVALID_ARG: a null pointer, an
 * odd or negative rot_dim, base or factor not above 0 or not finite, and by parts
 * high_turns <= low_turns or original_length < 1; GTMS_ERR_UNSUPPORTED: an
 * unknown kind. Host-only, enqueues nothing.
 */
typedef enum { GTMS_ROTARY_PLAIN = 0, GTMS_ROTARY_LINEAR = 1, GTMS_ROTARY_BY_PARTS = 2 } gtms_rotary_scaling;
int gtms_rotary_frequencies(int64_t rot_dim, double base, int scaling, double factor, double low_turns,
                            double high_turns, int64_t original_length, float* inv_freq);

/* Static, NUL-terminated name of a status code ("GTMS_OK", ...). */
const char* gtms_status_string(int status);

/* GTMS_VERSION of the built library. */
int gtms_version(void);

/*
 * Name of the kernel variant that gtms_forward (direction 0), gtms_backward
 * (direction 1) or gtms_forward_staged (direction 2) launches for this row
 * length, dtype and alignment (aligned16 != 0: every pointer is 16-byte
 * aligned). Static string; "none" for unsupported arguments. Host-only,
 * enqueues nothing.
 */
const char* gtms_kernel_name(int direction, int64_t S, int dtype, int aligned16);

/*
 * Name of the kernel variant that gtms_forward_masked (direction 0) or
 * gtms_backward_masked (direction 1) launches for this row length, dtype,
 * alignment, mask kind and window. Mask kinds 1 and 2 append ",maskK" to the
 * per-row kernel's name; a narrow sliding window may take a band kernel
 * instead. Static string; "none" for unsupported arguments. Host-only,
 * enqueues nothing.
 */
const char* gtms_kernel_name_masked(int direction, int64_t S, int dtype, int aligned16, int mask_kind,
                                    int64_t window);

/*
 * Name of the kernel variant that gtms_forward_explicit (direction 0) or
 * gtms_backward_explicit (direction 1) launches for this row length and dtype
 * (16-byte-aligned buffers). Static string; "none" for arguments those calls
 * reject. Host-only, enqueues nothing.
 */
const char* gtms_kernel_name_explicit(int direction, int64_t S, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* GTMS_H */
