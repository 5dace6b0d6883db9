/*
 * vit_ops.h -- operator entry points of libvit_b200 beside the stages of vit_stages.h: what a text
 * tower, a decoder over patch tokens or a packed batch of images needs next to the encoder.
 * Attention over packed sequences (grouped heads, causal or full, whole prompts and single tokens
 * over a cache), rotary positions, the root-mean-square norm with the residual's addition, and
 * linear layers on 8-bit rows.  Forward only: no operator has a backward pass (vit_op_rope's inverse is its own).
 *
 * Conventions as in vit.h: caller-owned device memory of the current device, work enqueued on
 * `stream` without synchronising, host validation before any launch.  Nothing is allocated and
 * nothing is kept from one call for the next, so calls may run side by side on any streams (with
 * a workspace each where one is taken) and be captured into CUDA graphs.  Where a call has no work
 * (no rows, no tokens) it returns VIT_OK and enqueues nothing.
 *   - Strides are in elements; the last dimension is contiguous.
 *   - `status`: device int32, zero at the start, that a kernel sets when one of its pipeline waits
 *     gives up (what that call was to write is then undefined) and that later kernels on the same word check on
 *     entry: they return without work while it is set.  NULL selects a word of the library per device,
 *     which all such calls share: it stops nobody, vit_op_poll reads and clears it, and a caller who has to know
 *     about its own calls beside others' gives a word of its own.  `wait_ns`: limit of the waits in
 *     nanoseconds, 0 for the default 2 s.
 */
#ifndef VIT_B200_OPS_H
#define VIT_B200_OPS_H

#include "vit.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum vit_dtype {
  VIT_DT_BF16 = 0,
  VIT_DT_F16 = 1,
  VIT_DT_F32 = 2,
  VIT_DT_E4M3 = 3 /* 8-bit floating point, 4 exponent and 3 mantissa bits, largest value 448 */
} vit_dtype;

/* Root-mean-square norm of rows, with the residual's addition:
 *   h = x + r          (r = NULL: h = x);   residual_out = h, rounded to r's type
 *   y = h * weight / sqrt(mean(h^2) + eps)
 *   out_type = x_type: out = y.
 *   out_type = E4M3:   scales[i] = max(max_j |y_ij|, 2^-100) / 448, out_ij = e4m3(y_ij / scales[i]).
 * Sums and products in fp32, on h before its rounding.  A NaN or an infinity in a row makes its
 * outputs what the formulas make of it; other rows are not touched by it.
 *   x: [rows, D], leading dimension x_ld, bf16 / fp16 / fp32.
 *   residual, residual_out: both or neither; same shape, x's type or fp32; may be the same memory.
 *   weight: [D], x's type or fp32.       out: [rows, D].      scales: fp32 [rows], E4M3 only.
 * out may be x, residual_out residual, with the same bytes from row to row (E4M3 on a 16-bit x: out_ld = 2 x_ld);
 * otherwise nothing that is written overlaps what the call reads or writes.
 * 1 <= D <= 32768; pointers aligned to their element type.  Rows on 16-byte aligned pointers (an 8-bit out: 8)
 * take 16-byte accesses if their leading dimensions are the same modulo 8, fastest where those and D are
 * multiples of 8. */
vit_status vit_op_rms_norm(const void *x, vit_dtype x_type, int64_t x_ld, const void *residual, int64_t residual_ld,
                           void *residual_out, int64_t residual_out_ld, vit_dtype residual_type, const void *weight,
                           vit_dtype weight_type, float eps, int64_t rows, int32_t D, void *out, vit_dtype out_type,
                           int64_t out_ld, float *scales, vit_stream_t stream);

/* Rows in 8 bits: scales[i] = max(max_j |x_ij|, 2^-100) / 448, out_ij = e4m3(x_ij / scales[i]); the
 * weights and activations of vit_op_linear_fp8.  Arguments as in vit_op_rms_norm. */
vit_status vit_op_quant_rows(const void *x, vit_dtype x_type, int64_t x_ld, int64_t rows, int32_t D, void *out,
                             int64_t out_ld, float *scales, vit_stream_t stream);

/* Linear layer on 8-bit rows:
 *   out[m, n] = bf16(a_scales[m] * w_scales[n] * sum_k A[m, k] W[n, k] + bias[n])
 *   A: e4m3 [M, K], W: e4m3 [N, K] (nn.Linear layout), K contiguous, leading dimensions lda, ldw
 *   (multiples of 16); a_scales fp32 [M], w_scales fp32 [N], bias fp32 [N] or NULL; out bf16
 *   [M, N], leading dimension ldo (a multiple of 8).  K a multiple of 16, N a multiple of 8,
 *   pointers 16-byte aligned (a_scales: 4).  Products are accumulated in fp32. */
vit_status vit_op_linear_fp8(const void *A, int64_t lda, const float *a_scales, const void *W, int64_t ldw,
                             const float *w_scales, const float *bias, int32_t M, int32_t N, int32_t K, void *out,
                             int64_t ldo, int32_t *status, uint64_t wait_ns, vit_stream_t stream);

/* Which values of a head make a pair: i and i + rotary_dim / 2, or 2 i and 2 i + 1. */
enum { VIT_ROPE_HALF = 0, VIT_ROPE_INTERLEAVED = 1 };

/* How vit_op_rope_freqs stretches the frequencies for contexts longer than `original_len`:
 * not at all; all divided by `factor`; a larger base, base * factor^(p / (p - 1)) for p pairs; or
 * by parts: those that turn more than beta_fast times over original_len stay, those that turn
 * less than beta_slow times are divided by `factor`, a linear blend in between. */
enum { VIT_ROPE_PLAIN = 0, VIT_ROPE_LINEAR = 1, VIT_ROPE_BASE = 2, VIT_ROPE_PARTS = 3 };

/* Host helper: freqs[i] = base^(-i / p), i < p = pairs / axes, stretched as `scaling` says, repeated
 * for each of `axes` position axes: pairs doubles, in radians per position. */
vit_status vit_op_rope_freqs(double base, int32_t pairs, int32_t axes, int32_t scaling, double factor,
                             double original_len, double beta_fast, double beta_slow, double *freqs);

/* One tensor of heads [T, heads, head_dim] in and out (strides in elements; 0 to read the same head or token
 * again, while the heads of an output do not overlap); in == NULL: none. */
typedef struct vit_rope_tensor {
  const void *in;
  void *out; /* may be `in`, with its strides; otherwise overlaps nothing that the call reads or writes */
  int64_t in_token, in_head, out_token, out_head;
  int32_t heads;
} vit_rope_tensor;

/* Rotary positions on queries and keys: pair i of token t is turned by pos[a][t] * freqs[i] with
 * axis a = i / (pairs / axes); the values past rotary_dim are copied.
 *   (x, y) -> gain * (x cos - y sin, x sin + y cos);  inverse != 0: by minus the angle (which is
 *   also the gradient's rotation).
 *   positions: device [axes, T], int32, or int64 if pos64.  Whole turns drop out exactly; for freqs up to 1 the
 *   angle is off by at most 2^-33 + |position| 2^-64 turns (and the sine's fp32): 1.5e-9 rad up to 2^31.
 *   freqs: HOST array of rotary_dim / 2 doubles, radians per position, read during the call.
 *   rotary_dim: even, 2..256, <= head_dim, rotary_dim / 2 a multiple of axes; axes 1..4. */
vit_status vit_op_rope(const vit_rope_tensor *q, const vit_rope_tensor *k, vit_dtype type, int64_t T, int32_t head_dim,
                       int32_t rotary_dim, const void *positions, int32_t pos64, int32_t axes, const double *freqs,
                       int32_t layout, float gain, int32_t inverse, vit_stream_t stream);

/* Attention over packed sequences.  Sequence i has the query rows cu_q[i] .. cu_q[i+1] - 1 and the key
 * rows cu_k[i] .. cu_k[i+1] - 1, of which the first len_k[i] count (len_k = NULL: all); with a
 * cache of room per sequence, cu_k holds where each sequence's room begins.  Query head h reads
 * key head h / (heads_q / heads_k).  Query t of lq sees keys 0 .. lk - 1, or with `causal` keys
 * 0 .. t + lk - lq.
 *   out = sum_j softmax_j(scale * q . k_j) v_j; zero for a row that sees no key.
 * Rows of `out` outside every sequence are left as they are; whatever the key rows of no sequence
 * or past len_k hold (NaN included) does not matter.  V must be finite in a sequence's own rows.
 *   q [Tq, heads_q, head_dim], k, v [Tk, heads_k, head_dim], out as q: `type` bf16 or fp16, head_dim
 *   64 or 128, strides multiples of 8 (0 to read the same head or token again), pointers 16-byte aligned.
 *   The heads of `out` overlap neither one another nor what the call reads.
 *   cu_q, cu_k: device int32 [n + 1], not decreasing; len_k: device int32 [n].  Read on the device
 *   (a captured call takes new lengths on replay); values outside the buffers are clamped.
 *   max_q: the longest query length if the caller knows it, 0 if not.  The choice between three kernels
 *   goes by it, with n, Tk / n (the key rows a sequence has on average) and the heads: few query rows over long
 *   key rows, as single tokens over a cache, run on one that splits the keys' axis over the GPU (one
 *   token over 100003 keys, 32 heads on 8 of 128: 77 us; 1000 us with max_q = 0, since then tiles of 128 rows are
 *   taken, each of which walks its keys alone), short sequences on one without shared memory.  Any value
 *   is right; it decides the time, and within the precision below the last bits of the result.
 *   workspace: vit_op_attention_packed_workspace bytes of device memory, 16-byte aligned, that no
 *   other call uses before this one has run; needs no preparation.
 * Scores, softmax statistics and sums are fp32.  The kernel of tiles rounds the softmax's weights to
 * `type` for the product with V, the two others to twice its precision; the result is rounded once.  Bits are the
 * same from call to call, but not between the kernels, so that a sequence's result can differ in its last bits
 * with the batch it is in. */
typedef struct vit_attn_packed {
  const void *q, *k, *v;
  void *out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
  const int32_t *cu_q, *cu_k, *len_k;
  int64_t Tq, Tk;
  int32_t n, heads_q, heads_k, head_dim, type, causal, max_q;
  float scale;
  int32_t *status;
  uint64_t wait_ns;
  void *workspace;
  size_t workspace_bytes;
} vit_attn_packed;

/* Workspace of a call with these arguments on the current device: 0 where none is used, at most 10 MB.  Reads n,
 * Tq, Tk, max_q, heads_q, heads_k, head_dim and type, no pointer. */
vit_status vit_op_attention_packed_workspace(const vit_attn_packed *a, size_t *bytes);

vit_status vit_op_attention_packed(const vit_attn_packed *a, vit_stream_t stream);

/* Synchronise `stream`, then read and clear the current device's library status word (the one that
 * calls with status = NULL use): VIT_OK, VIT_E_DEVICE_TIMEOUT or VIT_E_CUDA. */
vit_status vit_op_poll(vit_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* VIT_B200_OPS_H */
