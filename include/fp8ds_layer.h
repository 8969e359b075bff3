/*
 * fp8ds_layer.h -- C ABI of the operators around the FP8 linear: the norm that
 * feeds it, the product with an activation in its epilogue, and the gradients
 * of both.
 *
 * Conventions as fp8ds.h: caller-owned device memory, asynchronous on the
 * caller's stream and the current device, negative fp8_status on an error,
 * every argument checked on the host before anything is launched.  A ring's
 * words and an amax count as outputs where overlaps are refused.
 */
#ifndef FP8DS_LAYER_H_
#define FP8DS_LAYER_H_

#include "fp8ds.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8_rmsnorm -- root-mean-square norm with the residual's addition and an
 * FP8 output.  Per row of cols values, sums in float32:
 *   h = x + residual, rounded once to x's type (h = x without a residual);
 *       everything below reads the rounded h, the value the stream keeps
 *   r = 1 / sqrt(mean(h^2) + eps)
 *   v = (h * r) * gamma                     (float32)
 * and, of these outputs, those that are wanted:
 *   h      the residual stream, x's type (required with a residual)
 *   rstd   r, float32 [rows], what the backward needs
 *   y      v rounded to x's type
 *   codes  FP8 codes [rows, cols]:
 *          row_sinv NULL: saturate_rne(fp32(v * s)) with s = *ring.scale read
 *          at launch; ring folds amax = max |v| (NaN ignored) exactly as
 *          fp8_quantize folds its input's, in the same launch.  With amax_out
 *          set the ring's history, idx and scale are left alone: the launch
 *          writes amax there and 1/s to ring.scale_inv (as
 *          fp8_quantize_local; fp8_ring_fold folds later).
 *          row_sinv set: every row has its own current scale, FP8_MAX / max |v|
 *          of the row (1 when that is 0 or not finite); row_sinv[r] = 1/scale
 *          is what fp8_mm_act takes as a row-wise sinv_a.  ring is unused.
 *          Rows on their own scales suit serving: a call keeps no state.
 *          With a ring the codes' factor is *ring.scale_inv until the next call
 *          on that ring writes it: where codes are kept across such a call (a
 *          second forward before the backward), keep a copy of it with them.
 *
 * x, residual, h, y  [rows, cols] row-major, contiguous, element type dtype
 *         (fp8_in_dtype), any address aligned to the element.  h or y may be
 *         x or residual itself (in place).  Otherwise no output may overlap
 *         another argument.
 * gamma   [cols], of x's type or float32 (gamma_f32 != 0).
 * rows >= 0 (0 still folds amax 0 into a ring), 1 <= cols <= 16384, eps > 0.
 * Errors: FP8_ERR_INVALID_ARG (bad enum, negative size, cols 0, eps not
 *         positive and finite, NULL x or gamma, a residual without h, h
 *         without a residual, no output at all, codes without a complete ring
 *         or row_sinv, ring arguments without codes, a ring with row_sinv,
 *         an output that overlaps another argument);
 *         FP8_ERR_UNSUPPORTED (cols above 16384, rows of 2^31 or more, an address
 *         not aligned to its element, ring.scratch not 8-byte aligned).
 */
typedef struct {
  const void* x;
  const void* residual; /* NULL: h = x */
  int dtype;
  int64_t rows, cols;
  const void* gamma;
  int gamma_f32;
  float eps;
  void* h;
  void* y;
  float* rstd;
  uint8_t* codes;
  int fmt;
  fp8_ring ring;
  float* amax_out;
  float* row_sinv;
} fp8_rmsnorm_args;
int fp8_rmsnorm(const fp8_rmsnorm_args* args, fp8_stream_t stream);

/*
 * fp8_rmsnorm_backward -- the gradient of fp8_rmsnorm, with the codes' cast
 * taken as the identity.  With n = h * rstd and g = dy * gamma (float32):
 *   dx     = dres + rstd * (g - n * mean(g * n)), rounded once to h's type:
 *            the gradient of x and, the same values, of residual.  dres is the
 *            gradient that reaches h past the norm (NULL: none).
 *   dgamma = sum over rows of dy * n, float32 [cols] (NULL: not wanted).  The
 *            order of the sums depends on rows, cols, dtype and the device only, so
 *            repeated calls give the same bits, whatever the addresses.
 * dy, h, dres, dx  [rows, cols], contiguous, element type dtype; dx may be dy
 *         or dres itself.
 * workspace  at least fp8_rmsnorm_backward_workspace_bytes(rows, cols) bytes,
 *         4-byte aligned, no initial value; unused (may be NULL) without
 *         dgamma.  Calls that may overlap on the GPU need one each.
 * Errors as fp8_rmsnorm; FP8_ERR_INVALID_ARG also for a workspace that is
 *         missing or too small.  rows == 0 sets dgamma to 0.
 */
typedef struct {
  const void* dy;
  const void* h;
  const void* dres;
  int dtype;
  int64_t rows, cols;
  const float* rstd;
  const void* gamma;
  int gamma_f32;
  void* dx;
  float* dgamma;
  void* workspace;
  size_t workspace_bytes;
} fp8_rmsnorm_backward_args;
int fp8_rmsnorm_backward(const fp8_rmsnorm_backward_args* args, fp8_stream_t stream);
size_t fp8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols);

/* Activations of fp8_mm_act and fp8_act_backward: value and slope at z.
 *   RELU  max(z, 0), slope 0 for z <= 0, else 1; where it is 0, dz is 0
 *         whatever dy and u are
 *   GELU  the tanh form: z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2
 *   SILU  z / (1 + e^-z) */
typedef enum { FP8_ACT_NONE = 0, FP8_ACT_RELU = 1, FP8_ACT_GELU = 2, FP8_ACT_SILU = 3 } fp8_act;

/* What fp8_mm_act does with its bf16 operand: y = act(z) + aux, or act(z) * aux. */
typedef enum { FP8_AUX_ADD = 0, FP8_AUX_MUL = 1 } fp8_aux_op;

/*
 * fp8_mm_act -- the scaled FP8 product with an activation, and a residual or a
 * gate, in its epilogue.  In float32, for m in [0, M), n in [0, N):
 *   z[m,n] = fp32_acc(sum_k A[m,k] B[n,k]) * (sinv_a * sinv_b) + bias[n]
 *            (one fused multiply-add, as fp8_mm)
 *   t = act(z);  y = t, t + aux[m,n] or t * aux[m,n]
 * and rounded once from there:
 *   z      bf16 [M, N], or NULL: the pre-activation for fp8_act_backward
 *   out    out_kind FP8_MM_OUT_BF16: bf16 [M, N]; FP8_MM_OUT_E4M3 / _E5M2: FP8
 *          codes of fp32(y * s), s = *out_ring.scale read at launch, with
 *          max |y| folded into out_ring (or written to out_amax) as fp8_mm_ex.
 *
 * A, B    FP8 codes [M, K] and [N, K], K contiguous; layout: FP8_MM_A_E5M2 and
 *         FP8_MM_B_E5M2 only.
 * sinv_a  one float, or (sinv_a_rows != 0) M floats: a factor per row of A, as
 *         fp8_rmsnorm's row_sinv gives them.
 * bias    float32 [N] or NULL.  aux: bf16 [M, N] or NULL.  All contiguous.
 *         out may be aux itself (a residual stream updated in place); sinv_a or
 *         sinv_b may be a word of out_ring, as it was before the call.
 * M, N >= 0, K >= 0 with K % 16 == 0; K == 0 gives z = bias; an empty output
 * still folds amax 0.  A few rows of A (8, or up to 32 with short K) take a
 * kernel that reads B once, straight into registers; a few hundred
 * rows, whose tiles leave SMs idle, share each tile's K among the CTAs of a
 * cluster.  Their sums run in other orders than the whole-tile kernel's, within
 * the same bound; the order depends on the sizes and the device only.  From the
 * sum on all of them compute the same bits.
 * Errors as fp8_mm_ex; FP8_ERR_INVALID_ARG also for an unknown act or aux_op,
 *         other layout bits, an output that overlaps another argument;
 *         FP8_ERR_UNSUPPORTED for an address not aligned to its element.
 */
typedef struct {
  const uint8_t* A;
  const uint8_t* B;
  int64_t M, N, K;
  int layout;
  const float* sinv_a;
  int sinv_a_rows;
  const float* sinv_b;
  const float* bias;
  int act;
  const uint16_t* aux;
  int aux_op;
  uint16_t* z;
  int out_kind;
  void* out;
  fp8_ring out_ring;
  float* out_amax;
} fp8_mm_act_args;
int fp8_mm_act(const fp8_mm_act_args* args, fp8_stream_t stream);

/*
 * fp8_act_backward -- the gradient of fp8_mm_act's epilogue, cast to FP8 for
 * the backward products.  In float32, per element of [rows, cols]:
 *   without u:  dz = dy * act'(z)
 *   with u:     dz = dy * u * act'(z),  du = dy * act(z)
 *               (y = act(z) * u, the gated form)
 *   dzq    FP8 codes of dz on ring's delayed scale; ring folds max |dz| in the
 *          same launch, exactly as fp8_quantize folds its input's.  What
 *          fp8_mm's backward products take as the output gradient.
 *   duq    the same of du with ring_u (required with u).
 *   db     column sums of dz, float32 [cols], or NULL: the bias gradient.
 *   dbu    column sums of du, or NULL (needs u and db).
 * amax_out / amax_out_u set: that ring is left to fp8_ring_fold, as in
 * fp8_quantize_local.  The gradient of an added residual is dy itself.
 *
 * dy      [rows, cols] contiguous, element type dtype (fp8_in_dtype).
 * z, u    [rows, cols] contiguous bf16: the pre-activation that fp8_mm_act
 *         saved, and the operand it multiplied by.  With FP8_ACT_NONE and no
 *         u, z may be NULL: a cast of dy that also gives the bias gradient.
 * The sums' order depends on rows, cols and the device only: repeated calls
 * give the same bits, whatever the addresses.  workspace: at least
 * fp8_act_backward_workspace_bytes(rows, cols, gated) bytes, 4-byte aligned,
 * no initial value; unused without db.  Calls that may overlap need one each.
 * rows, cols >= 0; an empty call still folds amax 0, and sets db to 0.
 * Errors: FP8_ERR_INVALID_ARG (bad enum, negative size, a missing or
 *         superfluous pointer, rings that share a word, one amax for both outputs, a
 *         workspace that is missing or too small, an output that overlaps another argument);
 *         FP8_ERR_UNSUPPORTED (an address not aligned to its element, a ring's
 *         scratch not 8-byte aligned, cols above 2^30, rows of 2^31 or more).
 */
typedef struct {
  const void* dy;
  int dtype;
  const void* z;
  const void* u;
  int64_t rows, cols;
  int act;
  int fmt;
  fp8_ring ring, ring_u;
  float* amax_out;
  float* amax_out_u;
  uint8_t* dzq;
  uint8_t* duq;
  float* db;
  float* dbu;
  void* workspace;
  size_t workspace_bytes;
} fp8_act_backward_args;
int fp8_act_backward(const fp8_act_backward_args* args, fp8_stream_t stream);
size_t fp8_act_backward_workspace_bytes(int64_t rows, int64_t cols, int gated);

#ifdef __cplusplus
}
#endif

#endif /* FP8DS_LAYER_H_ */
