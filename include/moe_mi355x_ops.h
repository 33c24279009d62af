/*
 * moe_mi355x_ops.h - operators around the expert layer, forward and backward
 * (libmoe_mi355x.so): the RMS norm in front of the router, token rows laid out
 * by expert and brought back, the experts' matrix products over such rows, rows and
 * weights in 4 bits, and the clipping of all gradients by their norm.
 *
 * One expert block at prefill or training width runs as
 *   moe_add_rms_norm -> moe_router_topk -> moe_align -> moe_permute ->
 *   moe_grouped_linear (gate+up, SwiGLU) -> moe_grouped_linear (down) ->
 *   moe_unpermute,
 * either in bf16 or with 8-bit rows and weights all along (the norm, the
 * permutation and the first product hand on e4m3fn rows with their scales).  The
 * router reads bf16 rows: a block in 8 bits calls the norm twice on the same x and
 * residual, for bf16 rows and for 8-bit ones (both are roundings of the same y), and
 * the second call may update the stream in place.
 * In 4 bits it runs as moe_add_rms_norm -> router, align -> moe_mxfp4_quantize (whose rows
 * go to their sorted places) -> moe_grouped_linear_mxfp4 twice (the first one hands on MXFP4
 * rows) -> moe_unpermute; with bf16 rows the same weights train, their gradient being
 * that of the values they stand for.
 * The backward entry points run the same chain the other way, but for the
 * router, which has none: moe_unpermute_backward gives the gradient of its
 * weights, the caller takes that through the softmax over the chosen logits
 * (dl = w (dw - sum over k of w dw)), and the dense products' gradients do the
 * rest, whose dx is added to the experts'.
 *
 * The conventions of moe_mi355x.h hold: device memory owned by the caller,
 * nothing allocated, no synchronisation, no device data read on the host, every
 * call capturable in a HIP graph (kernels only), work enqueued on `stream`, host
 * checks first (a refused call launches nothing and leaves a message for
 * moe_last_error()), no atomics: results are bit-identical run to run.  On top:
 *   - Every buffer a call writes must not overlap another buffer of the call
 *     unless its description says so.
 *   - Matrices are row-major.  Two calls that share a workspace must not overlap
 *     in time.
 *   - 8-bit rows are OCP e4m3fn codes [rows, C] with one float32 scale per 128
 *     columns, [rows, C/128]; a value is code * scale.  The scale of a block is
 *     its absolute maximum over 448, at least 2^-126, and 1 for a block of
 *     zeros, and a code is the nearest (ties to even) to the float32 value over the
 *     scale, both quotients rounded to float32 (where the exact quotient lies on the
 *     border of two codes, the rounding of the float32 value decides); a block with a
 *     NaN or an infinity gets a NaN scale, so all of it reads as NaN.
 *   - MXFP4 rows are E2M1 codes [rows, C/2], two per byte, the even column in the
 *     lower nibble, with one E8M0 byte per 32 columns, [rows, C/32], as the MXFP4
 *     weights of moe_mi355x.h are; a value is code * 2^(byte - 127).  The byte of a
 *     block made here is the exponent of its absolute maximum less 2, so that the
 *     maximum over the scale lies in [4, 8), at least 2, and 127 for a block of zeros;
 *     a code is the nearest (ties to even) to the value over the scale, at most 6.  A
 *     block with a NaN or an infinity gets the byte 255, E8M0's NaN, and zero codes.
 *   - Sorted rows: expert e's rows are [expert_offsets[e], expert_offsets[e] +
 *     expert_counts[e]) of a [rows, C] matrix, as moe_align lays them out (the
 *     offsets padded to its block size).  Rows outside every expert's run
 *     (padding, and those behind the last run) are neither read into a result
 *     nor written.  `rows` is the matrix's allocated height; an expert's run is
 *     cut off there.
 */
#ifndef MOE_MI355X_OPS_H
#define MOE_MI355X_OPS_H

#include "moe_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of this header's declarations (increases when one changes;
 * moe_abi_version() is that of moe_mi355x.h). */
int32_t moe_ops_abi_version(void);

typedef enum { MOE_DT_BF16 = 0, MOE_DT_F32 = 1, MOE_DT_E4M3 = 2, MOE_DT_MXFP4 = 3 } moe_dtype;

/* ------------------------------------------------------------------ norm -- */

/* Largest row length of the norm. */
#define MOE_NORM_MAX_H 32768

/* For each of M rows of H columns:
 *   z   = x + residual, rounded to the residual's type (z = x without one)
 *   y   = z * (mean(z^2) + eps)^(-1/2) * weight
 * x is bf16 with `ldx` elements from row to row (ldx >= H), weight bf16 [H];
 * residual (NULL: none) is bf16 or float32 (`rdt`) [M, H], contiguous.  z is
 * written to residual_out [M, H] (same type; NULL: not written; may be residual
 * itself, to update the stream in place), so that the row stored is the row
 * that was normalised.  y goes to `out`: bf16 (odt MOE_DT_BF16; may be x itself
 * where ldx == H) or 8-bit rows (odt MOE_DT_E4M3, out_scale [M, H/128], H a
 * multiple of 128).  rstd (NULL: not wanted) gets (mean(z^2) + eps)^(-1/2),
 * float32 [M], for the backward call (rounded where it is subnormal, an infinity
 * where it passes float32's range; y is right there too).  Sums are float32.  A
 * row's bits do not depend on the other rows or on their number.  Any H from 1 to
 * MOE_NORM_MAX_H and any element alignment; fastest with 16-byte aligned rows.
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE (M < 0, H, ldx, eps negative or not
 * finite, a type, residual_out without residual), MOE_ERR_LIMIT (H above the
 * limit, M >= 2^31), MOE_ERR_HIP. */
int moe_add_rms_norm(const void* x_bf16, int64_t ldx, const void* residual, moe_dtype rdt, void* residual_out,
                     const void* weight_bf16, float eps, void* out, moe_dtype odt, float* out_scale, float* rstd,
                     int64_t M, int32_t H, hipStream_t stream);

/* Bytes of workspace moe_add_rms_norm_backward needs (0 for sizes it refuses). */
size_t moe_add_rms_norm_backward_workspace_bytes(int64_t M, int32_t H);

/* Gradients of moe_add_rms_norm.  z is the normalised row (residual_out, or x
 * where there was no residual), bf16 or float32 (`zdt`) [M, H]; rstd what the
 * forward call wrote; dy bf16 [M, H] the gradient of y; dz (NULL: none, same type
 * as z) the gradient that arrives along the residual stream.
 *   t       = dy * weight,  n = z * rstd
 *   dx      = dz + rstd * (t - n * mean(t * n))     type of z, [M, H]
 *   dweight = sum over rows of dy * n               float32 [H]
 * dx is the gradient of x and of the residual alike; dx may be dz or dy's buffer
 * (dy's only where z is bf16).  dweight NULL: not computed.  With M == 0 dweight
 * is set to zero.  The column sums are float32 in a fixed order (workspace:
 * 16-byte aligned device memory of the size above, NULL where that is 0 or
 * dweight is NULL).  Errors as above, plus MOE_ERR_WORKSPACE. */
int moe_add_rms_norm_backward(const void* dy_bf16, const void* z, moe_dtype zdt, const void* weight_bf16,
                              const float* rstd, const void* dz, void* dx, float* dweight, int64_t M, int32_t H,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------- rows by expert and back again -- */

/* out[token_to_perm[t*top_k + k], :] = x[t, :] for every slot whose position is in
 * [0, rows).  x is [M, H] (bf16 or e4m3fn codes, `dt`) and out [rows, H] of the
 * same type; with e4m3fn rows x_scale [M, H/128] goes to out_scale [rows,
 * H/128] alike (H a multiple of 128).  Rows of `out` no slot maps to are not
 * written.  Positions in [0, rows) differ from slot to slot here and in
 * moe_unpermute_backward, as moe_align makes them: a row that two slots map to
 * gets the values of either.  Its gradient is moe_unpermute without weights.
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_LIMIT (M*top_k or rows >= 2^31),
 * MOE_ERR_HIP. */
int moe_permute(const void* x, moe_dtype dt, const float* x_scale, const int32_t* token_to_perm, int64_t M,
                int32_t top_k, int32_t H, void* out, float* out_scale, int64_t rows, hipStream_t stream);

/* out[t, :] = bf16(sum over k = 0..top_k-1, in that order, of w[t, k] *
 * y[token_to_perm[t*top_k + k], :]), float32 fused multiply-adds (plain adds
 * with topk_weights NULL, where every weight is 1), slots whose position is not
 * in [0, rows) skipped.  y bf16 [rows, H], out bf16 [M, H], topk_weights float32
 * [M, top_k].  A token without a slot gets zeros.  Errors as for moe_permute. */
int moe_unpermute(const void* y_bf16, const int32_t* token_to_perm, const float* topk_weights, int64_t M,
                  int32_t top_k, int32_t H, void* out_bf16, int64_t rows, hipStream_t stream);

/* Gradients of the weighted moe_unpermute, p = token_to_perm[t*top_k + k]:
 *   dy[p, :]          = bf16(w[t, k] * dout[t, :])
 *   dweights[t, k]    = <dout[t, :], y[p, :]>   (float32; 0 for a skipped slot)
 * Rows of dy no slot maps to are not written.  dy may be y's buffer. */
int moe_unpermute_backward(const void* dout_bf16, const void* y_bf16, const int32_t* token_to_perm,
                           const float* topk_weights, int64_t M, int32_t top_k, int32_t H, void* dy_bf16,
                           float* dweights, int64_t rows, hipStream_t stream);

/* --------------------------------------------------- the experts' products -- */

/* Activation of a product's epilogue: none, z*sigmoid(z), gelu (the tanh form:
 * z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))), and silu(z) * u with a second
 * product u (SwiGLU).  A sigmoid below e^-87, where float32's normal range ends,
 * counts as 0, in the gradients too. */
typedef enum { MOE_ACT_NONE = 0, MOE_ACT_SILU = 1, MOE_ACT_GELU = 2, MOE_ACT_SWIGLU = 3 } moe_act;

/* One product over sorted rows, for row p of expert e:
 *   z = W[e] x[p] + bias[e],  u = W_up[e] x[p] + up_bias[e] (SwiGLU only)
 *   y[p] = act(z[, u]) + residual[p]
 * accumulated in float32; z and u are not rounded on the way to y.
 *   w, up       row-major [E, N, K]: bf16 (wdt MOE_W_BF16) or e4m3fn codes with
 *               128x128 block scales (wdt MOE_W_FP8_E4M3)
 *   x           [rows, K]: bf16, or with e4m3fn weights 8-bit rows with x_scale
 *   bias        bf16 [E, N] or NULL; up_bias alike
 *   residual    bf16 [rows, N] or NULL
 *   y           [rows, N] of type ydt: bf16, or 8-bit rows with y_scale
 *   preact      NULL, or bf16 [rows, N] (SwiGLU: [rows, 2N], z then u): what
 *               moe_grouped_act_backward takes
 * expert_offsets (E + 1 entries) and expert_counts (E) NULL: one expert (E == 1)
 * that holds every row, i.e. a dense projection.
 * Shapes: bf16 needs K and N multiples of 8, e4m3fn multiples of 128; 8-bit y
 * needs N a multiple of 128.  x, w, up, bias, up_bias, y, residual and preact
 * 16-byte aligned.  The kernels' tiles are chosen by `rows` (over E, on average), in
 * which the alignment's padding counts: fastest with its block size no larger than
 * the experts' runs.
 * A bf16 y may be residual's buffer; an 8-bit y that overlaps it is refused.
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_LIMIT (E > MOE_MAX_EXPERTS, rows
 * >= 2^31, a matrix of one expert or 256 rows of x or y past 2^31 bytes, 2^31
 * tiles of 16 x 16 or nearly so), MOE_ERR_HIP. */
typedef struct {
  int64_t rows;
  int32_t E, N, K;
  moe_weight_dtype wdt;
  moe_act act;
  moe_dtype ydt;
  const int32_t* expert_offsets;
  const int32_t* expert_counts;
  const void* x;
  const float* x_scale;
  moe_weight w, up;
  const void* bias;
  const void* up_bias;
  const void* residual;
  void* y;
  float* y_scale;
  void* preact;
} moe_linear_desc;

int moe_grouped_linear(const moe_linear_desc* d, hipStream_t stream);

/* dz[p] from dy[p] (bf16 [rows, N]) and the pre-activations: silu and gelu
 * dy * act'(z), [rows, N]; SwiGLU dy * u * silu'(z) then dy * silu(z),
 * [rows, 2N].  All bf16, arithmetic in float32.  dz may be preact's buffer.
 * N a multiple of 8, pointers 16-byte aligned.  Offsets and counts as above. */
int moe_grouped_act_backward(const void* dy_bf16, const void* preact_bf16, moe_act act,
                             const int32_t* expert_offsets, const int32_t* expert_counts, int64_t rows, int32_t E,
                             int32_t N, void* dz_bf16, hipStream_t stream);

/* dx[p] = W[e]^T dz[p] (+ W_up[e]^T dz_up[p] with `up` non-NULL, where dz is
 * [rows, 2N]); dz bf16, w and up bf16 [E, N, K], dx bf16 [rows, K].  Shapes and
 * errors as for the bf16 moe_grouped_linear. */
int moe_grouped_linear_backward_x(const void* dz_bf16, const void* w_bf16, const void* up_bf16,
                                  const int32_t* expert_offsets, const int32_t* expert_counts, int64_t rows,
                                  int32_t E, int32_t N, int32_t K, void* dx_bf16, hipStream_t stream);

/* dw[e] = sum over the expert's rows p of dz[p]^T x[p] ([E, N, K], `wdt` bf16 or
 * float32) and, where db is non-NULL, db[e] = sum of dz[p] (float32 [E, N]).  With
 * `gated` non-zero dz is [rows, 2N] and dup, dup_b get its second half's.  An
 * expert without a row gets zeros.  db and dup_b are given together or not at
 * all (gated).  Float32 sums in a fixed order: where E * N * K is too small to
 * fill the GPU, each expert's rows are summed in equal parts that meet in the
 * workspace (16-byte aligned device memory of the size the query gives; NULL where
 * that is 0).  Shapes and errors as above, plus MOE_ERR_WORKSPACE. */
size_t moe_grouped_linear_backward_w_workspace_bytes(int64_t rows, int32_t E, int32_t N, int32_t K, int32_t gated,
                                                     int32_t bias);
int moe_grouped_linear_backward_w(const void* dz_bf16, const void* x_bf16, int32_t gated,
                                  const int32_t* expert_offsets, const int32_t* expert_counts, int64_t rows,
                                  int32_t E, int32_t N, int32_t K, moe_dtype wdt, void* dw, void* dup, float* db,
                                  float* dup_b, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* -------------------------------------------------------------- 4-bit rows -- */

/* Rows of x ([M, H], bf16 or float32 by `xdt`, `ldx` >= H elements from row to row,
 * H a multiple of 32) as MXFP4 rows.  With token_to_perm ([M * top_k]) the codes of
 * token t go to row token_to_perm[t*top_k + k] for every slot whose position is in
 * [0, rows), as moe_permute lays rows out: rows no slot maps to are not written, and
 * positions in [0, rows) differ from slot to slot.  With token_to_perm NULL row t goes
 * to row t (top_k 1, rows M).  Weights [E, N, K] are E * N rows of K, and the result
 * is what MOE_W_MXFP4 stands for.  codes 16-byte aligned, x at its element's
 * alignment, scales at any.  Errors: MOE_ERR_NULL, MOE_ERR_SHAPE (a size, a type, an
 * alignment), MOE_ERR_LIMIT (M*top_k or rows >= 2^31, H >= 2^29), MOE_ERR_HIP. */
int moe_mxfp4_quantize(const void* x, moe_dtype xdt, int64_t ldx, const int32_t* token_to_perm, int64_t M,
                       int32_t top_k, int32_t H, void* codes, uint8_t* scales, int64_t rows, hipStream_t stream);

/* The values of MXFP4 rows ([rows, H], H a multiple of 32), bf16 or float32 (`odt`):
 * exact, an infinity where they pass the type's largest value, NaN with the byte 255.
 * codes and out 16-byte aligned.  Errors as above. */
int moe_mxfp4_dequantize(const void* codes, const uint8_t* scales, int64_t rows, int32_t H, void* out, moe_dtype odt,
                         hipStream_t stream);

/* moe_grouped_linear on row-major MXFP4 weights:
 *   w, up       codes [E, N, K/2] with scale bytes [E, N, K/32]
 *   x           [rows, K] by `xdt`: bf16 (x_scale NULL), or MXFP4 rows with x_scale
 *   y           [rows, N] by `ydt`: bf16, or MXFP4 rows with y_scale
 * and everything else as there.  Weights and MXFP4 rows enter the products as the
 * values they stand for, sums are float32 (scale bytes 2 to 252 are exact; 255 makes
 * NaN of its block's products; the others' results are not specified).
 * Shapes: K a multiple of 32, N of 8, with MXFP4 y of 32.  x, w.w, up.w, bias,
 * up_bias, y, residual and preact 16-byte aligned, scale bytes at any alignment.  A
 * bf16 y may be residual's buffer; an MXFP4 y that overlaps it is refused.  Errors as
 * for moe_grouped_linear. */
typedef struct {
  int64_t rows;
  int32_t E, N, K;
  moe_dtype xdt;
  moe_act act;
  moe_dtype ydt;
  const int32_t* expert_offsets;
  const int32_t* expert_counts;
  const void* x;
  const uint8_t* x_scale;
  moe_weight w, up;
  const void* bias;
  const void* up_bias;
  const void* residual;
  void* y;
  uint8_t* y_scale;
  void* preact;
} moe_linear_mxfp4_desc;

int moe_grouped_linear_mxfp4(const moe_linear_mxfp4_desc* d, hipStream_t stream);

/* moe_grouped_linear_backward_x on such weights (`up` NULL: one product): dz bf16
 * [rows, N] (or [rows, 2N]), dx bf16 [rows, K].  The weights' own gradient does not
 * depend on them: moe_grouped_linear_backward_w gives it, from bf16 rows. */
int moe_grouped_linear_mxfp4_backward_x(const void* dz_bf16, const moe_weight* w, const moe_weight* up,
                                        const int32_t* expert_offsets, const int32_t* expert_counts, int64_t rows,
                                        int32_t E, int32_t N, int32_t K, void* dx_bf16, hipStream_t stream);

/* ------------------------------------------------------- gradients, clipped -- */

/* One of many gradients: `n` elements of type `dt` (bf16 or float32), contiguous, at
 * their element's alignment (n may be 0).  `out` is where moe_grad_clip writes it: g
 * itself or a buffer that overlaps no tensor of the list; the norm does not use it. */
typedef struct {
  const void* g;
  void* out;
  int64_t n;
  moe_dtype dt;
} moe_grad_tensor;

/* Bytes of workspace (8-byte aligned device memory) for `count` tensors; 0 for a count
 * the calls refuse. */
size_t moe_grad_norm_workspace_bytes(int64_t count);

/* norm[0] = (sum over the tensors' elements of g^2)^(1/2): summed in 64 bits in a
 * fixed order, rounded to float32 (0 without an element, an infinity past its range).
 * `list` is host memory and is read before the call returns.  Errors: MOE_ERR_NULL,
 * MOE_ERR_SHAPE (a count or size negative, a type, an alignment, a workspace that lies
 * over a gradient or the norm), MOE_ERR_LIMIT (2^20 tensors, 2^44 elements),
 * MOE_ERR_WORKSPACE, MOE_ERR_HIP. */
int moe_grad_norm(const moe_grad_tensor* list, int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                  hipStream_t stream);

/* out = g * c for every tensor, rounded to its type, with c = max_norm / norm[0] where
 * norm[0] is past max_norm (finite, not negative), else 1; also 1 where norm[0] is NaN or
 * infinite: gradients that it cannot scale stay as they are, and the norm tells.  norm
 * is device memory and not an output.  A gradient that stays as it is and where it is is
 * not written.  Errors as above, plus MOE_ERR_SHAPE for max_norm, for an `out` that
 * overlaps another tensor of the list or a part of its own, and for a norm that lies over
 * an output. */
int moe_grad_clip(const moe_grad_tensor* list, int64_t count, const float* norm, float max_norm, hipStream_t stream);

/* moe_grad_norm, then moe_grad_clip with its result: the same bits in fewer launches,
 * except that finite gradients whose norm passes float32's range (norm[0] is an infinity
 * then) are scaled by the norm as it was summed, in 64 bits.  The norm is written while
 * gradients are read, so it may not lie over one of them either (MOE_ERR_SHAPE). */
int moe_clip_grad_norm(const moe_grad_tensor* list, int64_t count, float max_norm, float* norm, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_OPS_H */
