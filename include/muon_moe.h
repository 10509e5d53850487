/*
 * muon_moe.h — C ABI of the operators of a block with experts, whose matrices
 * the Muon step of muon_ns.h trains as one stack: root-mean-square norm with
 * the residual's addition, the router, the products grouped by expert, and the
 * weighted sum that brings the experts' rows back to their tokens, each with its
 * gradient; and the 8-bit storage (e4m3 with a scale for each block of 128) that
 * the norm writes and the grouped product reads.  Exported by the same library
 * (libmuon_ns.so).
 *
 * Conventions, as in muon_lm.h:
 *   - Device pointers owned by the caller, contiguous row-major arrays.  Work
 *     is enqueued on `stream`; nothing is allocated, nothing synchronises, so
 *     every call can be captured in a CUDA graph.
 *   - Arguments are validated on the host before anything is launched and a
 *     status code of muon_ns.h is returned.  Workspaces are device memory,
 *     256-byte aligned, of at least the size the _workspace_size function
 *     gives; their contents need not be initialised and carry nothing from one
 *     call to the next.  Where that size is 0, the workspace is not looked at.
 *   - Element types are MUON_LM_BF16 or MUON_LM_F32.  Sums and statistics are
 *     held in fp32 whatever the element type, and results are rounded once.
 *   - Results are deterministic: the same inputs at addresses of the same
 *     alignment give the same bits, with no floating-point atomics.
 *
 * 8-bit storage: values in e4m3 (largest 448) and fp32 scales; the value stood
 * for is the product of the two.  A block's scale is its largest magnitude
 * divided by 448 (by the quantiser rounded up where it is below the normal
 * numbers), 1 if that magnitude is zero.  A block that holds a NaN or an infinity
 * has a scale of NaN, so that all of it stands for NaN.  Blocks at an edge are
 * shorter.
 */
#ifndef MUON_MOE_H
#define MUON_MOE_H

#include "muon_lm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Root-mean-square norm over the last axis, with the residual's addition:
 *   s = x + residual (rounded to x_type; x itself without a residual),
 *   r = 1 / sqrt(mean(s^2) + eps),  y = s r weight.
 * x, residual, s, y, dy, dsum, ds: [rows][dim] of x_type; weight: [dim] of
 * w_type; rstd ([rows], r) and dweight: fp32.  Limits: rows <= 2^30,
 * 1 <= dim <= 2^20 (dim 0 with rows > 0 is an error: its mean does not exist).
 * Any dim and any pointer aligned to its element type; the widest accesses that
 * dim and the pointers allow are used.  The mean of squares is an fp32 number: where
 * it passes the largest r is 0, and squares below the smallest are lost.
 * ------------------------------------------------------------------------- */

/* residual may be NULL (s is then not written: it is x, which y may not be where the
 * gradient is wanted), s and rstd may be NULL (not wanted).  s may be x or residual,
 * and y may be x or residual, but s and y are not the same; otherwise outputs overlap
 * nothing. */
int muon_rms_norm(const void* x, int x_type, const void* residual, const void* weight, int w_type, long long rows,
                  int dim, float eps, void* s, void* y, float* rstd, cudaStream_t stream);

/* y in 8 bits, not rounded to x_type before: y e4m3 [rows][dim], scales fp32
 * [rows][ceil(dim / 128)].  y and scales overlap nothing.  (r goes into the scales,
 * so the products s weight have to be within fp32.) */
int muon_rms_norm8(const void* x, int x_type, const void* residual, const void* weight, int w_type, long long rows,
                   int dim, float eps, void* s, void* y, float* scales, float* rstd, cudaStream_t stream);

/* 0 for few rows: the workspace may then be NULL. */
int muon_rms_norm_grad_workspace_size(long long rows, int dim, size_t* bytes);

/* Gradient, from the s and rstd of the forward pass.  With xh = s rstd and
 * a = dy weight,
 *   ds = rstd (a - xh mean_row(a xh)) + dsum,  dweight = sum_rows dy xh:
 * ds is the gradient of x and of the residual alike.  dsum, the gradient that
 * reaches s past the norm, may be NULL (none).  ds may be dy, s or dsum; otherwise
 * outputs and workspace overlap nothing. */
int muon_rms_norm_grad(const void* dy, const void* s, int x_type, const void* weight, int w_type, const float* rstd,
                       const void* dsum, long long rows, int dim, void* ds, float* dweight, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/* x into 8-bit storage.  square = 0: a scale for each 128 columns of a row,
 * scales fp32 [batch][rows][ceil(dim / 128)].  square = 1: one for each block of
 * 128 rows and 128 columns of each of the batch's matrices, fp32
 * [batch][ceil(rows / 128)][ceil(dim / 128)], as muon_experts8 takes W.
 *   x  [batch][rows][dim] of x_type, q  e4m3 of the same shape; no overlap of any.
 * Limits: batch <= 65535, rows <= 2^30, dim <= 2^20. */
int muon_quantize8(const void* x, int x_type, long long batch, long long rows, int dim, int square, void* q,
                   float* scales, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Router.  Each token takes the k experts of largest logit, in that order, ties
 * to the lower index.  An expert whose logit is -inf (or NaN) is not to be had:
 * a token with fewer than k to be had takes those, and its other choices are -1
 * with gate 0.  gates are softmax(logits) at the choices, over all experts, or
 * with renormalize != 0 over the token's choices.  A token with a NaN among its
 * logits has NaN gates.
 * The plan puts the choices in the order of experts, then of tokens:
 *   logits  [tokens][experts] of type; gates fp32, chosen and slots int32
 *   [tokens][k]; token_of int32 [tokens k]; offsets int32 [experts + 1];
 *   offsets[e] .. offsets[e + 1] are the rows of expert e, slots[t][j] the row of
 *   token t's choice j (-1 for none) and token_of[row] its token, -1 from
 *   offsets[experts] on.  muon_embed(x, token_of) brings the tokens' rows of x
 *   there, muon_combine brings rows back.  Outputs overlap nothing.
 * Limits: 1 <= k <= 32, k <= experts <= 1024, tokens k <= 2^30.
 * ------------------------------------------------------------------------- */

/* 0 for up to 256 tokens: the workspace may then be NULL. */
int muon_route_workspace_size(long long tokens, int experts, int k, size_t* bytes);

int muon_route(const void* logits, int type, long long tokens, int experts, int k, int renormalize, float* gates,
               int* chosen, int* slots, int* token_of, int* offsets, void* workspace, size_t workspace_bytes,
               cudaStream_t stream);

/* Gradient of sum(dgates gates): dlogits [tokens][experts] of type, which
 * overlaps nothing.  The choice itself has no gradient.  chosen as muon_route
 * writes it, an expert once a token.  Renormalised, the choices' logits alone are
 * read: a NaN among the others is in the gates, not here. */
int muon_route_grad(const float* dgates, const void* logits, int type, const int* chosen, long long tokens, int experts,
                    int k, int renormalize, void* dlogits, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Combination of the experts' rows:
 *   out[t] = sum_j gates[t][j] y[slots[t][j]],
 *   dy[slots[t][j]] = gates[t][j] dout[t],  dgates[t][j] = <dout[t], y[slots[t][j]]>.
 * y, dy [rows][dim], out, dout [tokens][dim] of type; slots int32, gates and
 * dgates fp32 [tokens][k].  A slot outside [0, rows) is left out (its dgates are
 * 0).  gates NULL: all 1; muon_combine is then also the gradient of the tokens'
 * dispatch by muon_embed(x, token_of).
 * For the gradient a row is named by one slot at most, as muon_route does: of one
 * that is named twice dy holds either term.  Rows that no slot names are left as
 * they were.  dy or dgates may be NULL (not wanted).  Outputs overlap nothing
 * (dy may be y where dgates is NULL).
 * Limits: 1 <= k <= 32, tokens, rows <= 2^30, dim <= 2^20; any alignment.
 * ------------------------------------------------------------------------- */

int muon_combine(const void* y, int type, const int* slots, const float* gates, long long tokens, int k, long long rows,
                 int dim, void* out, cudaStream_t stream);

int muon_combine_grad(const void* dout, const void* y, int type, const int* slots, const float* gates, long long tokens,
                      int k, long long rows, int dim, void* dy, float* dgates, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Products grouped by expert.  Row r of x belongs to expert e where
 * offsets[e] <= r < offsets[e + 1]:
 *   y_r = W_e x_r,   dx_r = W_e^T dy_r,   dW_e = sum_r dy_r x_r^T.
 *   x, dx  bf16 [rows][dim], W  bf16 [experts][out_dim][dim], y, dy  bf16
 *   [rows][out_dim], dW  [experts][out_dim][dim] of dW_type;
 *   offsets  device int32 [experts + 1], not decreasing (muon_route writes
 *   them).  An expert may have no rows: its W is not read, its dW is zero.
 *   Rows of no expert (before offsets[0], from offsets[experts] on) are not
 *   read, and their rows of y and dx are left as they were.  Offsets outside
 *   [0, rows] count as the nearest bound, and nothing outside the arrays is
 *   touched whatever they hold (where they decrease, some rows may get no value).
 * Limits: rows <= 2^30, experts <= 1024, out_dim, dim <= 2^20, fewer than 2^30
 * tiles of 128 rows x 256 features (dW: of 256 x 256); out_dim and dim multiples of 8 (for muon_experts8 dim a
 * multiple of 16) and arrays 16-byte aligned: MUON_NS_ERR_ALIGNMENT otherwise.
 * Outputs (`device_error` among them) overlap nothing.  Products accumulate in fp32 on
 * the tensor cores.
 * `device_error` is an optional device int32 (may be NULL), as in muon_ns_gram:
 * MUON_NS_DEVERR_WAIT_TIMEOUT is set in it if a bounded wait runs out
 * (muon_ns_set_wait_budget), and nothing is where none does.  What such a call
 * could not compute is NaN.
 * ------------------------------------------------------------------------- */

int muon_experts(const muon_bf16* x, const muon_bf16* W, const int* offsets, long long rows, int experts, int out_dim,
                 int dim, muon_bf16* y, int* device_error, cudaStream_t stream);

/* dx or dW may be NULL (not wanted; W or x may then be NULL).  accumulate != 0
 * (fp32 dW only): dW is added to.  An fp32 dW is what muon_step_ws takes as G. */
int muon_experts_grad(const muon_bf16* dy, const muon_bf16* x, const muon_bf16* W, const int* offsets, long long rows,
                      int experts, int out_dim, int dim, muon_bf16* dx, void* dW, int dW_type, int accumulate,
                      int* device_error, cudaStream_t stream);

/* y of 8-bit x and W:
 *   x  e4m3 [rows][dim], x_scales  fp32 [rows][ceil(dim / 128)],
 *   W  e4m3 [experts][out_dim][dim], W_scales  fp32 [experts][ceil(out_dim / 128)][ceil(dim / 128)].
 * The products of each 128 of dim are summed by the tensor cores, then scaled
 * and added in fp32. */
int muon_experts8(const void* x, const float* x_scales, const void* W, const float* W_scales, const int* offsets,
                  long long rows, int experts, int out_dim, int dim, muon_bf16* y, int* device_error,
                  cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MOE_H */
