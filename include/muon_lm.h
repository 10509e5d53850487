/*
 * muon_lm.h — C ABI of the operators at the ends of a language model, for the
 * training step around the Muon update of muon_ns.h: the token embedding, the
 * layer norm and the output head's cross entropy, each with its gradient.
 * Exported by the same library (libmuon_ns.so).
 *
 * Conventions, as in muon_ns.h:
 *   - Device pointers owned by the caller, contiguous row-major arrays.  Work
 *     is enqueued on `stream`; nothing is allocated, nothing synchronises, so
 *     every call can be captured in a CUDA graph.
 *   - Arguments are validated on the host before anything is launched and a
 *     status code of muon_ns.h is returned.  Workspaces are device memory,
 *     256-byte aligned, of at least the size the _workspace_size function
 *     gives; their contents need not be initialised and carry nothing from one
 *     call to the next.  Where that size is 0, the workspace is not looked at.
 *   - Element types are MUON_LM_BF16 or MUON_LM_F32.  Sums, norm statistics
 *     and softmax statistics are held in fp32 whatever the element type, and
 *     results are rounded once.
 *   - Results are deterministic: the same inputs at addresses of the same
 *     alignment give the same bits, with no floating-point atomics.  The order
 *     of a sum follows from the sizes and types, in the layer norm also from
 *     the pointers' alignment (which sets the width of accesses), and in the
 *     head from the targets (tokens are taken in their order, and how many have
 *     a loss sets the splits of dh).
 */
#ifndef MUON_LM_H
#define MUON_LM_H

#include "muon_ns.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { MUON_LM_BF16 = 0, MUON_LM_F32 = 1 };

/* ---------------------------------------------------------------------------
 * Token embedding.
 *   ids  device int32 or int64 [tokens] (ids_bits = 32 or 64).  An id outside
 *        [0, vocab), such as a padding id of -1, names no row: its output row
 *        is zero and it has no gradient.
 * Limits: tokens, vocab <= 2^30, dim <= 2^20.  Any dim and any pointer aligned
 * to its element type; the widest accesses that dim and the pointers allow are
 * used (16 bytes when dim is a multiple of 8 and the pointers of 16 bytes).
 * ------------------------------------------------------------------------- */

/* out[t] = scale * table[ids[t]], computed in fp32 and rounded once.
 *   table  [vocab][dim], out  [tokens][dim]; out must not overlap table. */
int muon_embed(const void* table, int table_type, long long vocab, int dim, const void* ids, int ids_bits,
               long long tokens, float scale, void* out, int out_type, cudaStream_t stream);

/* 0 up to 256 tokens: the workspace may then be NULL. */
int muon_embed_grad_workspace_size(long long tokens, long long vocab, int dim, size_t* bytes);

/* dtable[v] = scale * sum over the tokens t with ids[t] == v of dy[t]
 * (accumulate != 0: added to dtable[v], rows without tokens left alone; else
 * every row is written, zero where no token names it).
 *   dy  [tokens][dim], dtable  [vocab][dim]; no overlap.
 * More than 256 tokens are sorted by id (stable).  Each row is summed in fp32
 * in token order, long rows in fixed pieces that are then joined in order. */
int muon_embed_grad(const void* dy, int dy_type, const void* ids, int ids_bits, long long tokens, long long vocab,
                    int dim, float scale, void* dtable, int dtable_type, int accumulate, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Layer norm over the last axis: with mu = mean(x) and
 * r = 1 / sqrt(mean((x - mu)^2) + eps) of a row,
 *   y = (x - mu) r weight + bias.
 * x, y, dy, dx: [rows][dim] of x_type; weight, bias: [dim] of w_type; mean,
 * rstd, dweight, dbias: fp32.  Limits: rows <= 2^30, 1 <= dim <= 2^20 (dim 0
 * with rows > 0 is an error: its mean does not exist).
 * ------------------------------------------------------------------------- */

/* bias may be NULL (none).  mean and rstd ([rows] each) may be NULL if the
 * backward pass is not wanted.  y may be x. */
int muon_layer_norm(const void* x, int x_type, const void* weight, const void* bias, int w_type, long long rows,
                    int dim, float eps, void* y, float* mean, float* rstd, cudaStream_t stream);

/* 0 for few rows: the workspace may then be NULL. */
int muon_layer_norm_grad_workspace_size(long long rows, int dim, size_t* bytes);

/* Gradient, from the mean and rstd that muon_layer_norm wrote.  With
 * xh = (x - mean) rstd and a = dy weight,
 *   dx = rstd (a - mean_row(a) - xh mean_row(a xh)),
 *   dweight = sum_rows dy xh,  dbias = sum_rows dy.
 * dbias may be NULL (not wanted).  dx may be dy or x. */
int muon_layer_norm_grad(const void* dy, const void* x, int x_type, const void* weight, int w_type,
                         const float* mean, const float* rstd, long long rows, int dim, void* dx, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Output head: softmax cross entropy of h W^T over a large vocabulary.  The
 * logits are not kept: the losses alone hold none of them, the gradient holds
 * bf16 probabilities of one piece of the vocabulary (`pieces` below) in the
 * workspace.  For token n with target t,
 *   z = h_n W^T,  loss_n = log sum_v exp(z_v) - z_t,
 * and with g_n = dloss[n] (1 / (tokens with a loss) if dloss is NULL) and
 * p = softmax(z), the gradient of sum_n g_n loss_n is
 *   dh_n = g_n (sum_v p_v W_v - W_t),  dW_v = sum_n g_n (p_nv - [v = t_n]) h_n.
 *   h  bf16 [tokens][dim], W  bf16 [vocab][dim], loss  fp32 [tokens],
 *   dh  bf16 [tokens][dim], dW  [vocab][dim] of dW_type;
 *   targets  int32 or int64 [tokens] (target_bits).  A target outside
 *   [0, vocab) or equal to ignore_index takes the token out: loss 0, dh 0, no
 *   part in dW, whatever its row of h and its dloss hold, and no work.
 * dim must be a multiple of 8 (16-byte rows) and h, W, dh and dW 16-byte
 * aligned: MUON_NS_ERR_ALIGNMENT otherwise.  dh and dW overlap nothing.
 * Products accumulate in fp32 on the tensor cores; sums, logarithms and the
 * targets' terms are fp32: a target that holds nearly all of the probability
 * has its loss and its terms to the relative accuracy of the logits' differences.
 * The other probabilities enter dh and dW as bf16 operands, and h with its factor
 * g / sum exp enters dW as bf16, so an fp32 dW is no more exact than that.
 * The device error word is the first int of the workspace, as for muon_ns_ws
 * (muon_ns_read_error, muon_ns_check; waits bounded by
 * muon_ns_set_wait_budget); a call on no tokens or no vocabulary leaves it.
 * Where a wait ran out, every result of the call is NaN as well: loss, dh and
 * all of dW, accumulated or not.
 * ------------------------------------------------------------------------- */

/* Workspace of muon_head_loss (grad = 0) or muon_head_loss_grad (grad != 0).
 * pieces: pieces of the vocabulary that the gradient is taken in (of whole
 * 256 columns).  The workspace holds the probabilities of one piece in bf16
 * (tokens x piece).  With one piece 3 products are computed, with more the
 * probabilities of all but one piece are computed twice, up to 4.  0: as few
 * as keep a piece at about 4 GiB.  Ignored for grad = 0. */
int muon_head_workspace_size(long long tokens, long long vocab, int dim, int grad, int pieces, size_t* bytes);

/* The losses alone. */
int muon_head_loss(const muon_bf16* h, const muon_bf16* W, long long tokens, long long vocab, int dim,
                   const void* targets, int target_bits, long long ignore_index, float* loss, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream);

/* The losses and the gradient in one call.  accumulate != 0 (fp32 dW only):
 * dW is added to.  dloss: device fp32 [tokens], or NULL. */
int muon_head_loss_grad(const muon_bf16* h, const muon_bf16* W, long long tokens, long long vocab, int dim,
                        const void* targets, int target_bits, long long ignore_index, const float* dloss, int pieces,
                        float* loss, muon_bf16* dh, void* dW, int dW_type, int accumulate, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_LM_H */
