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
 *     call to the next.
 *   - Element types are MUON_LM_BF16 or MUON_LM_F32.  Sums, norm statistics
 *     and softmax statistics are held in fp32 whatever the element type, and
 *     results are rounded once.
 *   - Every result is deterministic: no floating-point atomics, and each sum
 *     is taken in an order that the sizes alone determine.
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

int muon_embed_grad_workspace_size(long long tokens, long long vocab, int dim, size_t* bytes);

/* dtable[v] = scale * sum over the tokens t with ids[t] == v of dy[t]
 * (accumulate != 0: added to dtable[v], rows without tokens left alone; else
 * every row is written, zero where no token names it).
 *   dy  [tokens][dim], dtable  [vocab][dim]; no overlap.
 * The tokens are sorted by id (stable), and each row is summed in fp32 in
 * token order, long rows in fixed pieces that are then joined in order. */
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

int muon_layer_norm_grad_workspace_size(long long rows, int dim, size_t* bytes);

/* Gradient, from the mean and rstd that muon_layer_norm wrote.  With
 * xh = (x - mean) rstd and a = dy weight,
 *   dx = rstd (a - mean_row(a) - xh mean_row(a xh)),
 *   dweight = sum_rows dy xh,  dbias = sum_rows dy.
 * dbias may be NULL (not wanted).  dx may be dy or x. */
int muon_layer_norm_grad(const void* dy, const void* x, int x_type, const void* weight, int w_type,
                         const float* mean, const float* rstd, long long rows, int dim, void* dx, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_LM_H */
