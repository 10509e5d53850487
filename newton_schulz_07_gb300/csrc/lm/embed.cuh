// Sorting tokens by id and summing rows by sorted token, shared by the
// embedding's gradient and the output head.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace mns {
namespace lm {

// Sorted positions a warp sums before it stores a partial row.
constexpr int kPiece = 32;

// Workspace of a sort of `tokens` ids below `vocab` and of the row sums.
struct SumLayout {
  size_t sorted, other, bitmap, partial, total;
  long long pieces;
};
SumLayout sum_layout(long long tokens, long long vocab, int dim);

struct SortBy {
  long long skip;  // an id to be taken as naming no row (-1: none more)
  int presence;    // sort by whether an id names a row alone (0: it does, 1: it does not); no bitmap
  int* count;      // optional, device: how many do
};

// Sorts the tokens by id (stable): sorted[p] = id << 32 | token, ids outside
// [0, vocab) last with id = vocab.  Bit v of `bitmap` says whether v occurs.
cudaError_t launch_sort(const void* ids, int ids64, long long tokens, long long vocab, const SortBy& by, uint8_t* ws,
                        const SumLayout& L, cudaStream_t stream);

// Row sums by sorted token: out[v] = scale * sum of src[t] over the tokens of
// v, every row of the table written (accumulate: added to).
cudaError_t launch_row_sums(const void* src, int src_type, long long tokens, long long vocab, int dim, float scale,
                            void* out, int out_type, int accumulate, uint8_t* ws, const SumLayout& L,
                            cudaStream_t stream);

// The same into compact rows: sum of coef[p] src[t] over the tokens t of v, p
// their sorted positions, goes to row q of out (fp32 [tokens][dim]), q the position of the first of
// them; slot[v] = q.  Rows of ids that do not occur have no slot (bitmap).
cudaError_t launch_row_sums_compact(const void* src, const float* coef, long long tokens, long long vocab, int dim,
                                    float* out, int* slot, uint8_t* ws, const SumLayout& L, cudaStream_t stream);

}  // namespace lm
}  // namespace mns
