// Sorting tokens by id and summing rows by sorted token, shared by the
// embedding's gradient and the output head.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "lm/common.cuh"

namespace mns {
namespace lm {

// Workspace of a sort of `tokens` ids below `vocab` and of the row sums.
struct SumLayout {
  size_t sorted, other, partial, total;
  long long pieces;
  int piece;  // sorted positions a warp sums before it stores a partial row
};
SumLayout sum_layout(long long tokens, int dim);

struct SortBy {
  const void* ids;
  int ids64;
  long long tokens, vocab;
  long long skip;  // an id to be taken as naming no row (-1: none more)
  int presence;    // sort by whether an id names a row alone (key 0: it does, 1: it does not)
  int* count;      // optional, device: how many do (written by a sort of more than kRankTokens)
};

// Key of an id that names no row.
MNS_HD long long none_of(const SortBy& by) { return by.presence ? 1 : by.vocab; }

__device__ __forceinline__ unsigned int sort_key(const SortBy& by, long long t) {
  long long id = load_id(by.ids, by.ids64, t, by.vocab);
  if (id == by.skip) id = -1;
  if (by.presence && id >= 0) id = 0;
  return static_cast<unsigned int>(id < 0 ? none_of(by) : id);
}

// Up to this many tokens are sorted by counting, for each, the smaller ones.
constexpr int kRankTokens = 4096;
constexpr int kRankBlock = 32;      // tokens a CTA of 1024 threads ranks
constexpr size_t kRankSmem = sizeof(unsigned int) * kRankTokens;

// Ranks tokens 32 b to 32 b + 31 among all, ties by token, by the 1024 threads
// of a CTA: warp t returns the rank of token 32 b + t, and its key.  Every
// warp compares the 32 tokens, a lane each, with a 32nd of the keys, four to a
// shared-memory read.
__device__ __forceinline__ int rank_tokens(const SortBy& by, int b, unsigned int* keys, unsigned int* key_out) {
  __shared__ int part[32][33];
  const int n = static_cast<int>(by.tokens), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pad = (n + 127) / 128 * 128;
  for (int i = tid; i < pad; i += 1024) keys[i] = i < n ? sort_key(by, i) : 0xFFFFFFFFu;  // past every key
  __syncthreads();
  const int i0 = b * kRankBlock, i = i0 + lane;
  const unsigned int mine = i < n ? keys[i] : 0u;
  int below = 0;
#pragma unroll 4
  for (int q = warp; q < pad / 4; q += 32) {
    const uint4 v = reinterpret_cast<const uint4*>(keys)[q];
    const int j = 4 * q;
    if (j >= i0 && j < i0 + kRankBlock) {
      below += (v.x < mine || (v.x == mine && j < i)) ? 1 : 0;
      below += (v.y < mine || (v.y == mine && j + 1 < i)) ? 1 : 0;
      below += (v.z < mine || (v.z == mine && j + 2 < i)) ? 1 : 0;
      below += (v.w < mine || (v.w == mine && j + 3 < i)) ? 1 : 0;
    } else {
      const unsigned int top = mine + (j < i0 ? 1u : 0u);  // earlier equal keys come first
      below += v.x < top ? 1 : 0;
      below += v.y < top ? 1 : 0;
      below += v.z < top ? 1 : 0;
      below += v.w < top ? 1 : 0;
    }
  }
  part[warp][lane] = below;
  __syncthreads();
  const int r = __reduce_add_sync(0xFFFFFFFFu, part[lane][warp]);
  *key_out = __shfl_sync(0xFFFFFFFFu, mine, warp);
  return r;
}

// How many of at most kRankTokens ids name a row, by the 1024 threads of a CTA.
__device__ __forceinline__ int count_live(const SortBy& by) {
  int live = 0;
#pragma unroll
  for (int k = 0; k < kRankTokens / 1024; ++k) {
    const int i = k * 1024 + static_cast<int>(threadIdx.x);
    live += __syncthreads_count(i < by.tokens && sort_key(by, i) < none_of(by) ? 1 : 0);
  }
  return live;
}

// Rows of a table to be set to zero where no token names them.
struct ZeroRows {
  void* table;       // null: none
  long long row_bytes;
};

// Sorts the tokens by id (stable): sorted[p] = id << 32 | token, ids that name
// no row last with id = none_of(by); and meanwhile zeroes the table's rows
// that do not occur.
cudaError_t launch_sort(const SortBy& by, const ZeroRows& zero, uint8_t* ws, const SumLayout& L, cudaStream_t stream);

// Row sums by sorted token: out[v] = scale * sum of src[t] over the tokens of
// v (accumulate: added to), for the v that occur.
cudaError_t launch_row_sums(const void* src, int src_type, long long tokens, long long vocab, int dim, float scale,
                            void* out, int out_type, int accumulate, uint8_t* ws, const SumLayout& L,
                            cudaStream_t stream);

// The same into compact rows: sum of coef[p] src[t] over the tokens t of v, p
// their sorted positions, goes to row q of out (fp32 [tokens][dim]), q the
// position of the first of them; slot[v] = q.  The slots of other v are not
// written: slot[v] is one if sorted[slot[v]] has key v.
cudaError_t launch_row_sums_compact(const void* src, const float* coef, long long tokens, long long vocab, int dim,
                                    float* out, int* slot, uint8_t* ws, const SumLayout& L, cudaStream_t stream);

}  // namespace lm
}  // namespace mns
