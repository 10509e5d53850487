// Token embedding and its gradient.
//
// Forward: Y[t] = s E[ids[t]], a gather of rows bound by HBM traffic; rows of
// repeated tokens come from L2.
//
// Gradient: dE[v] = s sum_{ids[t] = v} dY[t].  Atomics would give a sum whose
// order changes from run to run and would serialise on frequent tokens, so the
// tokens are sorted by id first:
//   token_sort     one cluster sorts (id, token) pairs by radix, stable, so a
//                  row's tokens follow one another in token order, and marks
//                  the ids that occur in a bitmap;
//   row_sums       a warp takes kPiece sorted positions and 256 columns, adds
//                  the rows in fp32 registers and writes a row of dE where it
//                  ends inside the piece; a row that crosses pieces leaves one
//                  partial row in each.  Other warps zero the rows of the ids
//                  that do not occur, so dE is written once;
//   row_sums_join  adds the partial rows of a row in piece order.
// dY is read once and dE written once: bound by HBM traffic.
#include <cmath>
#include <type_traits>

#include "lm/common.cuh"
#include "lm/embed.cuh"

namespace mns {
namespace lm {

namespace {

// ----------------------------------------------------------------- forward --

constexpr int kLookups = 4;  // tokens a thread has in flight

// A token's row is walked by 1 << lanes_log2 threads of a CTA of 256.
template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(256)
    embed_fwd(const TI* __restrict__ table, long long vocab, int dim, const void* __restrict__ ids, int ids64,
              long long tokens, float scale, TO* __restrict__ out, int lanes_log2) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lanes = 1 << lanes_log2;
  const int rows = 256 >> lanes_log2;
  const int tx = threadIdx.x & (lanes - 1), ty = threadIdx.x >> lanes_log2;
  const long long t0 = static_cast<long long>(blockIdx.x) * (rows * kLookups) + ty;
  long long id[kLookups];
#pragma unroll
  for (int u = 0; u < kLookups; ++u) {
    const long long t = t0 + u * rows;
    id[u] = t < tokens ? load_id(ids, ids64, t, vocab) : -1;
  }
  for (int c = tx * VEC; c < dim; c += lanes * VEC) {
    Vec<TI, VEC> v[kLookups];
#pragma unroll
    for (int u = 0; u < kLookups; ++u)
      if (id[u] >= 0) v[u] = load_global<TI, VEC>(table + id[u] * dim + c);
#pragma unroll
    for (int u = 0; u < kLookups; ++u) {
      const long long t = t0 + u * rows;
      if (t < tokens) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = id[u] >= 0 ? scale * to_f32(v[u].v[j]) : 0.0f;
        store_global<TO, VEC>(out + t * dim + c, o);
      }
    }
  }
}

// -------------------------------------------------------------------- sort --

constexpr int kMaxDigit = 9;            // bits a pass sorts by
constexpr int kBins = 1 << kMaxDigit;
constexpr int kSortWarps = 32;
constexpr int kSortUnroll = 8;          // elements a thread loads at once
constexpr int kSortCluster = 8;         // CTAs of the sort, at most
constexpr int kSortTokens = 2048;       // tokens a CTA of it should have, at least
constexpr size_t kSortSmem = sizeof(int) * kSortWarps * kBins;

// One cluster.  Each CTA owns a contiguous part of the tokens and each warp a
// contiguous part of that.  A pass counts digits per warp, turns the counts
// into the first output position of each (digit, CTA, warp) in that order, and
// writes every element to its warp's next position: stable, since a warp
// takes its elements in order and match_any ranks the lanes of one digit.
__global__ void __launch_bounds__(32 * kSortWarps)
    token_sort(const void* __restrict__ ids, int ids64, long long tokens, long long vocab, const SortBy by, int passes,
               int digit_bits, unsigned long long* buf_even, unsigned long long* buf_odd, unsigned int* bitmap,
               long long words) {
  extern __shared__ int cnt[];  // [kSortWarps][kBins]
  __shared__ int totals[kBins];
  __shared__ int base[kBins];
  __shared__ int scan_sh[kSortWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = static_cast<int>(gridDim.x);  // the whole grid is one cluster
  const int rank = static_cast<int>(blockIdx.x);
  const long long per_cta = ((tokens + ctas - 1) / ctas + 31) / 32 * 32;
  const long long per_warp = ((per_cta + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const long long cta_begin = rank * per_cta;
  long long cta_end = cta_begin + per_cta;
  if (cta_end > tokens) cta_end = tokens;
  const long long begin = cta_begin + warp * per_warp;
  long long end = begin + per_warp;
  if (end > cta_end) end = cta_end;
  const long long none = by.presence ? 1 : vocab;  // key of an id that names no row
  const int bins = 1 << digit_bits;
  int* mine = cnt + warp * kBins;

  for (long long i = static_cast<long long>(rank) * blockDim.x + tid; i < words;
       i += static_cast<long long>(ctas) * blockDim.x)
    bitmap[i] = 0u;

  for (int pass = 0; pass < passes; ++pass) {
    // Pass p writes buf_even if p is even; the last result is in the buffer
    // the host names.
    const unsigned long long* src = (pass & 1) ? buf_even : buf_odd;
    unsigned long long* dst = (pass & 1) ? buf_odd : buf_even;
    const int shift = 32 + pass * digit_bits;
    auto fetch = [&](long long i) -> unsigned long long {
      if (pass > 0) return __ldcg(src + i);
      long long id = load_id(ids, ids64, i, vocab);
      if (id == by.skip) id = -1;
      if (by.presence && id >= 0) id = 0;
      return (static_cast<unsigned long long>(id < 0 ? none : id) << 32) | static_cast<unsigned long long>(i);
    };
    for (int d = lane; d < bins; d += 32) mine[d] = 0;
    __syncwarp();
    auto walk = [&](auto&& take) {
      for (long long b = begin; b < end; b += 32 * kSortUnroll) {
        unsigned long long e[kSortUnroll];
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u) {
          const long long i = b + u * 32 + lane;
          if (i < end) e[u] = fetch(i);
        }
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u) {
          const long long i = b + u * 32 + lane;
          const bool live = i < end;
          const int d = live ? static_cast<int>((e[u] >> shift) & static_cast<unsigned>(bins - 1)) : kBins;
          const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
          const int before = __popc(same & ((1u << lane) - 1u));
          take(live, d, before, __popc(same), e[u]);
          __syncwarp();
        }
      }
    };
    walk([&](bool live, int d, int before, int n, unsigned long long) {
      if (live && before == 0) mine[d] += n;
    });
    __syncthreads();
    // Counts -> offsets of each warp inside its CTA, and the CTA's totals.
    if (tid < bins) {
      int run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w * kBins + tid];
        cnt[w * kBins + tid] = run;
        run += c;
      }
      totals[tid] = run;
    }
    __syncthreads();
    if (ctas > 1) ptx::cluster_sync();
    int before_cta = 0, all = 0;
    if (tid < bins) {
      for (int r = 0; r < ctas; ++r) {
        int c;
        if (ctas > 1) {
          const uint32_t a = ptx::mapa(ptx::smem_u32(&totals[tid]), static_cast<uint32_t>(r));
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(a) : "memory");
        } else {
          c = totals[tid];
        }
        if (r < rank) before_cta += c;
        all += c;
      }
    }
    // Exclusive scan of the digits' totals.
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan_sh[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int v = scan_sh[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += up;
      }
      scan_sh[lane] = v;
    }
    __syncthreads();
    if (tid < bins) base[tid] = incl - all + (warp > 0 ? scan_sh[warp - 1] : 0) + before_cta;
    __syncthreads();
    walk([&](bool live, int d, int before, int n, unsigned long long e) {
      if (live) dst[base[d] + mine[d] + before] = e;
      __syncwarp();
      if (live && before == 0) mine[d] += n;
    });
    // The pass's writes are read by every CTA; totals and counts are reused.
    if (ctas > 1)
      ptx::cluster_sync();
    else
      __syncthreads();
  }
  if (words == 0 && by.count == nullptr) return;
  const unsigned long long* sorted = (passes & 1) ? buf_even : buf_odd;
  for (long long i = static_cast<long long>(rank) * blockDim.x + tid; i < tokens;
       i += static_cast<long long>(ctas) * blockDim.x) {
    const unsigned int k = static_cast<unsigned int>(__ldcg(sorted + i) >> 32);
    const bool first = i == 0 || static_cast<unsigned int>(__ldcg(sorted + i - 1) >> 32) != k;
    const bool live = k < none;
    if (words > 0 && first && live) atomicOr(bitmap + (k >> 5), 1u << (k & 31));
    if (by.count != nullptr) {
      if (first && !live) *by.count = static_cast<int>(i);
      if (live && i == tokens - 1) *by.count = static_cast<int>(tokens);
    }
  }
}

// ---------------------------------------------------------------- row sums --

constexpr int kSliceCols = 256;  // columns of a warp: 8 a lane
constexpr int kSumWarps = 8;
constexpr int kSumUnroll = 8;    // rows a warp has in flight
constexpr int kZeroRows = 8;     // table rows a zeroing warp looks after

struct SumParams {
  const void* src;
  void* out;
  const unsigned long long* sorted;
  const unsigned int* bitmap;
  float* partial;  // [pieces][2][dim]: the row that began before the piece, the one that goes on after it
  const float* coef;  // COMPACT: factor of each sorted position
  int* slot;          // COMPACT
  long long tokens, vocab, pieces;
  int dim, slices, accumulate;
  float scale;
};

__device__ __forceinline__ unsigned int key_of(unsigned long long e) { return static_cast<unsigned int>(e >> 32); }
__device__ __forceinline__ unsigned int token_of(unsigned long long e) { return static_cast<unsigned int>(e); }

// Lane's columns of slice s: 8 / VEC vectors of VEC, 32 VEC columns apart.
template <int VEC>
__device__ __forceinline__ int slice_col(int s, int lane, int k) {
  return s * kSliceCols + (k * 32 + lane) * VEC;
}

template <typename TO, int VEC>
__device__ __forceinline__ void write_row(TO* row, int s, int lane, int dim, float scale, int accumulate,
                                          const float (&a)[8 / VEC][VEC]) {
#pragma unroll
  for (int k = 0; k < 8 / VEC; ++k) {
    const int c = slice_col<VEC>(s, lane, k);
    if (c < dim) {
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = scale * a[k][j];
      if (accumulate) {
        const Vec<TO, VEC> old = load_global<TO, VEC>(row + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += to_f32(old.v[j]);
      }
      store_global<TO, VEC>(row + c, o);
    }
  }
}

template <typename TS, typename TO, int VEC, bool COMPACT>
__global__ void __launch_bounds__(32 * kSumWarps) row_sums(const SumParams P) {
  constexpr int kK = 8 / VEC;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kSumWarps + (threadIdx.x >> 5);
  const long long sums = P.pieces * P.slices;
  TO* out = static_cast<TO*>(P.out);
  if (item >= sums) {
    if (COMPACT || P.accumulate) return;
    // Rows of ids that do not occur.
    const long long v0 = (item - sums) * kZeroRows;
    if (v0 >= P.vocab) return;
    const unsigned int bits = P.bitmap[v0 >> 5] >> (v0 & 31);
    const float zero[VEC] = {};
    for (int r = 0; r < kZeroRows; ++r)
      if (v0 + r < P.vocab && !((bits >> r) & 1u))
        for (int c = lane * VEC; c < P.dim; c += 32 * VEC) store_global<TO, VEC>(out + (v0 + r) * P.dim + c, zero);
    return;
  }
  const long long piece = item / P.slices;
  const int s = static_cast<int>(item - piece * P.slices);
  const long long p0 = piece * kPiece;
  const int n = static_cast<int>(P.tokens - p0 < kPiece ? P.tokens - p0 : kPiece);
  const unsigned int none = static_cast<unsigned int>(P.vocab);
  const unsigned long long e = lane < n ? P.sorted[p0 + lane] : (static_cast<unsigned long long>(none) << 32);
  const unsigned int key = key_of(e);
  // The keys around the piece, `none` past the ends.
  const unsigned int prev = p0 > 0 ? key_of(P.sorted[p0 - 1]) : none;
  const unsigned int next = p0 + n < P.tokens ? key_of(P.sorted[p0 + n]) : none;
  unsigned int follow = __shfl_down_sync(0xFFFFFFFFu, key, 1);
  if (lane == n - 1) follow = next;
  const unsigned int ends = __ballot_sync(0xFFFFFFFFu, lane < n && follow != key);
  const TS* src = static_cast<const TS*>(P.src);
  float a[kK][VEC] = {};
  // The run being summed began before this piece.
  bool head = prev == __shfl_sync(0xFFFFFFFFu, key, 0);
  int start = 0;
  for (int b = 0; b < n; b += kSumUnroll) {
    Vec<TS, VEC> v[kSumUnroll][kK];
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u) {
      const unsigned int ku = __shfl_sync(0xFFFFFFFFu, key, b + u);
      const long long t = __shfl_sync(0xFFFFFFFFu, token_of(e), b + u);
      if (ku != none) {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const int c = slice_col<VEC>(s, lane, k);
          if (c < P.dim) v[u][k] = load_global<TS, VEC>(src + t * P.dim + c);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u) {
      const int p = b + u;
      const unsigned int ku = __shfl_sync(0xFFFFFFFFu, key, p);
      if (ku == none) continue;
      float f = 1.0f;
      if (COMPACT) f = P.coef[p0 + p];
#pragma unroll
      for (int k = 0; k < kK; ++k)
        if (slice_col<VEC>(s, lane, k) < P.dim)
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            a[k][j] = COMPACT ? fmaf(f, to_f32(v[u][k].v[j]), a[k][j]) : a[k][j] + to_f32(v[u][k].v[j]);
      const bool ended = (ends >> p) & 1u;
      if (COMPACT && s == 0 && lane == 0 && p == start && !head) P.slot[ku] = static_cast<int>(p0 + p);
      if (ended || p == n - 1) {
        if (ended && !head) {
          const long long row = COMPACT ? p0 + start : static_cast<long long>(ku);
          write_row<TO, VEC>(out + row * P.dim, s, lane, P.dim, P.scale, P.accumulate, a);
        } else {
          float* row = P.partial + (piece * 2 + (head ? 0 : 1)) * P.dim;
          write_row<float, VEC>(row, s, lane, P.dim, 1.0f, 0, a);
        }
        head = false;
        start = p + 1;
#pragma unroll
        for (int k = 0; k < kK; ++k)
#pragma unroll
          for (int j = 0; j < VEC; ++j) a[k][j] = 0.0f;
      }
    }
  }
}

// A CTA looks at kSumWarps pieces; for each whose last row begins in it and
// goes on, the CTA's warps add that row's partial rows, each a contiguous part
// of the pieces, and the warps' sums are added in order.
template <typename TO, int VEC, bool COMPACT>
__global__ void __launch_bounds__(32 * kSumWarps) row_sums_join(const SumParams P) {
  constexpr int kK = 8 / VEC;
  __shared__ float red[kSumWarps][kSliceCols];
  __shared__ long long first_sh[kSumWarps], last_sh[kSumWarps];
  __shared__ unsigned int key_sh[kSumWarps];
  __shared__ int at_sh[kSumWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.y;
  const unsigned int none = static_cast<unsigned int>(P.vocab);
  const long long piece = static_cast<long long>(blockIdx.x) * kSumWarps + warp;
  long long lo = 0, hi = 0;
  unsigned int key = none;
  int at = 0;
  if (piece + 1 < P.pieces) {
    const long long p0 = piece * kPiece;
    const unsigned int k = key_of(P.sorted[p0 + lane]);
    key = __shfl_sync(0xFFFFFFFFu, k, 31);
    // Positions of this piece in the run, and whether it began in the piece.
    const unsigned int same = __ballot_sync(0xFFFFFFFFu, k == key);
    at = __ffs(same) - 1;
    const bool began = at > 0 || p0 == 0 || key_of(P.sorted[p0 - 1]) != key;
    if (key != none && began && key_of(P.sorted[p0 + kPiece]) == key) {
      // Last piece of the run: 32 probes a turn between lo (in the run) and hi.
      lo = piece + 1;
      hi = P.pieces;
      while (hi - lo > 1) {
        const long long step = (hi - lo + 31) / 32;
        const long long q = lo + (lane + 1) * step;
        const bool in = q < hi && key_of(P.sorted[q * kPiece]) == key;
        const int ok = __popc(__ballot_sync(0xFFFFFFFFu, in));  // monotone
        const long long nlo = lo + ok * step;
        if (nlo + step < hi) hi = nlo + step;
        lo = nlo;
      }
    } else {
      key = none;
    }
  }
  if (lane == 0) {
    first_sh[warp] = piece;
    last_sh[warp] = lo;
    key_sh[warp] = key;
    at_sh[warp] = at;
  }
  __syncthreads();
  for (int w = 0; w < kSumWarps; ++w) {
    if (key_sh[w] == none) continue;
    const long long first = first_sh[w], last = last_sh[w];
    const long long count = last - first + 1;  // partial rows, two at least
    const long long per = (count + kSumWarps - 1) / kSumWarps;
    const long long b = first + warp * per;
    const long long e = b + per < last + 1 ? b + per : last + 1;
    float a[kK][VEC] = {};
    for (long long q0 = b; q0 < e; q0 += 4) {
      Vec<float, VEC> v[4][kK];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u < e) {
          const float* row = P.partial + ((q0 + u) * 2 + (q0 + u == first ? 1 : 0)) * P.dim;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const int c = slice_col<VEC>(s, lane, k);
            if (c < P.dim) v[u][k] = load_global<float, VEC>(row + c);
          }
        }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (q0 + u < e)
#pragma unroll
          for (int k = 0; k < kK; ++k)
            if (slice_col<VEC>(s, lane, k) < P.dim)
#pragma unroll
              for (int j = 0; j < VEC; ++j) a[k][j] += v[u][k].v[j];
    }
    __syncthreads();  // the last turn's sums have been read
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) red[warp][(k * 32 + lane) * VEC + j] = a[k][j];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < kK; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          for (int g = 1; g < kSumWarps; ++g) a[k][j] += red[g][(k * 32 + lane) * VEC + j];
      const long long row = COMPACT ? first * kPiece + at_sh[w] : static_cast<long long>(key_sh[w]);
      write_row<TO, VEC>(static_cast<TO*>(P.out) + row * P.dim, s, lane, P.dim, P.scale, P.accumulate, a);
    }
  }
}

int bits_of(long long v) {
  int b = 1;
  while ((v >> b) != 0) ++b;
  return b;
}

// Passes and digit of the sort of keys from 0 to `largest`.
void sort_plan(long long largest, int* passes, int* digit) {
  const int bits = bits_of(largest);
  *passes = (bits + kMaxDigit - 1) / kMaxDigit;
  *digit = (bits + *passes - 1) / *passes;
}

template <typename TS, typename TO, int VEC, bool COMPACT>
cudaError_t launch_sums(const SumParams& P, cudaStream_t stream) {
  const long long zero = COMPACT || P.accumulate ? 0 : (P.vocab + kZeroRows - 1) / kZeroRows;
  const long long items = P.pieces * P.slices + zero;
  cudaError_t e = mns::launch_pdl(row_sums<TS, TO, VEC, COMPACT>,
                                  dim3(static_cast<unsigned>((items + kSumWarps - 1) / kSumWarps)),
                                  dim3(32 * kSumWarps), 0, stream, P);
  if (e != cudaSuccess || P.pieces < 2) return e;
  return mns::launch_pdl(row_sums_join<TO, VEC, COMPACT>,
                         dim3(static_cast<unsigned>((P.pieces + kSumWarps - 1) / kSumWarps), P.slices),
                         dim3(32 * kSumWarps), 0, stream, P);
}

SumParams sum_params(const void* src, long long tokens, long long vocab, int dim, float scale, void* out,
                     int accumulate, uint8_t* ws, const SumLayout& L) {
  SumParams P = {};
  P.src = src;
  P.out = out;
  P.sorted = reinterpret_cast<const unsigned long long*>(ws + L.sorted);
  P.bitmap = reinterpret_cast<const unsigned int*>(ws + L.bitmap);
  P.partial = reinterpret_cast<float*>(ws + L.partial);
  P.tokens = tokens;
  P.vocab = vocab;
  P.pieces = L.pieces;
  P.dim = dim;
  P.slices = (dim + kSliceCols - 1) / kSliceCols;
  P.accumulate = accumulate;
  P.scale = scale;
  return P;
}

int check(long long tokens, long long vocab, int dim, int ids_bits) {
  if (tokens < 0 || vocab < 0 || dim < 0 || tokens > kMaxRows || vocab > kMaxRows || dim > kMaxDim)
    return MUON_NS_ERR_INVALID_ARG;
  if (ids_bits != 32 && ids_bits != 64) return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

bool ids_aligned(const void* ids, int ids_bits) {
  return (reinterpret_cast<uintptr_t>(ids) & static_cast<uintptr_t>(ids_bits / 8 - 1)) == 0;
}

}  // namespace

SumLayout sum_layout(long long tokens, long long vocab, int dim) {
  SumLayout L;
  L.pieces = (tokens + kPiece - 1) / kPiece;
  size_t off = 0;
  L.sorted = off;
  off = align_up(off + 8 * static_cast<size_t>(tokens), 256);
  L.other = off;
  off = align_up(off + 8 * static_cast<size_t>(tokens), 256);
  L.bitmap = off;
  off = align_up(off + 4 * static_cast<size_t>((vocab + 31) / 32), 256);
  L.partial = off;
  off = align_up(off + 8 * static_cast<size_t>(L.pieces) * dim, 256);
  L.total = off;
  return L;
}

cudaError_t launch_sort(const void* ids, int ids64, long long tokens, long long vocab, const SortBy& by, uint8_t* ws,
                        const SumLayout& L, cudaStream_t stream) {
  int passes, digit;
  sort_plan(by.presence ? 1 : vocab, &passes, &digit);
  int ctas = 1;
  while (ctas < kSortCluster && static_cast<long long>(ctas) * kSortTokens < tokens) ctas *= 2;
  auto* last = reinterpret_cast<unsigned long long*>(ws + L.sorted);
  auto* other = reinterpret_cast<unsigned long long*>(ws + L.other);
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(configured.load() >> (dev & 63) & 1ull)) {
    e = cudaFuncSetAttribute(token_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSortSmem));
    if (e != cudaSuccess) return e;
    configured.fetch_or(1ull << (dev & 63));
  }
  return mns::launch_pdl_cluster(token_sort, dim3(ctas), dim3(32 * kSortWarps), kSortSmem, stream, ctas, ids, ids64,
                                 tokens, vocab, by, passes, digit, (passes & 1) ? last : other,
                                 (passes & 1) ? other : last, reinterpret_cast<unsigned int*>(ws + L.bitmap),
                                 by.presence ? 0 : (vocab + 31) / 32);
}

cudaError_t launch_row_sums(const void* src, int src_type, long long tokens, long long vocab, int dim, float scale,
                            void* out, int out_type, int accumulate, uint8_t* ws, const SumLayout& L,
                            cudaStream_t stream) {
  const SumParams P = sum_params(src, tokens, vocab, dim, scale, out, accumulate, ws, L);
  // The partial rows (fp32, 256-byte aligned) allow what dim allows.
  const int vec = min_vec(vec_of(dim, src, src_type), vec_of(dim, out, out_type));
  return with_type(src_type, [&](auto st) {
    return with_type(out_type, [&](auto ot) {
      return with_vec(vec, [&](auto vc) {
        return launch_sums<decltype(st), decltype(ot), decltype(vc)::value, false>(P, stream);
      });
    });
  });
}

cudaError_t launch_row_sums_compact(const void* src, const float* coef, long long tokens, long long vocab, int dim,
                                    float* out, int* slot, uint8_t* ws, const SumLayout& L, cudaStream_t stream) {
  SumParams P = sum_params(src, tokens, vocab, dim, 1.0f, out, 0, ws, L);
  P.coef = coef;
  P.slot = slot;
  return launch_sums<bf16, float, 8, true>(P, stream);  // the head's rows are multiples of 8
}

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_embed(const void* table, int table_type, long long vocab, int dim, const void* ids, int ids_bits,
               long long tokens, float scale, void* out, int out_type, cudaStream_t stream) {
  int s = check(tokens, vocab, dim, ids_bits);
  if (s != MUON_NS_OK) return s;
  if (!type_ok(table_type) || !type_ok(out_type) || !std::isfinite(scale)) return MUON_NS_ERR_INVALID_ARG;
  if (tokens == 0 || dim == 0) return MUON_NS_OK;
  if ((vocab > 0 && !table) || !ids || !out) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(table, table_type) || !element_aligned(out, out_type) || !ids_aligned(ids, ids_bits))
    return MUON_NS_ERR_ALIGNMENT;
  if (overlap(table, static_cast<size_t>(vocab) * dim * type_size(table_type), out,
              static_cast<size_t>(tokens) * dim * type_size(out_type)))
    return MUON_NS_ERR_INVALID_ARG;
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  const int vec = min_vec(vec_of(dim, table, table_type), vec_of(dim, out, out_type));
  int lanes_log2 = 0;
  while (lanes_log2 < 8 && ((1 << lanes_log2) * vec) < dim) ++lanes_log2;
  const long long per = static_cast<long long>(256 >> lanes_log2) * kLookups;
  const unsigned grid = static_cast<unsigned>((tokens + per - 1) / per);
  return with_type(table_type, [&](auto it) {
    return with_type(out_type, [&](auto ot) {
      return with_vec(vec, [&](auto vc) {
        using TI = decltype(it);
        using TO = decltype(ot);
        return status_of(mns::launch_pdl(embed_fwd<TI, TO, decltype(vc)::value>, dim3(grid), dim3(256), 0, stream,
                                         static_cast<const TI*>(table), vocab, dim, ids, ids_bits == 64 ? 1 : 0,
                                         tokens, scale, static_cast<TO*>(out), lanes_log2));
      });
    });
  });
}

int muon_embed_grad_workspace_size(long long tokens, long long vocab, int dim, size_t* bytes) {
  const int s = check(tokens, vocab, dim, 32);
  if (s != MUON_NS_OK) return s;
  if (!bytes) return MUON_NS_ERR_INVALID_ARG;
  *bytes = tokens == 0 || vocab == 0 || dim == 0 ? 0 : sum_layout(tokens, vocab, dim).total;
  return MUON_NS_OK;
}

int muon_embed_grad(const void* dy, int dy_type, const void* ids, int ids_bits, long long tokens, long long vocab,
                    int dim, float scale, void* dtable, int dtable_type, int accumulate, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  int s = check(tokens, vocab, dim, ids_bits);
  if (s != MUON_NS_OK) return s;
  if (!type_ok(dy_type) || !type_ok(dtable_type) || !std::isfinite(scale)) return MUON_NS_ERR_INVALID_ARG;
  if (vocab == 0 || dim == 0) return MUON_NS_OK;
  if (!dtable || (tokens > 0 && (!dy || !ids))) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(dy, dy_type) || !element_aligned(dtable, dtable_type) || !ids_aligned(ids, ids_bits))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t table_bytes = static_cast<size_t>(vocab) * dim * type_size(dtable_type);
  if (tokens > 0 && overlap(dy, static_cast<size_t>(tokens) * dim * type_size(dy_type), dtable, table_bytes))
    return MUON_NS_ERR_INVALID_ARG;
  const SumLayout L = sum_layout(tokens, vocab, dim);
  if (tokens > 0 && (!workspace || workspace_bytes < L.total)) return MUON_NS_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_NS_ERR_ALIGNMENT;
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  if (tokens == 0) return accumulate ? MUON_NS_OK : status_of(cudaMemsetAsync(dtable, 0, table_bytes, stream));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaError_t e = launch_sort(ids, ids_bits == 64 ? 1 : 0, tokens, vocab, SortBy{-1, 0, nullptr}, ws, L, stream);
  if (e != cudaSuccess) return status_of(e);
  return status_of(launch_row_sums(dy, dy_type, tokens, vocab, dim, scale, dtable, dtable_type, accumulate ? 1 : 0, ws,
                                   L, stream));
}

}  // extern "C"
