// Token embedding and its gradient.
//
// Forward: Y[t] = s E[ids[t]], a gather of rows bound by HBM traffic; rows of
// repeated tokens come from L2.
//
// Gradient: dE[v] = s sum_{ids[t] = v} dY[t].  Atomics would give a sum whose
// order changes from run to run and would serialise on frequent tokens, so the
// tokens are sorted by id first:
//   token_rank,   up to 4096 tokens: each token's place is the number of smaller
//   token_sort    ones, counted by all SMs; more: one cluster sorts (id, token)
//                 pairs by radix.  Both stable, so a row's tokens follow one
//                 another in token order.  The other CTAs of the launch zero
//                 the rows of dE that no token names, so dE is written once;
//   row_sums      a warp takes a piece of 8 or 32 sorted positions and 256 columns, adds
//                 the rows in fp32 registers and writes a row of dE where it
//                 ends inside the piece; a row that crosses pieces leaves one
//                 partial row in each;
//   row_sums_join adds the partial rows of a row in piece order.
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
// CTAs of the sort: 8, or 4 where the launch zeroes so much that this takes
// longer than the sort: clusters of 8 leave a sixth of the SMs without a CTA,
// clusters of 4 a twentieth (65536 tokens, 131072 rows: 8 KB a row 318 us with
// 8, 251 with 4; 32 bytes a row 64 and 98 us).
constexpr int kSortAlone = 8, kSortBeside = 4;
constexpr long long kMuchZeroing = 400LL << 20;  // bytes of the table, about 60 us
constexpr size_t kSortSmem = sizeof(int) * kSortWarps * kBins;
constexpr unsigned int kZeroWindow = 1 << 17;  // rows whose presence a zeroing CTA holds at once
constexpr unsigned int kFewWindow = 1 << 15;
static_assert(kZeroWindow / 8 <= kRankSmem && kZeroWindow / 8 <= kSortSmem, "presence bits");

template <typename V>
__device__ __forceinline__ void zero_row(uint8_t* row, long long bytes, int lane) {
  for (long long c = lane * sizeof(V); c < bytes; c += 32 * sizeof(V)) *reinterpret_cast<V*>(row + c) = V{};
}

// CTA `cta` of `ctas` zeroes, of rows cta, cta + ctas, ..., those
// that no token names, as its own reading of the ids says.  (Rows in turn, not
// in parts: frequent ids lie together.)
template <unsigned int kWindow>
__device__ __forceinline__ void zero_absent(const SortBy& by, const ZeroRows& zero, int cta, int ctas, unsigned int* bits) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned int n = static_cast<unsigned int>((by.vocab - cta + ctas - 1) / ctas);  // rows of this CTA
  const unsigned int inverse = 0xFFFFFFFFu / static_cast<unsigned int>(ctas);
  uint8_t* table = static_cast<uint8_t*>(zero.table);
  const long long rb = zero.row_bytes;
  const unsigned long long step = static_cast<unsigned long long>(rb) | reinterpret_cast<uintptr_t>(table);
  for (unsigned int a = 0; a < n; a += kWindow) {
    const unsigned int m = n - a < kWindow ? n - a : kWindow;
    for (unsigned int i = tid; i < (m + 31) / 32; i += blockDim.x) bits[i] = 0u;
    __syncthreads();
#pragma unroll 8
    for (long long t = tid; t < by.tokens; t += blockDim.x) {
      const unsigned int key = sort_key(by, t);
      // key / ctas and the remainder, from a quotient that may be a few short.
      unsigned int q = __umulhi(key, inverse), r = key - q * ctas;
      while (r >= static_cast<unsigned int>(ctas)) {
        ++q;
        r -= ctas;
      }
      if (r == static_cast<unsigned int>(cta) && q - a < m) {
        // Frequent ids find their bit set: no queue of atomics on one word.
        const unsigned int i = q - a, bit = 1u << (i & 31);
        if (!(*static_cast<volatile unsigned int*>(&bits[i >> 5]) & bit)) atomicOr(&bits[i >> 5], bit);
      }
    }
    __syncthreads();
    for (unsigned int i = warp; i < m; i += blockDim.x >> 5) {
      if ((bits[i >> 5] >> (i & 31)) & 1u) continue;
      uint8_t* row = table + (static_cast<long long>(a + i) * ctas + cta) * rb;
      if ((step & 31) == 0) {
        const float z[8] = {};
#pragma unroll 4
        for (long long c = lane * 32; c < rb; c += 1024) store_global<float, 8>(reinterpret_cast<float*>(row + c), z);
      } else if ((step & 15) == 0) {
        zero_row<uint4>(row, rb, lane);
      } else if ((step & 3) == 0) {
        zero_row<unsigned int>(row, rb, lane);
      } else {
        zero_row<unsigned short>(row, rb, lane);
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(1024)
    token_rank(const SortBy by, const ZeroRows zero, int blocks, unsigned long long* __restrict__ sorted) {
  extern __shared__ __align__(16) unsigned int keys[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (static_cast<int>(blockIdx.x) >= blocks) {
    zero_absent<kZeroWindow>(by, zero, static_cast<int>(blockIdx.x) - blocks, static_cast<int>(gridDim.x) - blocks, keys);
    return;
  }
  unsigned int key;
  const int r = rank_tokens(by, blockIdx.x, keys, &key);
  const long long t = static_cast<long long>(blockIdx.x) * kRankBlock + (threadIdx.x >> 5);
  if ((threadIdx.x & 31) == 0 && t < by.tokens) sorted[r] = (static_cast<unsigned long long>(key) << 32) | t;
}

// The grid's first cluster sorts.  Each of its CTAs owns a contiguous part of
// the tokens and each warp a contiguous part of that.  A pass counts digits per
// warp, turns the counts into the first output position of each (digit, CTA,
// warp) in that order, and writes every element to its warp's next position:
// stable, since a warp takes its elements in order and match_any ranks the
// lanes of one digit.
template <int ctas>
__global__ void __launch_bounds__(32 * kSortWarps)
    token_sort(const SortBy by, const ZeroRows zero, int passes, int digit_bits, unsigned long long* buf_even,
               unsigned long long* buf_odd) {
  extern __shared__ __align__(16) unsigned int sort_smem[];  // counts, [kSortWarps][kBins]
  __shared__ int totals[kBins];
  __shared__ int base[kBins];
  __shared__ int scan_sh[kSortWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x);
  if (rank >= ctas) {
    zero_absent<kZeroWindow>(by, zero, rank - ctas, static_cast<int>(gridDim.x) - ctas, sort_smem);
    return;
  }
  int* cnt = reinterpret_cast<int*>(sort_smem);
  const long long tokens = by.tokens;
  const long long per_cta = ((tokens + ctas - 1) / ctas + 31) / 32 * 32;
  const long long per_warp = ((per_cta + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const long long cta_begin = rank * per_cta;
  long long cta_end = cta_begin + per_cta;
  if (cta_end > tokens) cta_end = tokens;
  const long long begin = cta_begin + warp * per_warp;
  long long end = begin + per_warp;
  if (end > cta_end) end = cta_end;
  const int bins = 1 << digit_bits;
  int* mine = cnt + warp * kBins;

  for (int pass = 0; pass < passes; ++pass) {
    // Pass p writes buf_even if p is even; the last result is in the buffer
    // the host names.
    const unsigned long long* src = (pass & 1) ? buf_even : buf_odd;
    unsigned long long* dst = (pass & 1) ? buf_odd : buf_even;
    const int shift = 32 + pass * digit_bits;
    auto fetch = [&](long long i) -> unsigned long long {
      if (pass > 0) return __ldcg(src + i);
      return (static_cast<unsigned long long>(sort_key(by, i)) << 32) | static_cast<unsigned long long>(i);
    };
    for (int d = lane; d < bins; d += 32) mine[d] = 0;
    __syncwarp();
    // f of the element of each position of the warp's part, in order.
    auto walk = [&](auto&& f) {
      for (long long b = begin; b < end; b += 32 * kSortUnroll) {
        unsigned long long e[kSortUnroll];
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u) {
          const long long i = b + u * 32 + lane;
          if (i < end) e[u] = fetch(i);
        }
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u) {
          const bool live = b + u * 32 + lane < end;
          f(live, live ? static_cast<int>((e[u] >> shift) & static_cast<unsigned>(bins - 1)) : kBins, e[u]);
        }
      }
    };
    walk([&](bool live, int d, unsigned long long) {
      if (live) atomicAdd(&mine[d], 1);
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
    ptx::cluster_sync();
    int before_cta = 0, all = 0;
    if (tid < bins) {
      int c[ctas];
#pragma unroll
      for (int r = 0; r < ctas; ++r) {
        const uint32_t from = ptx::mapa(ptx::smem_u32(&totals[tid]), static_cast<uint32_t>(r));
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c[r]) : "r"(from));
      }
#pragma unroll
      for (int r = 0; r < ctas; ++r) {
        if (r < rank) before_cta += c[r];
        all += c[r];
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
    walk([&](bool live, int d, unsigned long long e) {
      const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int at = live ? mine[d] : 0;
      __syncwarp();
      if (live && before == 0) mine[d] = at + __popc(same);
      if (live) dst[base[d] + at + before] = e;
      __syncwarp();
    });
    // The pass's writes are read by every CTA; totals and counts are reused.
    ptx::cluster_sync();
  }
  if (by.count == nullptr) return;
  const unsigned long long* sorted = (passes & 1) ? buf_even : buf_odd;
  const unsigned int none = static_cast<unsigned int>(none_of(by));
  for (long long i = static_cast<long long>(rank) * blockDim.x + tid; i < tokens;
       i += static_cast<long long>(ctas) * blockDim.x) {
    const bool live = static_cast<unsigned int>(__ldcg(sorted + i) >> 32) < none;
    if (!live && (i == 0 || static_cast<unsigned int>(__ldcg(sorted + i - 1) >> 32) < none))
      *by.count = static_cast<int>(i);
    if (live && i == tokens - 1) *by.count = static_cast<int>(tokens);
  }
}

// ---------------------------------------------------------------- row sums --

constexpr int kSliceCols = 256;  // columns of a warp: 8 a lane
constexpr int kSumWarps = 8;
// Rows a warp has in flight.  (65536 tokens x 2048 bf16 take 88 us; 16 rows
// leave fewer warps an SM and take half as long again.)
constexpr int kSumUnroll = 8;

struct SumParams {
  const void* src;
  void* out;
  const unsigned long long* sorted;
  float* partial;  // [pieces][2][dim]: the row that began before the piece, the one that goes on after it
  const float* coef;  // COMPACT: factor of each sorted position
  int* slot;          // COMPACT
  long long tokens, vocab, pieces;
  int piece;  // sorted positions of a piece, at most 32
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
  if (item >= sums) return;
  const long long piece = item / P.slices;
  const int s = static_cast<int>(item - piece * P.slices);
  const long long p0 = piece * P.piece;
  const int n = static_cast<int>(P.tokens - p0 < P.piece ? P.tokens - p0 : P.piece);
  const unsigned int none = static_cast<unsigned int>(P.vocab);
  const unsigned long long e = lane < n ? P.sorted[p0 + lane] : (static_cast<unsigned long long>(none) << 32);
  const unsigned int key = key_of(e);
  const float coef = COMPACT && lane < n ? P.coef[p0 + lane] : 1.0f;
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
      if (COMPACT) f = __shfl_sync(0xFFFFFFFFu, coef, p);
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

// Few tokens: a warp takes a token and 256 columns and, if no earlier token has
// its id, adds the rows of all that do, in token order, so no sort and no
// partial rows are needed; other CTAs zero the rows that no token names.
// (256 tokens into 50257 rows, added: 8 us against 13 us by sorting, 29 us where
// nine in ten are the same; 1000 tokens 10 to 27 us, and 109 us.)
constexpr int kFewTokens = 256;
constexpr int kFewUnroll = 16;  // rows a warp has in flight: a frequent id's are one warp's

template <typename TS, typename TO, int VEC>
__global__ void __launch_bounds__(32 * kSumWarps)
    row_sums_few(const SortBy by, const ZeroRows zero, int blocks, const SumParams P) {
  constexpr int kK = 8 / VEC;
  __shared__ unsigned int bits[kFewWindow / 32];
  __shared__ unsigned int keys[kFewTokens];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (static_cast<int>(blockIdx.x) >= blocks) {
    zero_absent<kFewWindow>(by, zero, static_cast<int>(blockIdx.x) - blocks, static_cast<int>(gridDim.x) - blocks, bits);
    return;
  }
  const int n = static_cast<int>(by.tokens);
  const unsigned int none = static_cast<unsigned int>(none_of(by));
  for (int t = threadIdx.x; t < (n + 31) / 32 * 32; t += 32 * kSumWarps) keys[t] = t < n ? sort_key(by, t) : none;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kSumWarps + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(n) * P.slices) return;
  const int t0 = static_cast<int>(item / P.slices), s = static_cast<int>(item - static_cast<long long>(t0) * P.slices);
  const unsigned int key = keys[t0];
  if (key == none) return;
  for (int b = 0; b < t0; b += 32)
    if (__any_sync(0xFFFFFFFFu, b + lane < t0 && keys[b + lane] == key)) return;
  const TS* src = static_cast<const TS*>(P.src);
  float a[kK][VEC] = {};
  for (int b = t0 & ~31; b < n; b += 32) {
    unsigned int same = __ballot_sync(0xFFFFFFFFu, b + lane >= t0 && keys[b + lane] == key);
    while (same != 0u) {
      Vec<TS, VEC> v[(sizeof(TS) == 2 ? kFewUnroll : kSumUnroll)][kK];
      unsigned int m = same;
#pragma unroll
      for (int u = 0; u < (sizeof(TS) == 2 ? kFewUnroll : kSumUnroll); ++u) {
        if (m != 0u) {
          const long long t = b + __ffs(m) - 1;
          m &= m - 1u;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const int c = slice_col<VEC>(s, lane, k);
            if (c < P.dim) v[u][k] = load_global<TS, VEC>(src + t * P.dim + c);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < (sizeof(TS) == 2 ? kFewUnroll : kSumUnroll); ++u) {
        if (same != 0u) {
          same &= same - 1u;
#pragma unroll
          for (int k = 0; k < kK; ++k)
            if (slice_col<VEC>(s, lane, k) < P.dim)
#pragma unroll
              for (int j = 0; j < VEC; ++j) a[k][j] += to_f32(v[u][k].v[j]);
        }
      }
    }
  }
  write_row<TO, VEC>(static_cast<TO*>(P.out) + static_cast<long long>(key) * P.dim, s, lane, P.dim, P.scale,
                     P.accumulate, a);
}

// Few sorted tokens into compact rows: a warp takes a sorted position and 256
// columns and, if a row begins there, adds all of it.
template <int VEC>
__global__ void __launch_bounds__(32 * kSumWarps) row_sums_runs(const SumParams P) {
  static_assert(VEC == 8, "the head's rows");
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kSumWarps + (threadIdx.x >> 5);
  if (item >= P.tokens * P.slices) return;
  const int p0 = static_cast<int>(item / P.slices), s = static_cast<int>(item - static_cast<long long>(p0) * P.slices);
  const int n = static_cast<int>(P.tokens);
  const unsigned int key = key_of(P.sorted[p0]);
  if (key == static_cast<unsigned int>(P.vocab) || (p0 > 0 && key_of(P.sorted[p0 - 1]) == key)) return;
  if (s == 0 && lane == 0) P.slot[key] = p0;
  const int c = slice_col<VEC>(s, lane, 0);
  const bf16* src = static_cast<const bf16*>(P.src);
  float a[1][VEC] = {};
  for (int b = p0; b < n; b += 32) {
    const unsigned long long e = b + lane < n ? P.sorted[b + lane] : ~0ull;
    const float coef = b + lane < n ? P.coef[b + lane] : 0.0f;
    const int m = __popc(__ballot_sync(0xFFFFFFFFu, key_of(e) == key));  // contiguous from b
    for (int q = 0; q < m; q += kSumUnroll) {
      Vec<bf16, VEC> v[kSumUnroll];
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u) {
        const long long t = __shfl_sync(0xFFFFFFFFu, token_of(e), (q + u) & 31);
        if (q + u < m && c < P.dim) v[u] = load_global<bf16, VEC>(src + t * P.dim + c);
      }
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u) {
        const float f = __shfl_sync(0xFFFFFFFFu, coef, (q + u) & 31);
        if (q + u < m && c < P.dim)
#pragma unroll
          for (int j = 0; j < VEC; ++j) a[0][j] = fmaf(f, to_f32(v[u].v[j]), a[0][j]);
      }
    }
    if (m < 32) break;
  }
  write_row<float, VEC>(static_cast<float*>(P.out) + static_cast<long long>(p0) * P.dim, s, lane, P.dim, 1.0f, 0, a);
}

constexpr int kShortRun = 12;  // pieces of a row that one warp joins

// Sum over pieces [b, e) of a row's partial rows, `first` being the piece it
// began in.
template <int VEC>
__device__ __forceinline__ void add_pieces(const SumParams& P, long long b, long long e, long long first, int s,
                                           int lane, float (&a)[8 / VEC][VEC]) {
  constexpr int kK = 8 / VEC;
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
}

// A warp looks at a piece: if its last row begins in it and goes on, the row's
// partial rows are added in order, by the warp where they are few, else by the
// CTA's warps, each a contiguous part of them, and the warps' sums in order.
template <typename TO, int VEC, bool COMPACT>
__global__ void __launch_bounds__(32 * kSumWarps) row_sums_join(const SumParams P) {
  constexpr int kK = 8 / VEC;
  __shared__ float red[kSumWarps][kSliceCols];
  __shared__ long long last_sh[kSumWarps], row_sh[kSumWarps];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.y;
  const unsigned int none = static_cast<unsigned int>(P.vocab);
  const long long first0 = static_cast<long long>(blockIdx.x) * kSumWarps;
  const long long piece = first0 + warp;
  TO* out = static_cast<TO*>(P.out);
  long long last = -1;  // last piece of a row for the CTA to join
  if (piece + 1 < P.pieces) {
    const long long p0 = piece * P.piece;
    const bool in_piece = lane < P.piece;
    const unsigned int k = in_piece ? key_of(P.sorted[p0 + lane]) : none;
    const unsigned int after = key_of(P.sorted[p0 + P.piece]);
    const unsigned int prev = p0 > 0 ? key_of(P.sorted[p0 - 1]) : none;
    const unsigned int key = __shfl_sync(0xFFFFFFFFu, k, P.piece - 1);
    // The row's first position in this piece, and whether it began there.
    const int at = __ffs(__ballot_sync(0xFFFFFFFFu, in_piece && k == key)) - 1;
    if (key != none && after == key && (at > 0 || prev != key)) {
      // Last piece of the row: 32 probes a turn between lo (in the row) and hi.
      long long lo = piece + 1, hi = P.pieces;
      long long step = 1;  // the next 32 pieces first: most rows end there
      while (hi - lo > 1) {
        const long long q = lo + (lane + 1) * step;
        const bool in = q < hi && key_of(P.sorted[q * P.piece]) == key;
        const int ok = __popc(__ballot_sync(0xFFFFFFFFu, in));  // monotone
        lo += ok * step;
        if (ok < 32 && lo + step < hi) hi = lo + step;
        step = (hi - lo + 31) / 32;
      }
      const long long row = COMPACT ? p0 + at : static_cast<long long>(key);
      if (lo - piece < kShortRun) {
        float a[kK][VEC] = {};
        add_pieces<VEC>(P, piece, lo + 1, piece, s, lane, a);
        write_row<TO, VEC>(out + row * P.dim, s, lane, P.dim, P.scale, P.accumulate, a);
      } else {
        last = lo;
        if (lane == 0) row_sh[warp] = row;
      }
    }
  }
  if (lane == 0) last_sh[warp] = last;
  if (!__syncthreads_or(last >= 0 ? 1 : 0)) return;
  for (int w = 0; w < kSumWarps; ++w) {
    if (last_sh[w] < 0) continue;
    const long long first = first0 + w, end = last_sh[w] + 1;
    const long long per = (end - first + kSumWarps - 1) / kSumWarps;
    const long long b = first + warp * per;
    float a[kK][VEC] = {};
    add_pieces<VEC>(P, b, b + per < end ? b + per : end, first, s, lane, a);
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
      write_row<TO, VEC>(out + row_sh[w] * P.dim, s, lane, P.dim, P.scale, P.accumulate, a);
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
  const long long items = P.pieces * P.slices;
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
  P.partial = reinterpret_cast<float*>(ws + L.partial);
  P.tokens = tokens;
  P.vocab = vocab;
  P.pieces = L.pieces;
  P.piece = L.piece;
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

SumLayout sum_layout(long long tokens, int dim) {
  SumLayout L;
  // Short pieces give few tokens more warps; long ones leave fewer partial
  // rows.
  L.piece = tokens <= kRankTokens ? 8 : 32;
  L.pieces = (tokens + L.piece - 1) / L.piece;
  size_t off = 0;
  L.sorted = off;
  off = align_up(off + 8 * static_cast<size_t>(tokens), 256);
  L.other = off;
  off = align_up(off + 8 * static_cast<size_t>(tokens), 256);
  L.partial = off;
  off = align_up(off + 8 * static_cast<size_t>(L.pieces) * dim, 256);
  L.total = off;
  return L;
}

cudaError_t launch_sort(const SortBy& by, const ZeroRows& zero, uint8_t* ws, const SumLayout& L, cudaStream_t stream) {
  auto* last = reinterpret_cast<unsigned long long*>(ws + L.sorted);
  auto* other = reinterpret_cast<unsigned long long*>(ws + L.other);
  const int sms = sm_count();
  if (by.tokens <= kRankTokens) {
    const int blocks = static_cast<int>((by.tokens + kRankBlock - 1) / kRankBlock);
    // Zeroing CTAs: two fit an SM.
    const int zeros = zero.table == nullptr ? 0 : static_cast<int>(by.vocab < 2 * sms ? by.vocab : 2 * sms);
    return mns::launch_pdl(token_rank, dim3(blocks + zeros), dim3(1024), kRankSmem, stream, by, zero, blocks, last);
  }
  int passes, digit;
  sort_plan(none_of(by), &passes, &digit);
  unsigned long long *even = (passes & 1) ? last : other, *odd = (passes & 1) ? other : last;
  const auto launch = [&](auto kernel, int ctas, std::atomic<unsigned long long>* configured) {
    const cudaError_t e = allow_smem(kernel, static_cast<int>(kSortSmem), configured);
    if (e != cudaSuccess) return e;
    // One CTA fits an SM, and not every SM a cluster.
    int clusters = zero.table == nullptr ? 1 : (ctas == kSortBeside ? sms * 19 / 20 : sms * 5 / 6) / ctas;
    if (zero.table != nullptr && clusters < 2) clusters = 2;
    return mns::launch_pdl_cluster(kernel, dim3(clusters * ctas), dim3(32 * kSortWarps), kSortSmem, stream, ctas, by,
                                   zero, passes, digit, even, odd);
  };
  static std::atomic<unsigned long long> configured[2];
  if (zero.table != nullptr && by.vocab * zero.row_bytes > kMuchZeroing)
    return launch(token_sort<kSortBeside>, kSortBeside, &configured[0]);
  return launch(token_sort<kSortAlone>, kSortAlone, &configured[1]);
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

// Both for few tokens, in one launch.
cudaError_t launch_few(const SortBy& by, const ZeroRows& zero, const void* src, int src_type, int dim, float scale,
                       void* out, int out_type, int accumulate, cudaStream_t stream) {
  SumLayout L = {};
  const SumParams P = sum_params(src, by.tokens, by.vocab, dim, scale, out, accumulate, nullptr, L);
  const int vec = min_vec(vec_of(dim, src, src_type), vec_of(dim, out, out_type));
  const int blocks = static_cast<int>((by.tokens * P.slices + kSumWarps - 1) / kSumWarps);
  const int most = 8 * sm_count();
  const int zeros = zero.table == nullptr ? 0 : static_cast<int>(by.vocab < most ? by.vocab : most);
  return with_type(src_type, [&](auto st) {
    return with_type(out_type, [&](auto ot) {
      return with_vec(vec, [&](auto vc) {
        return mns::launch_pdl(row_sums_few<decltype(st), decltype(ot), decltype(vc)::value>, dim3(blocks + zeros),
                               dim3(32 * kSumWarps), 0, stream, by, zero, blocks, P);
      });
    });
  });
}

cudaError_t launch_row_sums_compact(const void* src, const float* coef, long long tokens, long long vocab, int dim,
                                    float* out, int* slot, uint8_t* ws, const SumLayout& L, cudaStream_t stream) {
  SumParams P = sum_params(src, tokens, vocab, dim, 1.0f, out, 0, ws, L);
  P.coef = coef;
  P.slot = slot;
  if (tokens <= kFewTokens)
    return mns::launch_pdl(row_sums_runs<8>, dim3(static_cast<unsigned>((tokens * P.slices + kSumWarps - 1) / kSumWarps)),
                           dim3(32 * kSumWarps), 0, stream, P);
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
  *bytes = tokens <= kFewTokens || vocab == 0 || dim == 0 ? 0 : sum_layout(tokens, dim).total;
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
  const SumLayout L = sum_layout(tokens, dim);
  if (tokens > kFewTokens) {
    if (!workspace || workspace_bytes < L.total) return MUON_NS_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_NS_ERR_ALIGNMENT;
  }
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  if (tokens == 0) return accumulate ? MUON_NS_OK : status_of(cudaMemsetAsync(dtable, 0, table_bytes, stream));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const SortBy by = {ids, ids_bits == 64 ? 1 : 0, tokens, vocab, -1, 0, nullptr};
  const ZeroRows zero = {accumulate ? nullptr : dtable, static_cast<long long>(dim) * type_size(dtable_type)};
  if (tokens <= kFewTokens)
    return status_of(launch_few(by, zero, dy, dy_type, dim, scale, dtable, dtable_type, accumulate ? 1 : 0, stream));
  const cudaError_t e = launch_sort(by, zero, ws, L, stream);
  if (e != cudaSuccess) return status_of(e);
  return status_of(launch_row_sums(dy, dy_type, tokens, vocab, dim, scale, dtable, dtable_type, accumulate ? 1 : 0, ws,
                                   L, stream));
}

}  // extern "C"
