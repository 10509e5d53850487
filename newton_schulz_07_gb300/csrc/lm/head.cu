// The output head's cross entropy and its gradient.  No logits are kept: the
// losses alone need none in memory, the gradient holds bf16 exponentials of one
// piece of the vocabulary.
//
//   z = h W^T, loss_n = log sum_v exp z_nv - z_nt, p = softmax(z),
//   dz_nv = g_n (p_nv - [v = t_n]), dh = dz W, dW = dz^T h.
//
// Every row is referred to its target's logit c_n, one dot product known before
// the large one: with e_nv = exp(z_nv - c_n), s_n the sum of e_nv over v != t and
// e_nt the target's own (1, but where the reference is another),
//   loss_n = log(1 + s_n / e_nt),  dz_nv = g_n e_nv / (s_n + e_nt) for v != t,
//   dz_nt = -g_n s_n / (s_n + e_nt).
// So the large product's epilogue takes exponentials and their sum in one
// pass with no running maximum, and e needs no second pass once s is known:
// g_n / (s_n + e_nt) is a factor of row n of dh, and of row n of h in dW.
//
// The target stays out of s and of the stored e: a token with p near 1 has its
// loss and its target's term, both about 1 - p, to the relative accuracy of the
// logits' differences.  (In the sum, the target's exponential is 1 and the
// difference of two orders of summation: losses down to -6e-4 at dim 4096 and
// logits of 40.)  The target's term is added to dh and dW in fp32.
//
// Only a logit far above the target's (a loss above log kTopSum = 44) can leave
// the range: such rows take their largest logit as reference and the tiles that
// hold them are computed again; the launches that do so leave at once when there
// are none.
//
// Tokens without a loss (target out of range or ignored) are sorted to the
// end and take no part in the products.  The rest is sorted by target, so the
// targets' terms of dW are row sums by sorted token, as in the embedding's
// gradient.
//
// The vocabulary is taken in pieces.  With one piece e (bf16, tokens x piece)
// is held from the first product: 3 products in all.  With more, a first pass
// over the pieces takes only the sums and keeps the last piece's e; the others
// are computed again when their turn comes, into the same buffer.
//
// Bound by the tensor cores for more than about 200 tokens; below that by
// reading W twice and writing dW.
#include <atomic>
#include <cmath>

#include <cudaTypedefs.h>

#include "lm/common.cuh"
#include "lm/embed.cuh"
#include "lm/head_gemm.cuh"

namespace mns {
namespace lm {

namespace {

constexpr float kTopSum = 1.8446744e19f;  // 2^64
// Below it (only where the reference is the largest logit) the target's
// exponential may have lost digits, or be zero.
constexpr float kLeastTarget = 5.421011e-20f;  // 2^-64
constexpr int kHeadPairs = kSms / 2;      // CTA pairs the splits are chosen for
// Pair rows walked together: of e or W as many are read again as there are
// bands.  (8 to 32 for the logits differ by half a percent at 8192 tokens.)
constexpr int kHeadGroup = 8, kLogitsGroup = 16;
constexpr long long kPieceBytes = 1LL << 32;  // e of one piece, at most, by default

constexpr int kSplitTiles = 16 * kHeadPairs;  // tiles of all splits of dh, at most

// Splits of the vocabulary in dh, by all threads of a CTA: output tiles alone
// may be too few for the pairs, or fill their last turn badly (256 tiles on 76
// pairs take 4 turns for 3.4; in two halves 7 for 6.7).  A turn costs its
// k-blocks and an epilogue worth about 6 of them; the fewest splits of least
// cost are taken, of 8 k-blocks each at least.
__device__ __forceinline__ int choose_splits(long long all_tiles, int kb) {
  __shared__ unsigned int best_sh[32];
  if (all_tiles >= kSplitTiles) return 1;
  const int tiles = static_cast<int>(all_tiles);
  // Cost and splits in one word (costs past 2^20 blocks are all the same).
  unsigned int best = ~0u;
  for (int s = threadIdx.x + 1; s * tiles <= kSplitTiles && (s == 1 || kb / s >= 8); s += blockDim.x) {
    const int turns = (tiles * s + kHeadPairs - 1) / kHeadPairs;
    const int cost = turns * ((kb + s - 1) / s + 6);
    const unsigned int c = (static_cast<unsigned int>(cost < (1 << 20) ? cost : (1 << 20) - 1) << 11) | s;
    best = c < best ? c : best;
  }
  best = __reduce_min_sync(0xFFFFFFFFu, best);
  if ((threadIdx.x & 31) == 0) best_sh[threadIdx.x >> 5] = best;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) best = best_sh[w] < best ? best_sh[w] : best;
  return static_cast<int>(best & 2047u);
}

struct HeadRows {
  const unsigned long long* sorted;  // key << 32 | token, live tokens first
  const void* targets;
  int ids64;
  long long tokens, vocab;
  int dim;
  int* ctl;
  int* redo;   // per pair row
  int* col;    // target
  float* zt;   // its logit
  float* ref;  // reference of the exponentials
  float* scale;  // g / (s + e_t)
  float* coef;   // -g s / (s + e_t)
};

// Clears the control words and chooses dh's splits: one CTA, all threads.
__device__ __forceinline__ void start_call(const HeadRows& R, int count, int pair_rows, int split_kb) {
  for (int i = threadIdx.x; i < pair_rows; i += blockDim.x) R.redo[i] = 0;
  const int splits =
      choose_splits(static_cast<long long>(token_pairs(count)) * ((R.dim + kHeadRows - 1) / kHeadRows), split_kb);
  if (threadIdx.x == 0) {
    R.ctl[kCtlErr] = 0;
    R.ctl[kCtlRedo] = 0;
    R.ctl[kCtlSplits] = splits;
  }
}

// Row p of the compact copy of h, its target and the target's logit: one warp.
__device__ __forceinline__ void start_row(const HeadRows& R, const bf16* __restrict__ h, const bf16* __restrict__ W,
                                          bf16* __restrict__ hc, long long p, long long token) {
  const int lane = threadIdx.x & 31;
  const long long t = load_id(R.targets, R.ids64, token, R.vocab);
  const bf16* hr = h + token * R.dim;
  const bf16* wr = W + t * R.dim;
  bf16* out = hc + p * R.dim;
  float a[8] = {};
#pragma unroll 4
  for (int c = lane * 8; c < R.dim; c += 256) {
    const Vec<bf16, 8> x = load_vec<bf16, 8>(hr + c), w = load_vec<bf16, 8>(wr + c);
    *reinterpret_cast<Vec<bf16, 8>*>(out + c) = x;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = fmaf(to_f32(x.v[j]), to_f32(w.v[j]), a[j]);
  }
  const float z = warp_sum(((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7])));
  if (lane == 0) {
    R.col[p] = static_cast<int>(t);
    R.zt[p] = z;
    R.ref[p] = z;
  }
}

// Up to kRankTokens tokens: a CTA ranks 32 and starts their rows; the last one
// counts the live tokens and chooses the splits.
__global__ void __launch_bounds__(1024)
    head_rank(const SortBy by, const HeadRows R, const bf16* __restrict__ h, const bf16* __restrict__ W,
              bf16* __restrict__ hc, int pair_rows, int split_kb, unsigned long long* __restrict__ sorted) {
  extern __shared__ __align__(16) unsigned int keys[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (blockIdx.x == gridDim.x - 1) {
    const int count = count_live(by);
    if (threadIdx.x == 0) R.ctl[kCtlCount] = count;
    start_call(R, count, pair_rows, split_kb);
    return;
  }
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kRankBlock + (threadIdx.x >> 5);
  if (t < by.tokens) {
    // The rows are on their way to L2 while the tokens are ranked.
    const long long id = load_id(by.ids, by.ids64, t, by.vocab);
    if (id >= 0 && id != by.skip)
      for (int c = lane * 64; c < R.dim; c += 2048) {
        prefetch_l2(h + t * R.dim + c);
        prefetch_l2(W + id * R.dim + c);
      }
  }
  unsigned int key;
  const int p = rank_tokens(by, blockIdx.x, keys, &key);
  if (t < by.tokens) {
    if (lane == 0) sorted[p] = (static_cast<unsigned long long>(key) << 32) | t;
    if (key < none_of(by)) start_row(R, h, W, hc, p, t);
  }
}

// More tokens, after their sort.
__global__ void __launch_bounds__(256)
    head_start(const HeadRows R, const bf16* __restrict__ h, const bf16* __restrict__ W, bf16* __restrict__ hc,
               int pair_rows, int split_kb) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int count = R.ctl[kCtlCount];
  if (blockIdx.x == 0) start_call(R, count, pair_rows, split_kb);
  const long long p = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (p < count) start_row(R, h, W, hc, p, static_cast<unsigned int>(R.sorted[p]));
}

// A call whose waits ran out answers with NaN alone: the error word lies in a
// workspace that the caller may not hold.
constexpr uint32_t kNanWord = 0x7FFF7FFFu;  // of fp32 and of bf16 alike

struct HeadFinish {
  const float2* stat;
  int halves;  // statistics a row
  int again;   // second pass: the rows of tiles that were computed again
  const float* dloss;  // per token, or null: 1 / count
  float* loss;         // per token
  // gradient
  const bf16* hc;
  bf16* hs;   // scale h, rows up to a multiple of 64 zero
};

// A CTA a sorted position: joins the row's sums in a fixed order, and from
// them the loss, the factors of the gradient and the scaled row of h.
__global__ void __launch_bounds__(128) head_finish(const HeadRows R, const HeadFinish F) {
  __shared__ float red[2][4];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  if (F.again) {
    const int4 ctl = *reinterpret_cast<const int4*>(R.ctl);
    static_assert(kCtlErr == 0 && kCtlRedo == 3, "control words");
    if (ctl.x != 0)
      for (long long i = blockIdx.x * 128LL + threadIdx.x; i < R.tokens; i += gridDim.x * 128LL)
        F.loss[i] = __uint_as_float(kNanWord);
    if (ctl.x != 0 || ctl.w == 0) return;
  }
  const int count = R.ctl[kCtlCount];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (long long p = blockIdx.x; p < R.tokens; p += gridDim.x) {
    const unsigned int token = static_cast<unsigned int>(R.sorted[p]);
    if (p >= count) {
      if (F.again) continue;
      if (tid == 0) F.loss[token] = 0.0f;
      // dW's last k-block reads rows up to a multiple of 64.
      if (F.hs != nullptr && p < (count > 0 ? (count + 63) / 64 * 64 : 64))
        for (int c = tid * 8; c < R.dim; c += 1024)
          *reinterpret_cast<uint4*>(F.hs + p * R.dim + c) = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    if (F.again && R.redo[p / kHeadRows] == 0) continue;
    // Loaded before the sums are joined; all independent of one another.
    const float zt = R.zt[p], c = R.ref[p];
    const float g = F.hs == nullptr ? 0.0f : F.dloss != nullptr ? F.dloss[token] : 1.0f / static_cast<float>(count);
    const bool one = F.hs != nullptr && R.dim <= 1024;  // a vector a thread
    Vec<bf16, 8> x = {};
    if (one && tid * 8 < R.dim) x = load_vec<bf16, 8>(F.hc + p * R.dim + tid * 8);
    const float2* st = F.stat + p * F.halves;
    float mx = -INFINITY, s = 0.0f;
#pragma unroll 4
    for (int i = tid; i < F.halves; i += 128) {
      const float2 v = st[i];
      mx = fmaxf(mx, v.x);
      s += v.y;
    }
    s = warp_sum(s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    __syncthreads();  // the last row's sums have been read
    if (lane == 0) {
      red[0][warp] = s;
      red[1][warp] = mx;
    }
    __syncthreads();
    s = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
    mx = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
    // The target's exponential, as the epilogue takes the others'.
    const float et = exp2_approx(fmaf(zt, kLog2e, -(c * kLog2e)));
    if (!F.again && !(s <= kTopSum)) {  // out of range, or not a number
      if (tid == 0) {
        R.ref[p] = mx;
        R.redo[p / kHeadRows] = 1;
        R.ctl[kCtlRedo] = 1;
      }
      continue;
    }
    const auto put_loss = [&] {
      if (tid == 0) F.loss[token] = et >= kLeastTarget ? log1pf(s / et) : logf(s + et) + (c - zt);
    };
    if (F.hs == nullptr) {
      put_loss();
      continue;
    }
    const float f = g / (s + et);
    // hs is the MMAs' bf16 operand: one more rounding, up to 2^-8, in each term of
    // dW but the targets', which are added in fp32.
    for (int col = tid * 8; col < R.dim; col += 1024) {
      if (!one) x = load_vec<bf16, 8>(F.hc + p * R.dim + col);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = f * to_f32(x.v[j]);
      store_vec<bf16, 8>(F.hs + p * R.dim + col, o);
    }
    if (tid == 0) {
      R.scale[p] = f;
      R.coef[p] = -g * (s / (s + et));
    }
    put_loss();
  }
}

// dh[token] = scale (sum of the splits, in order) + coef W[target].  An item is
// a row and 256 of its columns.  With many items a warp takes one; with few
// (SHARED), where splits are many, a CTA's warps share one, a contiguous part of
// the splits each.
//
// The gradient's last kernel: where a wait ran out, dh becomes NaN here, and
// loss and dW (dW_vecs 16-byte words) by one CTA more, which else does nothing.
// (CTAs an SM: with the registers of 3 in place of 5, 8192 x 2048 took 47 us for
// 39, 36 in this form.)
template <bool SHARED>
__global__ void __launch_bounds__(256, SHARED ? 4 : 5)
    head_join_dh(const HeadRows R, const float* __restrict__ part, const bf16* __restrict__ W, bf16* __restrict__ dh,
                 int slices, float* __restrict__ loss, uint4* __restrict__ dW, long long dW_vecs) {
  __shared__ float red[SHARED ? 8 : 1][256];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int4 ctl = *reinterpret_cast<const int4*>(R.ctl);
  static_assert(kCtlErr == 0 && kCtlCount == 1 && kCtlSplits == 2, "control words");
  if (blockIdx.x == gridDim.x - 1) {
    if (ctl.x == 0) return;
#pragma unroll 1
    for (long long i = threadIdx.x; i < R.tokens; i += 256) loss[i] = __uint_as_float(kNanWord);
#pragma unroll 1
    for (long long i = threadIdx.x; i < dW_vecs; i += 256) dW[i] = make_uint4(kNanWord, kNanWord, kNanWord, kNanWord);
    return;
  }
  const int count = ctl.y, splits = ctl.z;
  const long long rows = static_cast<long long>(token_pairs(count)) * kHeadRows;
  const long long items = R.tokens * slices;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto add = [&](long long p, int c, int s0, int s1, float (&o)[8]) {
#pragma unroll 8
    for (int s = s0; s < s1; ++s) {
      const Vec<float, 8> v = load_global<float, 8>(part + (s * rows + p) * R.dim + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += v.v[j];
    }
  };
  const long long i = SHARED ? blockIdx.x : static_cast<long long>(blockIdx.x) * 8 + warp;
  if (i >= items) return;
  const long long p = i / slices;
  const int c = static_cast<int>(i - p * slices) * 256 + lane * 8;
  const bool live = p < count && c < R.dim;
  const unsigned int token = static_cast<unsigned int>(R.sorted[p]);
  Vec<bf16, 8> w = {};
  float f = 0.0f, k = 0.0f;
  auto target = [&] {
    if (!live) return;
    w = load_vec<bf16, 8>(W + load_id(R.targets, R.ids64, token, R.vocab) * R.dim + c);
    f = R.scale[p];
    k = R.coef[p];
  };
  // With few items the target's row is asked for before the splits are added;
  // with many other warps hide it, and early loads cost more than they give
  // (8192 x 2048: 39 us against 55).
  if (SHARED && warp == 0) target();
  float o[8] = {};
  if (live) add(p, c, SHARED ? splits * warp / 8 : 0, SHARED ? splits * (warp + 1) / 8 : splits, o);
  if (SHARED) {
#pragma unroll
    for (int j = 0; j < 8; ++j) red[warp][j * 32 + lane] = o[j];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int g = 1; g < 8; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += red[g][j * 32 + lane];
  }
  if (c >= R.dim) return;
  if (!SHARED) target();
  float out[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    out[j] = ctl.x != 0 ? __uint_as_float(kNanWord) : live ? fmaf(f, o[j], k * to_f32(w.v[j])) : 0.0f;
  store_vec<bf16, 8>(dh + static_cast<long long>(token) * R.dim + c, out);
}

// -------------------------------------------------------------------- host --

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct HeadLayout {
  size_t redo, col, zt, ref, scale, coef, stat, sums, slot, hc, hs, addend, e, part, total;
  SumLayout sum;
  long long piece, pieces, lde, part_rows;
  int halves;
};

int check(long long tokens, long long vocab, int dim, int bits) {
  if (tokens < 0 || vocab < 0 || dim <= 0 || tokens > kMaxRows || vocab > kMaxRows || dim > kMaxDim)
    return MUON_NS_ERR_INVALID_ARG;
  if (bits != 32 && bits != 64) return MUON_NS_ERR_INVALID_ARG;
  if (dim % 8 != 0) return MUON_NS_ERR_ALIGNMENT;
  return MUON_NS_OK;
}

HeadLayout head_layout(long long tokens, long long vocab, int dim, bool grad, int pieces) {
  HeadLayout L = {};
  const long long pair_rows = (tokens + kHeadRows - 1) / kHeadRows;
  // Pieces of whole column tiles.
  long long n = grad ? pieces : 1;
  if (n <= 0) n = (2 * tokens * vocab + kPieceBytes - 1) / kPieceBytes;
  const long long tiles = vocab > 0 ? (vocab + kHeadRows - 1) / kHeadRows : 1;
  if (n > tiles) n = tiles;
  if (n < 1) n = 1;
  L.piece = (tiles + n - 1) / n * kHeadRows;
  L.pieces = (vocab + L.piece - 1) / L.piece;
  L.lde = L.piece;
  L.halves = static_cast<int>((vocab + kHeadHalf - 1) / kHeadHalf);
  size_t off = sizeof(int) * kCtlWords;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const size_t n_tok = static_cast<size_t>(tokens);
  L.redo = take(4 * static_cast<size_t>(pair_rows));
  L.col = take(4 * n_tok);
  L.zt = take(4 * n_tok);
  L.ref = take(4 * n_tok);
  L.scale = take(4 * n_tok);
  L.coef = take(4 * n_tok);
  L.stat = take(8 * n_tok * L.halves);
  L.sum = sum_layout(tokens, grad ? dim : 0);
  L.sums = take(L.sum.total);
  L.hc = take(2 * n_tok * dim);
  if (grad) {
    L.slot = take(4 * static_cast<size_t>(vocab));
    L.hs = take(2 * n_tok * dim);
    L.addend = take(4 * n_tok * dim);
    L.e = take(2 * n_tok * static_cast<size_t>(L.lde));
    // Rows of the splits: choose_splits takes one, or as many as make at most
    // kSplitTiles tiles.
    const long long tn = (dim + kHeadRows - 1) / kHeadRows;
    long long rows = kSplitTiles / tn;
    if (rows < pair_rows) rows = pair_rows;
    L.part_rows = rows * kHeadRows;
    L.part = take(4 * static_cast<size_t>(L.part_rows) * dim);
  }
  L.total = off;
  return L;
}

// Map over rows x inner elements with a row stride of ld elements.
bool map2d(CUtensorMap* map, const void* base, long long inner, long long rows, long long ld, int box_inner,
           int box_rows, bool f32 = false) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(mns::tensor_map_encoder());
  if (!fn) return false;
  const cuuint64_t eb = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows), 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * eb, static_cast<cuuint64_t>(ld) * eb * rows};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch_gemm(const HeadGemm& P, long long units, cudaStream_t stream) {
  if (units >= (1LL << 30)) return cudaErrorInvalidValue;  // 32-bit tile numbers in the kernel
  static std::atomic<int> resident[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int most = resident[dev & 63].load();
  if (most == 0) {
    e = cudaFuncSetAttribute(head_gemm<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeadSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kHeadThreads);
    cfg.dynamicSmemBytes = kHeadSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&most, head_gemm<MODE>, &cfg);
    if (e != cudaSuccess) return e;
    if (most < 1) return cudaErrorInvalidConfiguration;
    resident[dev & 63].store(most);
  }
  const unsigned n = static_cast<unsigned>(units < most ? units : most);
  return mns::launch_pdl_cluster(head_gemm<MODE>, dim3(2 * n), dim3(kHeadThreads), kHeadSmem, stream, 2, P);
}

struct HeadCall {
  const bf16 *h, *W;
  long long tokens, vocab;
  int dim;
  const void* targets;
  int ids64;
  long long skip;
  const float* dloss;
  float* loss;
  bf16* dh;
  void* dW;
  int dW_f32, accumulate;
  uint8_t* ws;
  cudaStream_t stream;
};

#define MNS_TRY(x)                                    \
  do {                                                \
    const cudaError_t mns_e = (x);                    \
    if (mns_e != cudaSuccess) return status_of(mns_e); \
  } while (0)

int run_head(const HeadCall& C, const HeadLayout& L) {
  const bool grad = C.dh != nullptr;
  uint8_t* ws = C.ws;
  const long long N = C.tokens, V = C.vocab;
  const int D = C.dim;
  const long long pair_rows = (N + kHeadRows - 1) / kHeadRows, dim_tiles = (D + kHeadRows - 1) / kHeadRows;
  auto at = [&](size_t off) { return ws + off; };
  auto f32_at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  HeadRows R = {};
  R.sorted = reinterpret_cast<const unsigned long long*>(at(L.sums + L.sum.sorted));
  R.targets = C.targets;
  R.ids64 = C.ids64;
  R.tokens = N;
  R.vocab = V;
  R.dim = D;
  R.ctl = reinterpret_cast<int*>(ws);
  R.redo = reinterpret_cast<int*>(at(L.redo));
  R.col = reinterpret_cast<int*>(at(L.col));
  R.zt = f32_at(L.zt);
  R.ref = f32_at(L.ref);
  R.scale = f32_at(L.scale);
  R.coef = f32_at(L.coef);
  bf16* hc = reinterpret_cast<bf16*>(at(L.hc));
  bf16* hs = reinterpret_cast<bf16*>(at(L.hs));
  bf16* e = reinterpret_cast<bf16*>(at(L.e));

  auto width = [&](long long j) { return V - j * L.piece < L.piece ? V - j * L.piece : L.piece; };
  // Splits are the same for every piece: chosen for the shortest.
  const int split_kb = static_cast<int>((width(L.pieces - 1) + kBlockK - 1) / kBlockK);
  // The losses alone need no order among the live tokens.
  const SortBy by = {C.targets, C.ids64, N, V, C.skip, grad ? 0 : 1, R.ctl + kCtlCount};
  if (N <= kRankTokens) {
    MNS_TRY(mns::launch_pdl(head_rank, dim3(static_cast<unsigned>((N + kRankBlock - 1) / kRankBlock + 1)), dim3(1024),
                            kRankSmem, C.stream, by, R, C.h, C.W, hc, static_cast<int>(pair_rows), split_kb,
                            reinterpret_cast<unsigned long long*>(at(L.sums + L.sum.sorted))));
  } else {
    MNS_TRY(launch_sort(by, ZeroRows{nullptr, 0}, at(L.sums), L.sum, C.stream));
    MNS_TRY(mns::launch_pdl(head_start, dim3(static_cast<unsigned>((N + 7) / 8)), dim3(256), 0, C.stream, R, C.h, C.W,
                            hc, static_cast<int>(pair_rows), split_kb));
  }

  HeadGemm G = {};
  G.ctl = R.ctl;
  G.dim = D;
  G.group = kHeadGroup;
  G.budget = mns::wait_budget();
  auto logits = [&](long long j, bool stats, bool store, const int* redo) -> int {
    HeadGemm P = G;
    P.vp = static_cast<int>(width(j));
    P.group = kLogitsGroup;
    P.ref = R.ref;
    P.target = R.col;
    P.v0 = j * L.piece;
    P.stat = stats ? reinterpret_cast<float2*>(at(L.stat)) : nullptr;
    P.stat_ld = L.halves;
    P.stat0 = static_cast<int>(j * L.piece / kHeadHalf);
    P.store = store ? 1 : 0;
    P.redo = redo;
    if (!map2d(&P.tmA, hc, D, N, D, kBlockK, kTileM) ||
        !map2d(&P.tmB, C.W + j * L.piece * D, D, P.vp, D, kBlockK, kTileN / 2))
      return MUON_NS_ERR_CUDA;
    P.out = e;
    P.ld = L.lde;
    P.rows = static_cast<int>(N);
    return status_of(launch_gemm<kLogits>(P, pair_rows * ((P.vp + kHeadRows - 1) / kHeadRows), C.stream));
  };
  const long long kept = L.pieces - 1;  // piece whose e the first pass leaves
  HeadFinish F = {};
  F.stat = reinterpret_cast<const float2*>(at(L.stat));
  F.halves = L.halves;
  F.dloss = C.dloss;
  F.loss = C.loss;
  if (grad) {
    F.hc = hc;
    F.hs = hs;
  }
  for (int again = 0; again < 2; ++again) {
    for (long long j = 0; j < L.pieces; ++j) {
      const int s = logits(j, true, grad && j == kept, again ? R.redo : nullptr);
      if (s != MUON_NS_OK) return s;
    }
    F.again = again;
    // (The second pass mostly has nothing to do: CTAs that start at once.)
    const long long most = static_cast<long long>(sm_count()) * (again ? 4 : 16);
    const unsigned finish_grid = static_cast<unsigned>(N < most ? N : most);
    MNS_TRY(mns::launch_pdl(head_finish, dim3(finish_grid), dim3(128), 0, C.stream, R, F));
  }
  if (!grad) return MUON_NS_OK;

  float* addend = f32_at(L.addend);
  int* slot = reinterpret_cast<int*>(at(L.slot));
  MNS_TRY(launch_row_sums_compact(C.h, R.coef, N, V, D, addend, slot, at(L.sums), L.sum, C.stream));
  for (long long i = 0; i < L.pieces; ++i) {
    const long long j = i == 0 ? kept : i - 1;
    const long long v0 = j * L.piece;
    const int vp = static_cast<int>(width(j));
    if (i > 0) {
      const int s = logits(j, false, true, nullptr);
      if (s != MUON_NS_OK) return s;
    }
    HeadGemm P = G;
    P.vp = vp;
    P.add = i > 0 ? 1 : 0;
    if (!map2d(&P.tmA, e, vp, N, L.lde, kBlockK, kTileM) || !map2d(&P.tmB, C.W + v0 * D, D, vp, D, 64, kBlockK) ||
        !map2d(&P.tmOut, at(L.part), D, L.part_rows, D, 32, 32, true))
      return MUON_NS_ERR_CUDA;
    const long long most = pair_rows * dim_tiles > kSplitTiles ? pair_rows * dim_tiles : kSplitTiles;
    MNS_TRY(launch_gemm<kDh>(P, most, C.stream));
    P = G;
    P.vp = vp;
    P.add = C.accumulate;
    P.addend = addend;
    P.slot = slot;
    P.sorted = R.sorted;
    P.v0 = v0;
    void* dst = static_cast<uint8_t*>(C.dW) + static_cast<size_t>(v0) * D * (C.dW_f32 ? 4 : 2);
    if (!map2d(&P.tmA, e, vp, N, L.lde, 64, kBlockK) || !map2d(&P.tmB, hs, D, N, D, 64, kBlockK) ||
        (C.dW_f32 && !map2d(&P.tmOut, dst, D, vp, D, 32, 32, true)))
      return MUON_NS_ERR_CUDA;
    P.out = dst;
    P.ld = D;
    P.rows = vp;
    P.sectors = D % 16 == 0 && aligned(dst, 32) ? 1 : 0;
    const long long units = static_cast<long long>((vp + kHeadRows - 1) / kHeadRows) * dim_tiles;
    MNS_TRY(C.dW_f32 ? launch_gemm<kDwF32>(P, units, C.stream) : launch_gemm<kDwBf16>(P, units, C.stream));
  }
  const int slices = static_cast<int>((D + 255) / 256);
  const long long items = N * slices;
  const bool shared = items <= 16LL * sm_count();
  MNS_TRY(mns::launch_pdl(shared ? head_join_dh<true> : head_join_dh<false>,
                          dim3(static_cast<unsigned>((shared ? items : (items + 7) / 8) + 1)), dim3(256), 0, C.stream, R,
                          static_cast<const float*>(f32_at(L.part)), C.W, C.dh, slices, C.loss,
                          static_cast<uint4*>(C.dW), V * D / (C.dW_f32 ? 4 : 8)));
  return MUON_NS_OK;
}

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_head_workspace_size(long long tokens, long long vocab, int dim, int grad, int pieces, size_t* bytes) {
  const int s = check(tokens, vocab, dim, 32);
  if (s != MUON_NS_OK) return s;
  if (!bytes || pieces < 0) return MUON_NS_ERR_INVALID_ARG;
  *bytes = tokens == 0 || vocab == 0 ? 0 : head_layout(tokens, vocab, dim, grad != 0, pieces).total;
  return MUON_NS_OK;
}

int muon_head_loss(const muon_bf16* h, const muon_bf16* W, long long tokens, long long vocab, int dim,
                   const void* targets, int target_bits, long long ignore_index, float* loss, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream) {
  int s = check(tokens, vocab, dim, target_bits);
  if (s != MUON_NS_OK) return s;
  if (tokens == 0) return MUON_NS_OK;
  if (!h || !targets || !loss || (vocab > 0 && !W)) return MUON_NS_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(loss, 4) || !aligned(targets, target_bits / 8))
    return MUON_NS_ERR_ALIGNMENT;
  const HeadLayout L = head_layout(tokens, vocab, dim, false, 1);
  if (vocab > 0) {
    if (!workspace || workspace_bytes < L.total) return MUON_NS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MUON_NS_ERR_ALIGNMENT;
  }
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  if (vocab == 0) return status_of(cudaMemsetAsync(loss, 0, sizeof(float) * tokens, stream));
  HeadCall C = {};
  C.h = h;
  C.W = W;
  C.tokens = tokens;
  C.vocab = vocab;
  C.dim = dim;
  C.targets = targets;
  C.ids64 = target_bits == 64 ? 1 : 0;
  C.skip = ignore_index;
  C.loss = loss;
  C.ws = static_cast<uint8_t*>(workspace);
  C.stream = stream;
  return run_head(C, L);
}

int muon_head_loss_grad(const muon_bf16* h, const muon_bf16* W, long long tokens, long long vocab, int dim,
                        const void* targets, int target_bits, long long ignore_index, const float* dloss, int pieces,
                        float* loss, muon_bf16* dh, void* dW, int dW_type, int accumulate, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  int s = check(tokens, vocab, dim, target_bits);
  if (s != MUON_NS_OK) return s;
  if (pieces < 0 || !type_ok(dW_type)) return MUON_NS_ERR_INVALID_ARG;
  if (accumulate && dW_type != MUON_LM_F32) return MUON_NS_ERR_INVALID_ARG;
  if (tokens > 0 && (!h || !targets || !loss || !dh)) return MUON_NS_ERR_INVALID_ARG;
  if (vocab > 0 && (!dW || (tokens > 0 && !W))) return MUON_NS_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(dh, 16) || !aligned(dW, 16) || !aligned(loss, 4) ||
      !aligned(dloss, 4) || !aligned(targets, target_bits / 8))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t hb = 2 * static_cast<size_t>(tokens) * dim, wb = 2 * static_cast<size_t>(vocab) * dim;
  const size_t db = static_cast<size_t>(vocab) * dim * type_size(dW_type);
  if (overlap(dh, hb, h, hb) || overlap(dh, hb, W, wb) || overlap(dW, db, h, hb) || overlap(dW, db, W, wb) ||
      overlap(dh, hb, dW, db))
    return MUON_NS_ERR_INVALID_ARG;
  const HeadLayout L = head_layout(tokens, vocab, dim, true, pieces);
  if (tokens > 0 && vocab > 0) {
    if (!workspace || workspace_bytes < L.total) return MUON_NS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MUON_NS_ERR_ALIGNMENT;
  }
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  if (tokens == 0 || vocab == 0) {
    cudaError_t e = cudaSuccess;
    if (tokens > 0) e = cudaMemsetAsync(loss, 0, sizeof(float) * tokens, stream);
    if (e == cudaSuccess && tokens > 0) e = cudaMemsetAsync(dh, 0, hb, stream);
    if (e == cudaSuccess && vocab > 0 && !accumulate) e = cudaMemsetAsync(dW, 0, db, stream);
    return status_of(e);
  }
  HeadCall C = {};
  C.h = h;
  C.W = W;
  C.tokens = tokens;
  C.vocab = vocab;
  C.dim = dim;
  C.targets = targets;
  C.ids64 = target_bits == 64 ? 1 : 0;
  C.skip = ignore_index;
  C.dloss = dloss;
  C.loss = loss;
  C.dh = dh;
  C.dW = dW;
  C.dW_f32 = dW_type == MUON_LM_F32 ? 1 : 0;
  C.accumulate = accumulate ? 1 : 0;
  C.ws = static_cast<uint8_t*>(workspace);
  C.stream = stream;
  return run_head(C, L);
}

}  // extern "C"
