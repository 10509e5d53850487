// Layer norm, per row: mu = mean(x), var = mean((x - mu)^2),
// r = 1/sqrt(var + eps), y = (x - mu) r w + b.
//
// A group of G threads (a power of two, 8 to 1024) keeps its row in
// registers, kFwdPer elements a thread at most, so x is read once and the
// variance is taken about the mean (no cancellation).  Bound by HBM traffic.
// Many rows go through a grid that stays (the _ring kernel): while a row is
// summed the next one is on its way to shared memory.  Rows too long for the
// registers take the _long kernel, which reads a row again from cache.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "lm/layer_norm.cuh"

namespace mns {
namespace lm {

namespace {

constexpr int kFwdPer = 32;  // elements a thread holds
constexpr int kFwdMax = 1024 * kFwdPer;
constexpr int kFwdRingSmem = 110 * 1024;

// Statistics and output of NR rows of each group, from the thread's units of
// them (rows row .. row + NR - 1, those below `rows`).  Every thread of the CTA
// takes part.
template <typename T, typename TW, int VEC, int G, int NR, typename C = Cols<VEC, G, kFwdPer>>
__device__ __forceinline__ void norm_rows(const Vec<T, C::kU> (&v)[NR][C::kK], const TW* __restrict__ w,
                                          const TW* __restrict__ b, long long row, long long rows, int dim,
                                          float inv_dim, float eps, T* y, float* __restrict__ mean,
                                          float* __restrict__ rstd, float (*red)[NR][32]) {
  const int tid = threadIdx.x & (G - 1);
  float mu[NR], r[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    float2 s = both(0.0f);
#pragma unroll
    for (int k = 0; k < C::kK; ++k)
      if (row + i < rows && C::first(k, tid) < dim) {
        float2 p[C::kP];
        to_pairs<T, C::kU>(v[i][k], p);
#pragma unroll
        for (int j = 0; j < C::kP; ++j) s = add2(s, p[j]);
      }
    mu[i] = s.x + s.y;
  }
  group_sums<G, NR>(mu, red[0]);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    mu[i] *= inv_dim;
    float2 s = both(0.0f);
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      const int c = C::first(k, tid);
      if (row + i < rows && c < dim) {
        float2 p[C::kP];
        to_pairs<T, C::kU>(v[i][k], p);
#pragma unroll
        for (int j = 0; j < C::kP; ++j) {
          float2 d = add2(p[j], both(-mu[i]));
          if (!C::second(c, dim)) d.y = 0.0f;
          s = fma2(d, d, s);
        }
      }
    }
    r[i] = s.x + s.y;
  }
  group_sums<G, NR>(r, red[1]);
#pragma unroll
  for (int i = 0; i < NR; ++i) r[i] = 1.0f / sqrtf(r[i] * inv_dim + eps);
#pragma unroll
  for (int k = 0; k < C::kK; ++k) {
    const int c = C::first(k, tid);
    if (c < dim) {
      float2 wp[C::kP], bp[C::kP];
      to_pairs<TW, C::kU>(C::load(w, c, dim), wp);
      if (b != nullptr) to_pairs<TW, C::kU>(C::load(b, c, dim), bp);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        if (row + i < rows) {
          float2 p[C::kP];
          to_pairs<T, C::kU>(v[i][k], p);
#pragma unroll
          for (int j = 0; j < C::kP; ++j) {
            p[j] = mul2(add2(p[j], both(-mu[i])), both(r[i]));
            p[j] = b != nullptr ? fma2(p[j], wp[j], bp[j]) : mul2(p[j], wp[j]);
          }
          C::store(y + (row + i) * dim, c, dim, p);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    if (tid == 0 && row + i < rows && mean != nullptr) mean[row + i] = mu[i];
    if (tid == 0 && row + i < rows && rstd != nullptr) rstd[row + i] = r[i];
  }
}

template <typename T, typename TW, int VEC, int G>
__global__ void __launch_bounds__(G > kNormCta ? G : kNormCta)
    layer_norm_fwd(const T* x, const TW* __restrict__ w, const TW* __restrict__ b, long long rows, int dim,
                   float inv_dim, float eps, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  using C = Cols<VEC, G, kFwdPer>;
  constexpr int kRows = (G > kNormCta ? G : kNormCta) / G;
  __shared__ float red[2][1][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (G - 1);
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / G;
  Vec<T, C::kU> v[1][C::kK];
#pragma unroll
  for (int k = 0; k < C::kK; ++k) {
    const int c = C::first(k, tid);
    if (row < rows && c < dim) v[0][k] = C::load(x + row * dim, c, dim);
  }
  norm_rows<T, TW, VEC, G, 1>(v, w, b, row, rows, dim, inv_dim, eps, y, mean, rstd, red);
}

// Rows a group takes in a turn of the ring: weight and bias are read once for
// all of them.  (They come from L1, which bounds the kernel with one row a
// turn: 85 % of its throughput at 4096 columns of bf16 with fp32 weights.)
template <typename T>
constexpr int kTurnRows = sizeof(T) == 2 ? 2 : 1;

// A thread copies and reads its own elements, so the copies need no barrier
// (except those by words).
template <typename T, typename TW, int VEC, int G>
__global__ void __launch_bounds__(G > kNormCta ? G : kNormCta, G > kNormCta ? 1 : 2)
    layer_norm_fwd_ring(const T* x, const TW* __restrict__ w, const TW* __restrict__ b, long long rows, int dim,
                        float inv_dim, float eps, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  using C = Cols<VEC, G, kFwdPer>;
  constexpr int NR = kTurnRows<T>;
  constexpr int kRows = (G > kNormCta ? G : kNormCta) / G * NR;
  __shared__ float red[2][NR][32];
  extern __shared__ __align__(16) uint8_t ring[];  // [2 turns][kRows][dim]
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (G - 1), grp = threadIdx.x / G;
  const long long stride = static_cast<long long>(gridDim.x) * kRows;
  constexpr bool kWords = kByWords<T, VEC>;
  const int pitch = kWords ? word_pitch(dim) : dim;
  T* mine = reinterpret_cast<T*>(ring) + grp * NR * pitch;
  auto fetch = [&](int st, long long row) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if (row + i < rows) {
        T* to = mine + (st * kRows + i) * pitch;
        if constexpr (kWords) {
          copy_words<G>(to, x, row + i, rows, dim, tid);
        } else {
#pragma unroll
          for (int k = 0; k < C::kK; ++k) {
            const int c = C::first(k, tid);
            if (c < dim) C::copy(to, x + (row + i) * dim, c, dim);
          }
        }
      }
    }
    copy_commit();
  };
  const long long first = static_cast<long long>(blockIdx.x) * kRows;
  fetch(0, first + grp * NR);
  int st = 0;
  // Every group of the CTA makes the same number of turns (barriers inside).
  for (long long r0 = first; r0 < rows; r0 += stride, st ^= 1) {
    const long long row = r0 + grp * NR;
    fetch(st ^ 1, row + stride);
    copy_wait<1>();
    if (kWords) group_barrier<G>();
    Vec<T, C::kU> v[NR][C::kK];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const T* from = mine + (st * kRows + i) * pitch + (kWords ? row_shift(x + (row + i) * dim) : 0);
#pragma unroll
      for (int k = 0; k < C::kK; ++k) {
        const int c = C::first(k, tid);
        if (row + i < rows && c < dim) v[i][k] = C::template load<true>(from, c, dim);
      }
    }
    // The next turn's copies go to the buffer after this one's other half: all
    // reads of it are behind the barriers of the sums.
    norm_rows<T, TW, VEC, G, NR>(v, w, b, row, rows, dim, inv_dim, eps, y, mean, rstd, red);
  }
  copy_wait<0>();
}

// Rows of more than kFwdMax elements: a CTA a row, three passes over it.
template <typename T, typename TW>
__global__ void __launch_bounds__(1024)
    layer_norm_fwd_long(const T* x, const TW* __restrict__ w, const TW* __restrict__ b, long long rows, int dim,
                        float inv_dim, float eps, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[2][1][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * dim;
    float sum = 0.0f, sq = 0.0f;
    for (int c = threadIdx.x; c < dim; c += 1024) sum += to_f32(xr[c]);
    const float mu = group_sum<1024>(sum, red[0]) * inv_dim;
    for (int c = threadIdx.x; c < dim; c += 1024) {
      const float d = to_f32(xr[c]) - mu;
      sq = fmaf(d, d, sq);
    }
    const float r = 1.0f / sqrtf(group_sum<1024>(sq, red[1]) * inv_dim + eps);
    for (int c = threadIdx.x; c < dim; c += 1024)
      y[row * dim + c] =
          from_f32<T>((to_f32(xr[c]) - mu) * r * to_f32(w[c]) + (b != nullptr ? to_f32(b[c]) : 0.0f));
    if (threadIdx.x == 0 && mean != nullptr) mean[row] = mu;
    if (threadIdx.x == 0 && rstd != nullptr) rstd[row] = r;
  }
}

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" int muon_layer_norm(const void* x, int x_type, const void* weight, const void* bias, int w_type,
                               long long rows, int dim, float eps, void* y, float* mean, float* rstd,
                               cudaStream_t stream) {
  int s = norm_check(rows, dim);
  if (s != MUON_NS_OK) return s;
  if (!type_ok(x_type) || !type_ok(w_type) || !(eps >= 0.0f) || !std::isfinite(eps)) return MUON_NS_ERR_INVALID_ARG;
  if (rows == 0) return MUON_NS_OK;
  if (!x || !weight || !y) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(x, x_type) || !element_aligned(y, x_type) || !element_aligned(weight, w_type) ||
      !element_aligned(bias, w_type) || !element_aligned(mean, MUON_LM_F32) || !element_aligned(rstd, MUON_LM_F32))
    return MUON_NS_ERR_ALIGNMENT;
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  const float inv = 1.0f / static_cast<float>(dim);
  return with_type(x_type, [&](auto xt) {
    return with_type(w_type, [&](auto wt) {
      using T = decltype(xt);
      using TW = decltype(wt);
      const T* xp = static_cast<const T*>(x);
      const TW *wp = static_cast<const TW*>(weight), *bp = static_cast<const TW*>(bias);
      T* yp = static_cast<T*>(y);
      if (dim > kFwdMax) {
        const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
        return status_of(mns::launch_pdl(layer_norm_fwd_long<T, TW>, dim3(grid), dim3(1024), 0, stream, xp, wp, bp,
                                         rows, dim, inv, eps, yp, mean, rstd));
      }
      int vec = min_vec(min_vec(norm_vec(dim, x, x_type), norm_vec(dim, y, x_type)), vec_of(dim, weight, w_type));
      if (bias) vec = min_vec(vec, vec_of(dim, bias, w_type));
      return with_norm_vec<T>(vec, [&](auto vc) {
        // Few rows leave threads to spare: a row takes four times as many, and
        // its loads and sums are that much shorter.
        const bool few = rows <= 2LL * sm_count();
        return with_group(group_of(dim, few ? kFwdPer / 4 : kFwdPer), [&](auto gc) {
          constexpr int V = decltype(vc)::value, G = decltype(gc)::value;
          constexpr int T1 = G > kNormCta ? G : kNormCta;
          const long long grid = (rows + T1 / G - 1) / (T1 / G);
          if constexpr (G <= 512) {
            constexpr int NR = kTurnRows<T>;
            const size_t smem = 2 * sizeof(T) * (T1 / G * NR) * (kByWords<T, V> ? word_pitch(dim) : dim);
            // The staying grid takes over where each of its CTAs has several
            // turns.
            const long long stay = static_cast<long long>(sm_count()) * (T1 > kNormCta ? 1 : 2);
            const bool words = !kByWords<T, V> || (reinterpret_cast<uintptr_t>(x) & 3) == 0;
            if (words && smem <= kFwdRingSmem && grid >= 3 * NR * stay) {
              auto kernel = layer_norm_fwd_ring<T, TW, V, G>;
              static std::atomic<unsigned long long> configured{0};
              const cudaError_t e = allow_smem(kernel, kFwdRingSmem, &configured);
              if (e != cudaSuccess) return status_of(e);
              return status_of(mns::launch_pdl(kernel, dim3(static_cast<unsigned>(stay)), dim3(T1), smem, stream, xp,
                                               wp, bp, rows, dim, inv, eps, yp, mean, rstd));
            }
          }
          return status_of(mns::launch_pdl(layer_norm_fwd<T, TW, V, G>, dim3(static_cast<unsigned>(grid)), dim3(T1), 0,
                                           stream, xp, wp, bp, rows, dim, inv, eps, yp, mean, rstd));
        });
      });
    });
  });
}
