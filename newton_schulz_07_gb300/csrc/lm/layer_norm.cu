// Layer norm and its gradient.
//
// Forward, per row: mu = mean(x), var = mean((x - mu)^2), r = 1/sqrt(var + eps),
// y = (x - mu) r w + b.  A group of G threads (a power of two, 32 to 1024)
// keeps its row in registers, kFwdPer elements a thread at most, so x is read
// once and the variance is taken about the mean (no cancellation).
//
// Backward, per row, with xh = (x - mu) r and a = dy w:
//   dx = r (a - mean(a) - xh mean(a xh)),
// and over the rows dw = sum dy xh, db = sum dy.  A CTA walks the rows with
// the grid's stride and holds its columns' dw and db in registers, so x and
// dy are read once; at its end it stores one partial row of each, and a second
// kernel adds the partials of a column in a fixed order.
//
// Both are bound by HBM traffic.  Rows too long for the registers take the
// _long kernels, which read a row again from cache.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "lm/common.cuh"

namespace mns {
namespace lm {

namespace {

constexpr int kFwdPer = 32;   // elements a thread holds, forward
constexpr int kBwdPer = 16;   // and backward (x, dy, dw and db)
constexpr int kThreads = 256; // CTA size for groups up to it
constexpr int kFwdMax = 1024 * kFwdPer;
constexpr int kBwdMax = 1024 * kBwdPer;

// Sum of v over the G threads of a group, the same value in each.  `red` holds
// one float per warp of the CTA; callers alternate between two of them, so one
// barrier a sum is enough.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* red) {
  v = warp_sum(v);
  if (G == 32) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  constexpr int kW = G / 32;
  const int first = warp / kW * kW;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kW; ++w) s += red[first + w];
  return s;
}

template <typename T, typename TW, int VEC, int G>
__global__ void __launch_bounds__(G > kThreads ? G : kThreads)
    layer_norm_fwd(const T* x, const TW* __restrict__ w, const TW* __restrict__ b, long long rows,
                   int dim, float inv_dim, float eps, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int kRows = (G > kThreads ? G : kThreads) / G;
  constexpr int kK = kFwdPer / VEC;
  __shared__ float red[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (G - 1);
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / G;
  const bool live = row < rows;
  const T* xr = x + (live ? row : 0) * dim;
  Vec<T, VEC> v[kK];
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = (k * G + tid) * VEC;
    if (live && c < dim) v[k] = load_vec<T, VEC>(xr + c);
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = (k * G + tid) * VEC;
    if (live && c < dim) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum += to_f32(v[k].v[j]);
    }
  }
  const float mu = group_sum<G>(sum, red[0]) * inv_dim;
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = (k * G + tid) * VEC;
    if (live && c < dim) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = to_f32(v[k].v[j]) - mu;
        sq = fmaf(d, d, sq);
      }
    }
  }
  const float r = 1.0f / sqrtf(group_sum<G>(sq, red[1]) * inv_dim + eps);
  if (!live) return;
  T* yr = y + row * dim;
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = (k * G + tid) * VEC;
    if (c < dim) {
      const Vec<TW, VEC> wv = load_vec<TW, VEC>(w + c);
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = (to_f32(v[k].v[j]) - mu) * r * to_f32(wv.v[j]);
      if (b != nullptr) {
        const Vec<TW, VEC> bv = load_vec<TW, VEC>(b + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += to_f32(bv.v[j]);
      }
      store_vec<T, VEC>(yr + c, o);
    }
  }
  if (tid == 0 && mean != nullptr) mean[row] = mu;
  if (tid == 0 && rstd != nullptr) rstd[row] = r;
}

// Rows of more than kFwdMax elements: a CTA a row, three passes over it.
template <typename T, typename TW>
__global__ void __launch_bounds__(1024)
    layer_norm_fwd_long(const T* x, const TW* __restrict__ w, const TW* __restrict__ b, long long rows, int dim,
                        float inv_dim, float eps, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[2][32];
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

// part: fp32 [gridDim.x][2][dim], this CTA's dw and db.
template <typename T, typename TW, int VEC, int G>
__global__ void __launch_bounds__(G > kThreads ? G : kThreads)
    layer_norm_bwd(const T* dy, const T* x, const TW* __restrict__ w, const float* __restrict__ mean,
                   const float* __restrict__ rstd, long long rows, int dim, float inv_dim, T* dx,
                   float* __restrict__ part) {
  constexpr int kRows = (G > kThreads ? G : kThreads) / G;
  constexpr int kK = kBwdPer / VEC;
  __shared__ float red[2][2][32];
  extern __shared__ float acc[];  // [kRows][2][dim], only with kRows > 1
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (G - 1), grp = threadIdx.x / G;
  float dw[kK][VEC] = {}, db[kK][VEC] = {};
  const long long stride = static_cast<long long>(gridDim.x) * kRows;
  int buf = 0;
  // Every group of the CTA makes the same number of turns (barriers inside).
  for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < rows; r0 += stride, buf ^= 1) {
    const long long row = r0 + grp;
    const bool live = row < rows;
    Vec<T, VEC> xv[kK], gv[kK];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = (k * G + tid) * VEC;
      if (live && c < dim) {
        xv[k] = load_vec<T, VEC>(x + row * dim + c);
        gv[k] = load_vec<T, VEC>(dy + row * dim + c);
      }
    }
    const float mu = live ? mean[row] : 0.0f, r = live ? rstd[row] : 0.0f;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = (k * G + tid) * VEC;
      if (live && c < dim) {
        const Vec<TW, VEC> wv = load_vec<TW, VEC>(w + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float g = to_f32(gv[k].v[j]), xh = (to_f32(xv[k].v[j]) - mu) * r;
          const float a = g * to_f32(wv.v[j]);
          dw[k][j] = fmaf(g, xh, dw[k][j]);
          db[k][j] += g;
          s1 += a;
          s2 = fmaf(a, xh, s2);
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (G > 32) {
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) {
        red[buf][0][warp] = s1;
        red[buf][1][warp] = s2;
      }
      __syncthreads();
      constexpr int kW = G / 32;
      const int first = warp / kW * kW;
      s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        s1 += red[buf][0][first + i];
        s2 += red[buf][1][first + i];
      }
    }
    const float m1 = s1 * inv_dim, m2 = s2 * inv_dim;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = (k * G + tid) * VEC;
      if (live && c < dim) {
        const Vec<TW, VEC> wv = load_vec<TW, VEC>(w + c);
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float g = to_f32(gv[k].v[j]), xh = (to_f32(xv[k].v[j]) - mu) * r;
          o[j] = r * (g * to_f32(wv.v[j]) - m1 - xh * m2);
        }
        store_vec<T, VEC>(dx + row * dim + c, o);
      }
    }
  }
  float* mine = part + static_cast<long long>(blockIdx.x) * 2 * dim;
  if (kRows > 1) {
    // The groups hold the same columns: added in group order.
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = (k * G + tid) * VEC;
      if (c < dim) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          acc[(2 * grp) * dim + c + j] = dw[k][j];
          acc[(2 * grp + 1) * dim + c + j] = db[k][j];
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * dim; i += blockDim.x) {
      float s = 0.0f;
#pragma unroll
      for (int g = 0; g < kRows; ++g) s += acc[2 * g * dim + i];
      mine[i] = s;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = (k * G + tid) * VEC;
      if (c < dim) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          mine[c + j] = dw[k][j];
          mine[dim + c + j] = db[k][j];
        }
      }
    }
  }
}

// Rows of more than kBwdMax elements: dx, a CTA a row.
template <typename T, typename TW>
__global__ void __launch_bounds__(1024)
    layer_norm_dx_long(const T* dy, const T* x, const TW* __restrict__ w, const float* __restrict__ mean,
                       const float* __restrict__ rstd, long long rows, int dim, float inv_dim, T* dx) {
  __shared__ float red[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * dim, *gr = dy + row * dim;
    const float mu = mean[row], r = rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < dim; c += 1024) {
      const float a = to_f32(gr[c]) * to_f32(w[c]);
      s1 += a;
      s2 = fmaf(a, (to_f32(xr[c]) - mu) * r, s2);
    }
    const float m1 = group_sum<1024>(s1, red[0]) * inv_dim, m2 = group_sum<1024>(s2, red[1]) * inv_dim;
    for (int c = threadIdx.x; c < dim; c += 1024) {
      const float xh = (to_f32(xr[c]) - mu) * r;
      dx[row * dim + c] = from_f32<T>(r * (to_f32(gr[c]) * to_f32(w[c]) - m1 - xh * m2));
    }
    __syncthreads();  // red is written again by the next row
  }
}

// Rows of more than kBwdMax elements: the partial sums of dw and db, grid
// (column blocks, row pieces), a thread a column.  Runs before the dx kernel,
// which may write over dy or x.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_dw_long(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
                       const float* __restrict__ rstd, long long rows, int dim, float* __restrict__ part) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= dim) return;
  float dw = 0.0f, db = 0.0f;
  for (long long row = blockIdx.y; row < rows; row += gridDim.y) {
    const float g = to_f32(dy[row * dim + c]);
    dw = fmaf(g, (to_f32(x[row * dim + c]) - mean[row]) * rstd[row], dw);
    db += g;
  }
  float* mine = part + static_cast<long long>(blockIdx.y) * 2 * dim;
  mine[c] = dw;
  mine[dim + c] = db;
}

// dweight and dbias from `parts` partial rows: a CTA takes 32 of the 2 dim
// columns, its warps every 8th partial, and the warps' sums are added in order.
__global__ void __launch_bounds__(kThreads)
    layer_norm_join(const float* __restrict__ part, int parts, int dim, float* __restrict__ dweight,
                    float* __restrict__ dbias) {
  __shared__ float red[8][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < 2 * dim) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 8) s += part[static_cast<long long>(p) * 2 * dim + i];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < 2 * dim) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][lane];
    if (i < dim)
      dweight[i] = s;
    else if (dbias != nullptr)
      dbias[i - dim] = s;
  }
}

// Threads a row takes with `per` elements each: 32 to 1024.
int group_of(int dim, int per) {
  int g = 32;
  while (g < 1024 && g * per < dim) g *= 2;
  return g;
}

template <typename F>
auto with_group(int g, F&& f) {
  switch (g) {
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 256: return f(std::integral_constant<int, 256>{});
    case 512: return f(std::integral_constant<int, 512>{});
    default: return f(std::integral_constant<int, 1024>{});
  }
}

// Partial rows of dw and db: CTAs of the backward kernel.  Two CTAs of 256
// threads an SM (one of more threads), but no more than there are rows.
int bwd_parts(long long rows, int dim) {
  const int sms = 152;
  if (dim > kBwdMax) return static_cast<int>(rows < 64 ? rows : 64);
  const int g = group_of(dim, kBwdPer);
  const long long per = g > kThreads ? 1 : kThreads / g;
  const long long need = (rows + per - 1) / per;
  const long long most = static_cast<long long>(sms) * (g > 512 ? 1 : 2);
  return static_cast<int>(need < most ? need : most);
}

int check(long long rows, int dim) {
  if (rows < 0 || dim < 0 || rows > kMaxRows || dim > kMaxDim) return MUON_NS_ERR_INVALID_ARG;
  if (rows > 0 && dim == 0) return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

}  // namespace

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  int n = known[dev].load();
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 1;
    known[dev].store(n);
  }
  return n;
}

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_layer_norm(const void* x, int x_type, const void* weight, const void* bias, int w_type, long long rows,
                    int dim, float eps, void* y, float* mean, float* rstd, cudaStream_t stream) {
  int s = check(rows, dim);
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
      int vec = min_vec(min_vec(vec_of(dim, x, x_type), vec_of(dim, y, x_type)), vec_of(dim, weight, w_type));
      if (bias) vec = min_vec(vec, vec_of(dim, bias, w_type));
      return with_vec(vec, [&](auto vc) {
        return with_group(group_of(dim, kFwdPer), [&](auto gc) {
          constexpr int V = decltype(vc)::value, G = decltype(gc)::value;
          constexpr int T1 = G > kThreads ? G : kThreads;
          const long long grid = (rows + T1 / G - 1) / (T1 / G);
          return status_of(mns::launch_pdl(layer_norm_fwd<T, TW, V, G>, dim3(static_cast<unsigned>(grid)), dim3(T1), 0,
                                           stream, xp, wp, bp, rows, dim, inv, eps, yp, mean, rstd));
        });
      });
    });
  });
}

int muon_layer_norm_grad_workspace_size(long long rows, int dim, size_t* bytes) {
  const int s = check(rows, dim);
  if (s != MUON_NS_OK) return s;
  if (!bytes) return MUON_NS_ERR_INVALID_ARG;
  *bytes = rows == 0 ? 0 : align_up(sizeof(float) * 2 * static_cast<size_t>(bwd_parts(rows, dim)) * dim, 256);
  return MUON_NS_OK;
}

int muon_layer_norm_grad(const void* dy, const void* x, int x_type, const void* weight, int w_type,
                         const float* mean, const float* rstd, long long rows, int dim, void* dx, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int s = check(rows, dim);
  if (s != MUON_NS_OK) return s;
  if (!type_ok(x_type) || !type_ok(w_type)) return MUON_NS_ERR_INVALID_ARG;
  if (dim == 0) return MUON_NS_OK;
  if (rows > 0 && (!dy || !x || !weight || !mean || !rstd || !dx)) return MUON_NS_ERR_INVALID_ARG;
  if (!dweight) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(dy, x_type) || !element_aligned(x, x_type) || !element_aligned(dx, x_type) ||
      !element_aligned(weight, w_type) || !element_aligned(mean, MUON_LM_F32) ||
      !element_aligned(rstd, MUON_LM_F32) || !element_aligned(dweight, MUON_LM_F32) ||
      !element_aligned(dbias, MUON_LM_F32))
    return MUON_NS_ERR_ALIGNMENT;
  size_t need = 0;
  muon_layer_norm_grad_workspace_size(rows, dim, &need);
  if (rows > 0 && (!workspace || workspace_bytes < need)) return MUON_NS_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_NS_ERR_ALIGNMENT;
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  if (rows == 0) {  // sums over no rows
    cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * dim, stream);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * dim, stream);
    return status_of(e);
  }
  const float inv = 1.0f / static_cast<float>(dim);
  float* part = static_cast<float*>(workspace);
  const int parts = bwd_parts(rows, dim);
  s = with_type(x_type, [&](auto xt) {
    return with_type(w_type, [&](auto wt) {
      using T = decltype(xt);
      using TW = decltype(wt);
      const T *gp = static_cast<const T*>(dy), *xp = static_cast<const T*>(x);
      const TW* wp = static_cast<const TW*>(weight);
      T* op = static_cast<T*>(dx);
      if (dim > kBwdMax) {
        cudaError_t e = mns::launch_pdl(layer_norm_dw_long<T>,
                                        dim3(static_cast<unsigned>((dim + kThreads - 1) / kThreads), parts),
                                        dim3(kThreads), 0, stream, gp, xp, mean, rstd, rows, dim, part);
        if (e != cudaSuccess) return status_of(e);
        const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
        return status_of(mns::launch_pdl(layer_norm_dx_long<T, TW>, dim3(grid), dim3(1024), 0, stream, gp, xp, wp,
                                         mean, rstd, rows, dim, inv, op));
      }
      const int vec = min_vec(min_vec(vec_of(dim, x, x_type), vec_of(dim, dy, x_type)),
                              min_vec(vec_of(dim, dx, x_type), vec_of(dim, weight, w_type)));
      return with_vec(vec, [&](auto vc) {
        return with_group(group_of(dim, kBwdPer), [&](auto gc) {
          constexpr int V = decltype(vc)::value, G = decltype(gc)::value;
          constexpr int T1 = G > kThreads ? G : kThreads;
          const size_t smem = T1 > G ? sizeof(float) * 2 * (T1 / G) * dim : 0;
          return status_of(mns::launch_pdl(layer_norm_bwd<T, TW, V, G>, dim3(parts), dim3(T1), smem, stream, gp, xp,
                                           wp, mean, rstd, rows, dim, inv, op, part));
        });
      });
    });
  });
  if (s != MUON_NS_OK) return s;
  return status_of(mns::launch_pdl(layer_norm_join, dim3(static_cast<unsigned>((2 * dim + 31) / 32)), dim3(kThreads), 0,
                                   stream, static_cast<const float*>(part), parts, dim, dweight, dbias));
}

}  // extern "C"
