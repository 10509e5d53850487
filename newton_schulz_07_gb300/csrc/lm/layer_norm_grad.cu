// Layer norm's gradient.  With xh = (x - mean) r and a = dy w of a row,
//   dx = r (a - mean(a) - xh mean(a xh)),
// and over the rows dw = sum dy xh, db = sum dy.
//
// A CTA walks the rows with the grid's stride and holds its columns' dw and db
// in registers, so x and dy are read once; at its end it stores one partial
// row of each, and a second kernel adds the partials of a column in a fixed
// order.  Bound by HBM traffic.  Rows too long for the registers take the
// _long kernels, which read a row again from cache.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "lm/layer_norm.cuh"

namespace mns {
namespace lm {

namespace {

constexpr int kBwdPer = 16;   // elements a thread holds (x, dy, dw and db)
constexpr int kRingPer = 32;  // with x and dy in shared memory (dw and db)
constexpr int kBwdMax = 1024 * kBwdPer;
constexpr int kRingMax = 512 * kRingPer;
constexpr int kRingSmem = 200 * 1024;
constexpr int kFewCta = 512;  // CTA size for few rows
constexpr int kFewSmem = sizeof(float) * 2 * kFewCta * kBwdPer;

// One row of each group, from its units of x and dy (unit(k, c): those of the
// thread's k-th unit, at column c): adds to the thread's dw and db and, after
// the sums over the row, writes dx.  Every thread of the CTA takes part.
//
// With d = x - mean and e = dy d: dw += r e, db += dy, and the row's sums are
// those of dy w and e w; xh mean(a xh) = r^2 d mean(e w).
template <typename T, typename TW, int VEC, int G, typename C, typename U>
__device__ __forceinline__ void grad_row(const U& unit, const TW* __restrict__ w, bool live, long long row, int dim,
                                         float inv_dim, float mu, float r, T* dx, float2 (&dw)[C::kK][C::kP],
                                         float2 (&db)[C::kK][C::kP], float (*red)[32]) {
  const int tid = threadIdx.x & (G - 1);
  float2 s1 = both(0.0f), s2 = both(0.0f);
  if (live) {
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      const int c = C::first(k, tid);
      if (c < dim) {
        float2 xp[C::kP], gp[C::kP], wp[C::kP];
        unit(k, c, xp, gp);
        to_pairs<TW, C::kU>(C::load(w, c, dim), wp);
#pragma unroll
        for (int j = 0; j < C::kP; ++j) {
          const float2 e = mul2(gp[j], add2(xp[j], both(-mu)));
          dw[k][j] = fma2(e, both(r), dw[k][j]);
          db[k][j] = add2(db[k][j], gp[j]);
          s1 = fma2(gp[j], wp[j], s1);
          s2 = fma2(e, wp[j], s2);
        }
      }
    }
  }
  float sum[2] = {s1.x + s1.y, s2.x + s2.y};
  group_sums<G, 2>(sum, red);
  const float m1 = -r * (sum[0] * inv_dim), m2 = -r * (r * (r * (sum[1] * inv_dim)));
  if (live) {
#pragma unroll
    for (int k = 0; k < C::kK; ++k) {
      const int c = C::first(k, tid);
      if (c < dim) {
        float2 xp[C::kP], gp[C::kP], wp[C::kP];
        unit(k, c, xp, gp);
        to_pairs<TW, C::kU>(C::load(w, c, dim), wp);
#pragma unroll
        for (int j = 0; j < C::kP; ++j) {
          const float2 d = add2(xp[j], both(-mu));
          xp[j] = fma2(mul2(gp[j], both(r)), wp[j], fma2(d, both(m2), both(m1)));
        }
        C::store(dx + row * dim, c, dim, xp);
      }
    }
  }
}

// part: fp32 [gridDim.x][2][dim], this CTA's dw and db.
// FEW: the grid is one cluster, whose CTAs add their sums through each other's
// shared memory (in rank order), so few rows take one launch and no workspace.
template <typename T, typename TW, int VEC, int G, bool FEW>
__global__ void __launch_bounds__(FEW ? kFewCta : (G > kNormCta ? G : kNormCta))
    layer_norm_bwd(const T* dy, const T* x, const TW* __restrict__ w, const float* __restrict__ mean,
                   const float* __restrict__ rstd, long long rows, int dim, float inv_dim, T* dx,
                   float* __restrict__ part, float* __restrict__ dweight, float* __restrict__ dbias) {
  constexpr int kRows = (FEW ? kFewCta : (G > kNormCta ? G : kNormCta)) / G;
  using C = Cols<VEC, G, kBwdPer>;
  constexpr int kK = C::kK;
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) float acc[];  // [kRows][2][dim], only with kRows > 1 or FEW
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (G - 1), grp = threadIdx.x / G;
  float2 dw[kK][C::kP] = {}, db[kK][C::kP] = {};
  const long long stride = static_cast<long long>(gridDim.x) * kRows;
  int buf = 0;
  Vec<T, C::kU> xv[kK], gv[kK], xn[FEW ? kK : 1], gn[FEW ? kK : 1];
  float mu = 0.0f, r = 0.0f, mu_next = 0.0f, r_next = 0.0f;
  auto fetch = [&](long long row, auto& xs, auto& gs, float& m, float& q) {
    if (row >= rows) return;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = C::first(k, tid);
      if (c < dim) {
        xs[k] = C::load(x + row * dim, c, dim);
        gs[k] = C::load(dy + row * dim, c, dim);
      }
    }
    m = mean[row];
    q = rstd[row];
  };
  const long long first = static_cast<long long>(blockIdx.x) * kRows;
  if constexpr (FEW) fetch(first + grp, xn, gn, mu_next, r_next);
  // Every group of the CTA makes the same number of turns (barriers inside).
  for (long long r0 = first; r0 < rows; r0 += stride, buf ^= 1) {
    const long long row = r0 + grp;
    const bool live = row < rows;
    if constexpr (FEW) {
      // One row ahead: a CTA an SM leaves nothing else to hide the loads.
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        xv[k] = xn[k];
        gv[k] = gn[k];
      }
      mu = mu_next;
      r = r_next;
      fetch(row + stride, xn, gn, mu_next, r_next);
    } else {
      fetch(row, xv, gv, mu, r);
    }
    const auto unit = [&](int k, int, float2(&xp)[C::kP], float2(&gp)[C::kP]) {
      to_pairs<T, C::kU>(xv[k], xp);
      to_pairs<T, C::kU>(gv[k], gp);
    };
    grad_row<T, TW, VEC, G, C>(unit, w, live, row, dim, inv_dim, mu, live ? r : 0.0f, dx, dw, db, red[buf]);
  }
  float* mine = FEW ? acc : part + static_cast<long long>(blockIdx.x) * 2 * dim;
  if (kRows > 1 || FEW) {
    // The groups hold the same columns: added in group order.
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int c = C::first(k, tid);
      if (c < dim) {
        C::template store<true>(acc + (2 * grp) * dim, c, dim, dw[k]);
        C::template store<true>(acc + (2 * grp + 1) * dim, c, dim, db[k]);
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
      const int c = C::first(k, tid);
      if (c < dim) {
        C::template store<true>(mine, c, dim, dw[k]);
        C::template store<true>(mine + dim, c, dim, db[k]);
      }
    }
  }
  if (FEW) {
    const int ctas = static_cast<int>(gridDim.x);
    __syncthreads();
    if (ctas > 1) ptx::cluster_sync();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < 2 * dim; i += ctas * blockDim.x) {
      float v[8];  // all loads in flight at once
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        v[r] = 0.0f;
        if (r < ctas) {
          if (ctas > 1)
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(v[r])
                         : "r"(ptx::mapa(ptx::smem_u32(&acc[i]), static_cast<uint32_t>(r))));
          else
            v[r] = acc[i];
        }
      }
      float s = v[0];
#pragma unroll
      for (int r = 1; r < 8; ++r) s += v[r];
      if (i < dim)
        dweight[i] = s;
      else if (dbias != nullptr)
        dbias[i - dim] = s;
    }
    if (ctas > 1) ptx::cluster_sync();  // no CTA leaves while another reads its sums
  }
}

// The same with the rows of x and dy copied to shared memory one turn ahead
// (cp.async; a thread copies and reads its own elements, so no barrier is
// needed for them, except for those copied by words) and read from there twice,
// which leaves the registers to kRingPer columns of dw and db a thread.
template <typename T, typename TW, int VEC, int G>
__global__ void __launch_bounds__(G > kNormCta ? G : kNormCta, G > kNormCta ? 1 : 2)
    layer_norm_bwd_ring(const T* dy, const T* x, const TW* __restrict__ w, const float* __restrict__ mean,
                        const float* __restrict__ rstd, long long rows, int dim, float inv_dim, T* dx,
                        float* __restrict__ part) {
  constexpr int kRows = (G > kNormCta ? G : kNormCta) / G;
  using C = Cols<VEC, G, kRingPer>;
  constexpr int kK = C::kK, kP = C::kP;
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) uint8_t ring[];  // [2 turns][x, dy][kRows][dim], then [kRows][2][dim] fp32
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (G - 1), grp = threadIdx.x / G;
  const long long stride = static_cast<long long>(gridDim.x) * kRows;
  constexpr bool kWords = kByWords<T, VEC>;
  const int pitch = kWords ? word_pitch(dim) : dim;
  T* mine_x = reinterpret_cast<T*>(ring) + grp * pitch;
  const int turn = 2 * kRows * pitch, to_dy = kRows * pitch;
  float mu_next = 0.0f, r_next = 0.0f;
  auto fetch = [&](int st, long long row) {
    if (row < rows) {
      if constexpr (kWords) {
        copy_words<G>(mine_x + st * turn, x, row, rows, dim, tid);
        copy_words<G>(mine_x + st * turn + to_dy, dy, row, rows, dim, tid);
      } else {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const int c = C::first(k, tid);
          if (c < dim) {
            C::copy(mine_x + st * turn, x + row * dim, c, dim);
            C::copy(mine_x + st * turn + to_dy, dy + row * dim, c, dim);
          }
        }
      }
      mu_next = mean[row];
      r_next = rstd[row];
    }
    copy_commit();
  };
  float2 dw[kK][kP] = {}, db[kK][kP] = {};
  const long long first = static_cast<long long>(blockIdx.x) * kRows;
  fetch(0, first + grp);
  int st = 0;
  // Every group of the CTA makes the same number of turns (barriers inside).
  for (long long r0 = first; r0 < rows; r0 += stride, st ^= 1) {
    const long long row = r0 + grp;
    const bool live = row < rows;
    const float mu = mu_next, r = live ? r_next : 0.0f;
    fetch(st ^ 1, row + stride);
    copy_wait<1>();
    if (kWords) group_barrier<G>();
    const T* xs = mine_x + st * turn + (kWords ? row_shift(x + row * dim) : 0);
    const T* gs = mine_x + st * turn + to_dy + (kWords ? row_shift(dy + row * dim) : 0);
    const auto unit = [&](int, int c, float2(&xp)[C::kP], float2(&gp)[C::kP]) {
      to_pairs<T, C::kU>(C::template load<true>(xs, c, dim), xp);
      to_pairs<T, C::kU>(C::template load<true>(gs, c, dim), gp);
    };
    grad_row<T, TW, VEC, G, C>(unit, w, live, row, dim, inv_dim, mu, r, dx, dw, db, red[st]);
    if (kWords) group_barrier<G>();  // the row has been read before its buffer is copied to
  }
  copy_wait<0>();
  float* out = part + static_cast<long long>(blockIdx.x) * 2 * dim;
  float* acc = reinterpret_cast<float*>(ring);
  if (kRows > 1) {
    __syncthreads();  // the groups' rows have been read
    acc += 2 * grp * dim;
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int c = C::first(k, tid);
    if (c < dim) {
      float* to = kRows > 1 ? acc : out;
      C::template store<true>(to, c, dim, dw[k]);
      C::template store<true>(to + dim, c, dim, db[k]);
    }
  }
  if (kRows > 1) {
    // The groups hold the same columns: added in group order.
    __syncthreads();
    acc = reinterpret_cast<float*>(ring);
    for (int i = threadIdx.x; i < 2 * dim; i += blockDim.x) {
      float s = 0.0f;
#pragma unroll
      for (int g = 0; g < kRows; ++g) s += acc[2 * g * dim + i];
      out[i] = s;
    }
  }
}

// Rows of more than kBwdMax elements: dx, a CTA a row.
template <typename T, typename TW>
__global__ void __launch_bounds__(1024)
    layer_norm_dx_long(const T* dy, const T* x, const TW* __restrict__ w, const float* __restrict__ mean,
                       const float* __restrict__ rstd, long long rows, int dim, float inv_dim, T* dx) {
  __shared__ float red[2][1][32];
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
__global__ void __launch_bounds__(kNormCta)
    layer_norm_dw_long(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
                       const float* __restrict__ rstd, long long rows, int dim, float* __restrict__ part) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int c = blockIdx.x * kNormCta + threadIdx.x;
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
__global__ void __launch_bounds__(kNormCta)
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

// Shared memory of the ring: two turns of the CTA's rows of x and dy, which
// also hold [rows][2][dim] fp32 at the end.
size_t ring_smem(int dim, int x_type) {
  const int g = group_of(dim, kRingPer);
  return static_cast<size_t>(4) * (g > kNormCta ? 1 : kNormCta / g) * word_pitch(dim) * type_size(x_type);
}

// The ring's two turns have to fit, and its copies are of 4 bytes at least.
bool use_ring(int dim, int x_type, int vec, const void* x, const void* dy) {
  const bool words = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dy)) & 3) == 0;
  return dim <= kRingMax && (vec * type_size(x_type) >= 4 || words) && ring_smem(dim, x_type) <= kRingSmem;
}

// CTAs of the one cluster that few rows take (1, 2, 4 or 8), or 0.  Up to 4
// turns of it: 517 rows of 768 bf16 take 9 turns and 21 us on the device,
// against 9 us by the two launches, which take 6 us longer to issue.
int few_ctas(long long rows, int dim) {
  const int g = group_of(dim, kBwdPer);
  if (g > kFewCta || rows > 4LL * 8 * (kFewCta / g)) return 0;
  int n = 1;
  while (n < 8 && n * (kFewCta / g) < rows) n *= 2;
  return n;
}

// Partial rows of dw and db: CTAs of the backward kernel.  Two CTAs of 256
// threads an SM, or one of more threads, but no more than there are rows.
int bwd_parts(long long rows, int dim, int per_thread) {
  if (dim > kBwdMax) return static_cast<int>(rows < 64 ? rows : 64);
  const int g = group_of(dim, per_thread);
  const long long per = g > kNormCta ? 1 : kNormCta / g;
  const long long need = (rows + per - 1) / per;
  const long long most = static_cast<long long>(kSms) * (g > kNormCta ? 1 : 2);
  return static_cast<int>(need < most ? need : most);
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

int muon_layer_norm_grad_workspace_size(long long rows, int dim, size_t* bytes) {
  const int s = norm_check(rows, dim);
  if (s != MUON_NS_OK) return s;
  if (!bytes) return MUON_NS_ERR_INVALID_ARG;
  // The type and the alignment of the call's rows choose between the kernels.
  const bool none = rows == 0 || few_ctas(rows, dim) > 0;
  const int a = none ? 0 : bwd_parts(rows, dim, kBwdPer), b = none ? 0 : bwd_parts(rows, dim, kRingPer);
  *bytes = align_up(sizeof(float) * 2 * static_cast<size_t>(a > b ? a : b) * dim, 256);
  return MUON_NS_OK;
}

int muon_layer_norm_grad(const void* dy, const void* x, int x_type, const void* weight, int w_type,
                         const float* mean, const float* rstd, long long rows, int dim, void* dx, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int s = norm_check(rows, dim);
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
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return MUON_NS_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_NS_ERR_ALIGNMENT;
  }
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  if (rows == 0) {  // sums over no rows
    cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * dim, stream);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * dim, stream);
    return status_of(e);
  }
  const float inv = 1.0f / static_cast<float>(dim);
  float* part = static_cast<float*>(workspace);
  const int vec = min_vec(min_vec(norm_vec(dim, x, x_type), norm_vec(dim, dy, x_type)),
                          min_vec(norm_vec(dim, dx, x_type), vec_of(dim, weight, w_type)));
  const int few = few_ctas(rows, dim);
  const bool ring = few == 0 && use_ring(dim, x_type, vec, x, dy);
  const int parts = bwd_parts(rows, dim, ring ? kRingPer : kBwdPer);
  s = with_type(x_type, [&](auto xt) {
    return with_type(w_type, [&](auto wt) {
      using T = decltype(xt);
      using TW = decltype(wt);
      const T *gp = static_cast<const T*>(dy), *xp = static_cast<const T*>(x);
      const TW* wp = static_cast<const TW*>(weight);
      T* op = static_cast<T*>(dx);
      if (dim > kBwdMax) {
        cudaError_t e = mns::launch_pdl(layer_norm_dw_long<T>,
                                        dim3(static_cast<unsigned>((dim + kNormCta - 1) / kNormCta), parts),
                                        dim3(kNormCta), 0, stream, gp, xp, mean, rstd, rows, dim, part);
        if (e != cudaSuccess) return status_of(e);
        const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
        return status_of(mns::launch_pdl(layer_norm_dx_long<T, TW>, dim3(grid), dim3(1024), 0, stream, gp, xp, wp,
                                         mean, rstd, rows, dim, inv, op));
      }
      if (ring)
        return with_norm_vec<T>(vec, [&](auto vc) {
          return with_group(group_of(dim, kRingPer), [&](auto gc) {
            constexpr int V = decltype(vc)::value, G = decltype(gc)::value;
            if constexpr (G > 512) {
              return static_cast<int>(MUON_NS_ERR_INVALID_ARG);  // use_ring says no
            } else {
              constexpr int T1 = G > kNormCta ? G : kNormCta;
              auto kernel = layer_norm_bwd_ring<T, TW, V, G>;
              static std::atomic<unsigned long long> configured{0};
              const cudaError_t e = allow_smem(kernel, kRingSmem, &configured);
              if (e != cudaSuccess) return status_of(e);
              return status_of(mns::launch_pdl(kernel, dim3(parts), dim3(T1), ring_smem(dim, x_type), stream, gp, xp,
                                               wp, mean, rstd, rows, dim, inv, op, part));
            }
          });
        });
      return with_norm_vec<T>(vec, [&](auto vc) {
        return with_group(group_of(dim, kBwdPer), [&](auto gc) {
          constexpr int V = decltype(vc)::value, G = decltype(gc)::value;
          constexpr int T1 = G > kNormCta ? G : kNormCta;
          const size_t smem = T1 > G ? sizeof(float) * 2 * (T1 / G) * dim : 0;
          if constexpr (G <= kFewCta) {
            if (few > 0) {
              auto kernel = layer_norm_bwd<T, TW, V, G, true>;
              static std::atomic<unsigned long long> configured{0};
              const cudaError_t e = allow_smem(kernel, kFewSmem, &configured);
              if (e != cudaSuccess) return status_of(e);
              return status_of(mns::launch_pdl_cluster(kernel, dim3(few), dim3(kFewCta),
                                                       sizeof(float) * 2 * (kFewCta / G) * dim, stream, few, gp, xp, wp,
                                                       mean, rstd, rows, dim, inv, op, part, dweight, dbias));
            }
          }
          return status_of(mns::launch_pdl(layer_norm_bwd<T, TW, V, G, false>, dim3(parts), dim3(T1), smem, stream, gp,
                                           xp, wp, mean, rstd, rows, dim, inv, op, part, dweight, dbias));
        });
      });
    });
  });
  if (s != MUON_NS_OK || few > 0) return s;
  return status_of(mns::launch_pdl(layer_norm_join, dim3(static_cast<unsigned>((2 * dim + 31) / 32)), dim3(kNormCta), 0,
                                   stream, static_cast<const float*>(part), parts, dim, dweight, dbias));
}

}  // extern "C"
