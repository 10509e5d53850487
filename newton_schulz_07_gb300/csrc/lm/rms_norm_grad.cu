// Gradient of the root-mean-square norm.  With xh = s r and a = dy w of a row,
//   ds = r (a - xh mean(a xh)) + dsum,
// and over the rows dw = sum dy xh.
//
// A CTA walks the rows with the grid's stride and holds its columns' dw in
// registers, 32 a thread.  Rows of s, dy and dsum are copied to shared memory one
// turn ahead (cp.async; a thread copies and reads its own elements, so no barrier
// is needed for them) and read from there twice.  They are read twice from global
// memory instead where their accesses are of 2 bytes, less than cp.async can copy, and
// where two turns of a CTA's rows pass 100 KB (200 KB of a CTA of 512 threads): most
// fp32 rows from 1024 columns on (16384 x 4096 with dsum: 309 us, 52 % of the copy
// rate; 16384 x 4266 through shared memory 292, 57 %).  At
// its end a CTA stores one partial row, and a second kernel adds those of a column
// in a fixed order; few rows are one cluster's, whose CTAs add their partial rows
// through each other's shared memory.  Bound by HBM traffic.  Rows too long for
// the registers take the _long kernels.
#include <atomic>
#include <cmath>

#include "lm/block8.cuh"
#include "muon_moe.h"

namespace mns {
namespace lm {

namespace {

constexpr int kGradPer = 32;              // dw columns a thread holds
constexpr int kGradMax = 512 * kGradPer;  // longest row of the register kernels
constexpr int kGradSmem = 200 * 1024;
constexpr int kFewCtas = 8;               // of the cluster that few rows take

// A group's columns in units of 128 / kLanes elements, as Blk<W>.
template <int W>
struct GradBlk : Blk<W> {
  static constexpr int kK = kGradPer / Blk<W>::kU;
};

template <typename T, typename TW>
struct RmsGrad {
  const T* dy;
  const T* s;
  const T* dsum;  // or null
  const TW* w;
  const float* rstd;
  long long rows;
  int dim;
  float inv_dim;
  T* ds;
  float* part;     // [gridDim.x][dim]
  float* dweight;  // the cluster's result
};

template <typename T, typename TW, int W, bool RING, bool FEW>
__global__ void __launch_bounds__(512) rms_norm_bwd(const RmsGrad<T, TW> R, int g) {
  using B = GradBlk<W>;
  constexpr int kK = B::kK, kH = B::kH, kP = B::kP;
  __shared__ float red[2][32];
  // [2 turns][dy, s, dsum][groups][dim] of T, then (again from its start) [groups][dim] fp32
  extern __shared__ __align__(16) uint8_t ring[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (g - 1), grp = threadIdx.x / g, groups = blockDim.x / g;
  const int lane = tid & (B::kLanes - 1), first = tid / B::kLanes, step = g / B::kLanes;
  const int dim = R.dim, slice = groups * dim, tensors = R.dsum != nullptr ? 3 : 2;
  T* mine = reinterpret_cast<T*>(ring) + grp * dim;
  const T* from[3] = {R.dy, R.s, R.dsum};
  auto fetch = [&](int st, long long row) {
    if (!RING) return;
    if (row < R.rows) {
      for (int i = 0; i < tensors; ++i) {
        const T* src = from[i] + row * dim;
        T* dst = mine + (st * tensors + i) * slice;
#pragma unroll
        for (int k = 0; k < kK; ++k)
#pragma unroll
          for (int p = 0; p < kP; ++p) {
            const int c = B::col(first + k * step, lane, p);
            if constexpr (W * sizeof(T) >= 4)
              if (c < dim) copy_async<W * sizeof(T)>(dst + c, src + c);
          }
      }
    }
    copy_commit();
  };
  // The columns are the same in every row: their weights stay in registers.
  Vec<TW, W> wv[kK][kP];
#pragma unroll
  for (int k = 0; k < kK; ++k) B::load(R.w, first + k * step, lane, dim, wv[k]);
  float2 dw[kK][kH] = {};
  const long long stride = static_cast<long long>(gridDim.x) * groups;
  const long long row0 = static_cast<long long>(blockIdx.x) * groups;
  float r_next = 0.0f;
  fetch(0, row0 + grp);
  if (row0 + grp < R.rows) r_next = R.rstd[row0 + grp];
  int st = 0;
  // Every group of the CTA makes the same number of turns (barriers inside).
  for (long long r0 = row0; r0 < R.rows; r0 += stride, st ^= 1) {
    const long long row = r0 + grp;
    const bool live = row < R.rows;
    const float r = r_next;
    fetch(st ^ 1, row + stride);
    if (row + stride < R.rows) r_next = R.rstd[row + stride];
    if (RING) copy_wait<1>();
    auto unit = [&](int i, int block, float2 (&f)[kH]) {
      Vec<T, W> v[kP];
      if (RING) {
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          const int c = B::col(block, lane, p);
          v[p] = c < dim ? load_vec<T, W>(mine + (st * tensors + i) * slice + c) : Vec<T, W>{};
        }
      } else {
        B::load(from[i] + row * dim, block, lane, dim, v);
      }
      B::widen(v, f);
    };
    float2 along = both(0.0f);
    if (live) {
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int block = first + k * step;
        if (block * kBlock8 >= dim) continue;
        float2 dy[kH], s[kH], w[kH];
        unit(0, block, dy);
        unit(1, block, s);
        B::widen(wv[k], w);
#pragma unroll
        for (int j = 0; j < kH; ++j) {
          const float2 e = mul2(dy[j], s[j]);
          dw[k][j] = fma2(e, both(r), dw[k][j]);
          along = fma2(e, w[j], along);
        }
      }
    }
    // r xh mean(a xh) = s r^3 mean(dy w s)
    const float c = -r * (r * (r * (group_total(along.x + along.y, g, red[st]) * R.inv_dim)));
    if (live) {
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int block = first + k * step;
        if (block * kBlock8 >= dim) continue;
        float2 dy[kH], s[kH], w[kH], o[kH];
        unit(0, block, dy);
        unit(1, block, s);
        B::widen(wv[k], w);
        if (R.dsum != nullptr)
          unit(2, block, o);
        else
#pragma unroll
          for (int j = 0; j < kH; ++j) o[j] = both(0.0f);
#pragma unroll
        for (int j = 0; j < kH; ++j) o[j] = fma2(mul2(dy[j], both(r)), w[j], fma2(s[j], both(c), o[j]));
        B::store(R.ds + row * dim, block, lane, dim, o);
      }
    }
  }
  if (RING) copy_wait<0>();
  // The groups hold the same columns: added in group order.
  float* acc = reinterpret_cast<float*>(ring);
  float* out = FEW ? acc : R.part + static_cast<long long>(blockIdx.x) * dim;
  const bool join = groups > 1;
  if (RING || FEW) __syncthreads();  // the rows in shared memory have been read
#pragma unroll
  for (int k = 0; k < kK; ++k) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const int col = B::col(first + k * step, lane, p);
      if (col < dim) {
#pragma unroll
        for (int i = 0; i < W; ++i) (join ? acc + grp * dim : out)[col + i] = (p * W + i) & 1 ? dw[k][(p * W + i) / 2].y : dw[k][(p * W + i) / 2].x;
      }
    }
  }
  if (join) {
    __syncthreads();
    for (int i = threadIdx.x; i < dim; i += blockDim.x) {
      float v = 0.0f;
      for (int q = 0; q < groups; ++q) v += acc[q * dim + i];
      out[i] = v;  // (FEW: the first group's, read by this thread alone)
    }
  }
  if (FEW) {
    const int ctas = static_cast<int>(gridDim.x);
    __syncthreads();
    ptx::cluster_sync();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < dim; i += ctas * blockDim.x) {
      float v[kFewCtas];  // all loads in flight at once
#pragma unroll
      for (int q = 0; q < kFewCtas; ++q) {
        v[q] = 0.0f;
        if (q < ctas)
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(v[q])
                       : "r"(ptx::mapa(ptx::smem_u32(&acc[i]), static_cast<uint32_t>(q))));
      }
      float sum = v[0];
#pragma unroll
      for (int q = 1; q < kFewCtas; ++q) sum += v[q];
      R.dweight[i] = sum;
    }
    ptx::cluster_sync();  // no CTA leaves while another reads its sums
  }
}

// Rows of more than kGradMax elements: ds, a CTA a row.
template <typename T, typename TW>
__global__ void __launch_bounds__(1024) rms_norm_ds_long(const RmsGrad<T, TW> R) {
  __shared__ float red[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  int buf = 0;
  for (long long row = blockIdx.x; row < R.rows; row += gridDim.x, buf ^= 1) {
    const long long at = row * R.dim;
    const float r = R.rstd[row];
    float along = 0.0f;
    for (int c = threadIdx.x; c < R.dim; c += 1024)
      along = fmaf(to_f32(R.dy[at + c]) * to_f32(R.s[at + c]), to_f32(R.w[c]), along);
    const float k = -r * (r * (r * (group_total(along, 1024, red[buf]) * R.inv_dim)));
    for (int c = threadIdx.x; c < R.dim; c += 1024)
      R.ds[at + c] = from_f32<T>(fmaf(to_f32(R.dy[at + c]) * r, to_f32(R.w[c]),
                                      fmaf(to_f32(R.s[at + c]), k, R.dsum != nullptr ? to_f32(R.dsum[at + c]) : 0.0f)));
  }
}

// Rows of more than kGradMax elements: the partial sums of dw, grid (column
// blocks, row pieces), a thread a column.  Runs before the ds kernel, which may
// write over dy or s.
template <typename T, typename TW>
__global__ void __launch_bounds__(256) rms_norm_dw_long(const RmsGrad<T, TW> R) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= R.dim) return;
  float dw = 0.0f;
  for (long long row = blockIdx.y; row < R.rows; row += gridDim.y)
    dw = fmaf(to_f32(R.dy[row * R.dim + c]) * to_f32(R.s[row * R.dim + c]), R.rstd[row], dw);
  R.part[static_cast<long long>(blockIdx.y) * R.dim + c] = dw;
}

// dweight from `parts` partial rows: a CTA takes 32 columns, its warps every 8th
// partial, and the warps' sums are added in order.
__global__ void __launch_bounds__(256)
    rms_norm_join(const float* part, int parts, int dim, float* dweight) {
  __shared__ float red[8][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < dim) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 8) s += part[static_cast<long long>(p) * dim + i];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < dim) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][lane];
    dweight[i] = s;
  }
}

int grad_cta(int g) { return g > kRowCta ? g : kRowCta; }

// CTAs of the one cluster that few rows take (1 to 8), or 0: up to 4 turns of it.
int few_ctas(long long rows, int dim) {
  if (dim > kGradMax) return 0;
  const int groups = grad_cta(row_group(dim, kGradPer)) / row_group(dim, kGradPer);
  if (rows > 4LL * kFewCtas * groups) return 0;
  int n = 1;
  while (n < kFewCtas && n * groups < rows) n *= 2;
  return n;
}

// Partial rows of dw: CTAs of the kernel, two of 256 threads an SM or one of 512,
// but no more than there are rows for.
int grad_parts(long long rows, int dim) {
  if (dim > kGradMax) return static_cast<int>(rows < 64 ? rows : 64);
  const int g = row_group(dim, kGradPer), cta = grad_cta(g);
  const long long need = (rows + cta / g - 1) / (cta / g), most = static_cast<long long>(kSms) * (cta > kRowCta ? 1 : 2);
  return static_cast<int>(need < most ? need : most);
}

int rms_check(long long rows, int dim) {
  if (rows < 0 || dim < 0 || rows > kMaxRows || dim > kMaxDim) return MUON_NS_ERR_INVALID_ARG;
  if (rows > 0 && dim == 0) return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_rms_norm_grad_workspace_size(long long rows, int dim, size_t* bytes) {
  const int st = rms_check(rows, dim);
  if (st != MUON_NS_OK) return st;
  if (!bytes) return MUON_NS_ERR_INVALID_ARG;
  const bool none = rows == 0 || few_ctas(rows, dim) > 0;
  *bytes = none ? 0 : align_up(sizeof(float) * static_cast<size_t>(grad_parts(rows, dim)) * dim, 256);
  return MUON_NS_OK;
}

int muon_rms_norm_grad(const void* dy, const void* s, int x_type, const void* weight, int w_type, const float* rstd,
                       const void* dsum, long long rows, int dim, void* ds, float* dweight, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  int st = rms_check(rows, dim);
  if (st != MUON_NS_OK) return st;
  if (!type_ok(x_type) || !type_ok(w_type)) return MUON_NS_ERR_INVALID_ARG;
  if (dim == 0) return MUON_NS_OK;
  if (rows > 0 && (!dy || !s || !weight || !rstd || !ds)) return MUON_NS_ERR_INVALID_ARG;
  if (!dweight) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(dy, x_type) || !element_aligned(s, x_type) || !element_aligned(dsum, x_type) ||
      !element_aligned(ds, x_type) || !element_aligned(weight, w_type) || !element_aligned(rstd, MUON_LM_F32) ||
      !element_aligned(dweight, MUON_LM_F32))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t bytes = static_cast<size_t>(rows) * dim * type_size(x_type);
  // ds may be one of the rows that it is made of, not a shifted one.
  for (const void* p : {dy, s, dsum})
    if (p && p != ds && overlap(ds, bytes, p, bytes)) return MUON_NS_ERR_INVALID_ARG;
  size_t need = 0;
  muon_rms_norm_grad_workspace_size(rows, dim, &need);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return MUON_NS_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_NS_ERR_ALIGNMENT;
  }
  const Span g = {dy, bytes}, v = {s, bytes}, past = {dsum, bytes}, o = {rows > 0 ? ds : nullptr, bytes},
             w = {weight, static_cast<size_t>(dim) * type_size(w_type)}, rs = {rstd, 4 * static_cast<size_t>(rows)},
             dw = {dweight, 4 * static_cast<size_t>(dim)}, ws = {workspace, need};
  if (overlaps(w, {o, dw, ws}) || overlaps(rs, {o, dw, ws}) || overlaps(dw, {g, v, past, o, ws}) || overlaps(ws, {g, v, past, o}))
    return MUON_NS_ERR_INVALID_ARG;
  if ((st = muon_ns_device_supported(-1)) != MUON_NS_OK) return st;
  if (rows == 0) return status_of(cudaMemsetAsync(dweight, 0, sizeof(float) * dim, stream));  // a sum over no rows
  float* part = static_cast<float*>(workspace);
  const int few = few_ctas(rows, dim), parts = grad_parts(rows, dim);
  st = with_type(x_type, [&](auto xt) {
    return with_type(w_type, [&](auto wt) {
      using T = decltype(xt);
      using TW = decltype(wt);
      RmsGrad<T, TW> R = {};
      R.dy = static_cast<const T*>(dy);
      R.s = static_cast<const T*>(s);
      R.dsum = static_cast<const T*>(dsum);
      R.w = static_cast<const TW*>(weight);
      R.rstd = rstd;
      R.rows = rows;
      R.dim = dim;
      R.inv_dim = 1.0f / static_cast<float>(dim);
      R.ds = static_cast<T*>(ds);
      R.part = part;
      R.dweight = dweight;
      if (dim > kGradMax) {
        const cudaError_t e = mns::launch_pdl(rms_norm_dw_long<T, TW>, dim3(static_cast<unsigned>((dim + 255) / 256), parts),
                                              dim3(256), 0, stream, R);
        if (e != cudaSuccess) return status_of(e);
        const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
        return status_of(mns::launch_pdl(rms_norm_ds_long<T, TW>, dim3(grid), dim3(1024), 0, stream, R));
      }
      const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
      int width = row_width(dim, x_type, at(dy) | at(s) | at(dsum) | at(ds));
      while (width > 1 && at(weight) % (width * type_size(w_type) > 16 ? 32 : width * type_size(w_type)) != 0)
        width = width > 2 ? 2 : 1;
      const int g = row_group(dim, kGradPer), cta = grad_cta(g);
      const size_t line = static_cast<size_t>(cta / g) * dim;  // elements of the CTA's rows
      const size_t rows_smem = line * 2 * (dsum ? 3 : 2) * type_size(x_type);
      const bool ring = width * type_size(x_type) >= 4 && rows_smem <= static_cast<size_t>(kGradSmem) / (cta > kRowCta ? 1 : 2);
      size_t smem = ring ? rows_smem : 0;
      if ((cta > g || few > 0) && smem < line * sizeof(float)) smem = line * sizeof(float);
      return with_row_width<T>(width, [&](auto wc) {
        constexpr int kW = decltype(wc)::value;
        auto launch = [&](auto kernel, std::atomic<unsigned long long>* configured) {
          cudaError_t e = allow_smem(kernel, kGradSmem, configured);
          if (e != cudaSuccess) return status_of(e);
          if (few > 0) return status_of(mns::launch_pdl_cluster(kernel, dim3(few), dim3(cta), smem, stream, few, R, g));
          return status_of(mns::launch_pdl(kernel, dim3(parts), dim3(cta), smem, stream, R, g));
        };
        static std::atomic<unsigned long long> done[4];
        if constexpr (kW * sizeof(T) >= 4)
          if (ring) return few > 0 ? launch(rms_norm_bwd<T, TW, kW, true, true>, &done[0])
                                   : launch(rms_norm_bwd<T, TW, kW, true, false>, &done[1]);
        return few > 0 ? launch(rms_norm_bwd<T, TW, kW, false, true>, &done[2])
                       : launch(rms_norm_bwd<T, TW, kW, false, false>, &done[3]);
      });
    });
  });
  if (st != MUON_NS_OK || few > 0) return st;
  return status_of(mns::launch_pdl(rms_norm_join, dim3(static_cast<unsigned>((dim + 31) / 32)), dim3(256), 0, stream,
                                   static_cast<const float*>(part), parts, dim, dweight));
}

}  // extern "C"
