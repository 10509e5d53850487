// Root-mean-square norm with the residual's addition.  Per row, with the sum
// rounded to the rows' type and kept:
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w,
// y in the rows' type, or in e4m3 with a scale for each 128 columns.
//
// A group of 32 to 1024 threads holds a row in registers, 16 elements a thread,
// so that x and the residual are read once and s and y written once, in blocks of
// 128 columns by 16 or 32 lanes: a block's largest magnitude takes shuffles alone.
// Bound by HBM traffic.  Longer rows take the _long kernel, which reads s again
// from cache.
#include <cmath>

#include "lm/block8.cuh"
#include "muon_moe.h"

namespace mns {
namespace lm {

namespace {

template <typename T, typename TW>
struct RmsRows {
  const T* x;
  const T* residual;  // or null
  const TW* w;
  long long rows;
  int dim;
  float inv_dim, eps;
  T* s;      // or null
  void* y;   // T, or bytes
  float* scales;
  float* rstd;  // or null
};

// WIDE: a row takes more than kRowCta threads.  (Five CTAs an SM: with four, 32768
// x 4096 of bf16 took 162 us for 152, with six 160.)
template <typename T, typename TW, int W, bool OUT8, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : kRowCta, WIDE ? 1 : 5)
    rms_norm_fwd(const RmsRows<T, TW> R, int g) {
  using B = Blk<W>;
  __shared__ float red[32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x & (g - 1), lane = tid & (B::kLanes - 1), first = tid / B::kLanes, step = g / B::kLanes;
  const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / g) + threadIdx.x / g;
  const bool live = row < R.rows;
  const long long at = row * R.dim;
  float2 f[B::kK][B::kH];
  float2 sq = both(0.0f);
  if (live) {
    Vec<T, W> v[B::kK][B::kP], a[B::kK][B::kP];
#pragma unroll
    for (int k = 0; k < B::kK; ++k) {
      B::load(R.x + at, first + k * step, lane, R.dim, v[k]);
      if (R.residual != nullptr) B::load(R.residual + at, first + k * step, lane, R.dim, a[k]);
    }
#pragma unroll
    for (int k = 0; k < B::kK; ++k) {
      B::widen(v[k], f[k]);
      if (R.residual != nullptr) {
        // The residual stream's rounding to its type: what is kept is what is
        // normalised, so that the gradient sees the same rows.
        float2 b[B::kH];
        B::widen(a[k], b);
#pragma unroll
        for (int j = 0; j < B::kH; ++j) f[k][j] = add2(f[k][j], b[j]);
        B::narrow(f[k], v[k]);
        if (R.s != nullptr) B::put(R.s + at, first + k * step, lane, R.dim, v[k]);
        B::widen(v[k], f[k]);
      }
#pragma unroll
      for (int j = 0; j < B::kH; ++j) sq = fma2(f[k][j], f[k][j], sq);
    }
  }
  const float r = 1.0f / sqrtf(group_total(sq.x + sq.y, g, red) * R.inv_dim + R.eps);
  if (live && tid == 0 && R.rstd != nullptr) R.rstd[row] = r;
  if (OUT8 && !(r > 0.0f && r < INFINITY)) {
#pragma unroll
    for (int k = 0; k < B::kK; ++k)
#pragma unroll
      for (int j = 0; j < B::kH; ++j) f[k][j] = mul2(f[k][j], both(r));
  }
#pragma unroll
  for (int k = 0; k < B::kK; ++k) {
    const int block = first + k * step;
    Vec<TW, W> wv[B::kP];
    float2 w[B::kH];
    B::load(R.w, block, lane, R.dim, wv);
    B::widen(wv, w);
    if (OUT8) {
      // r is in the scale alone; a block's values in units of it are p 448 / top,
      // p = s w.  Both factors are carried with what their rounding left over, so
      // that the quotient is rounded once before its own way into 8 bits.
      float2 q[B::kH];
#pragma unroll
      for (int j = 0; j < B::kH; ++j) {
        const float2 p = mul2(f[k][j], w[j]);
        w[j] = fma2(f[k][j], w[j], make_float2(-p.x, -p.y));
        f[k][j] = p;
      }
      // (Past the row's end stands 0: NaN only where all of the row is.)
      const uint32_t bits = lanes_max<B::kLanes>(live ? top_of(f[k]) : 0.0f);
      float top = __uint_as_float(bits), scale = top * r * (1.0f / kTop8);
      if (top < 0x1p-80f) {  // (448 / top would overflow)
        if (bits == 0u) scale = 1.0f;
        top = bits == 0u ? 1.0f : top * 0x1p64f;
#pragma unroll
        for (int j = 0; j < B::kH; ++j) f[k][j] = mul2(f[k][j], both(0x1p64f)), w[j] = mul2(w[j], both(0x1p64f));
      }
      const float a = kTop8 / top, a_lo = fmaf(-a, top, kTop8) * (a * (1.0f / kTop8));
#pragma unroll
      for (int j = 0; j < B::kH; ++j)
        q[j] = fma2(f[k][j], both(a), fma2(f[k][j], both(a_lo), mul2(w[j], both(a))));
      if (live && block * kBlock8 < R.dim) {
        put8<W>(static_cast<uint8_t*>(R.y) + at, block, lane, R.dim, q);
        if (lane == 0)
          R.scales[row * ((R.dim + kBlock8 - 1) / kBlock8) + block] = scale < INFINITY ? scale : __uint_as_float(0x7FFFFFFFu);
      }
    } else if (live) {
#pragma unroll
      for (int j = 0; j < B::kH; ++j) f[k][j] = mul2(mul2(f[k][j], both(r)), w[j]);
      B::store(static_cast<T*>(R.y) + at, block, lane, R.dim, f[k]);
    }
  }
}

// Rows of more than kRowMax elements: a CTA a row, a warp a block.
template <typename T, typename TW, bool OUT8>
__global__ void __launch_bounds__(1024) rms_norm_fwd_long(const RmsRows<T, TW> R) {
  __shared__ float red[2][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, blocks = (R.dim + kBlock8 - 1) / kBlock8;
  int buf = 0;
  for (long long row = blockIdx.x; row < R.rows; row += gridDim.x, buf ^= 1) {
    const T *xr = R.x + row * R.dim, *ar = R.residual == nullptr ? nullptr : R.residual + row * R.dim;
    auto sum = [&](int c) {
      const float v = to_f32(xr[c]);
      return ar == nullptr ? v : to_f32(from_f32<T>(v + to_f32(ar[c])));
    };
    float sq = 0.0f;
    for (int c = threadIdx.x; c < R.dim; c += 1024) {
      const float v = sum(c);
      sq = fmaf(v, v, sq);
    }
    const float r = 1.0f / sqrtf(group_total(sq, 1024, red[buf]) * R.inv_dim + R.eps);
    if (threadIdx.x == 0 && R.rstd != nullptr) R.rstd[row] = r;
    for (int b = threadIdx.x >> 5; b < blocks; b += 32) {
      float f[4];
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = b * kBlock8 + j * 32 + lane;
        f[j] = 0.0f;
        if (c < R.dim) {
          const float v = sum(c);
          // (x and the residual of this element have been read: s or y may be
          // either.)
          if (R.s != nullptr && ar != nullptr) R.s[row * R.dim + c] = from_f32<T>(v);
          f[j] = v * r * to_f32(R.w[c]);
          top = max_nan(top, f[j]);
          if (!OUT8) static_cast<T*>(R.y)[row * R.dim + c] = from_f32<T>(f[j]);
        }
      }
      if (OUT8) {
        const float scale = scale_of(lanes_max<32>(top));
        const float2 pairs[2] = {make_float2(f[0], f[1]), make_float2(f[2], f[3])};
        store8<1>(static_cast<uint8_t*>(R.y) + row * R.dim, b, lane, R.dim, pairs, scale);
        if (lane == 0) R.scales[row * blocks + b] = scale;
      }
    }
  }
}

int rms_check(long long rows, int dim) {
  if (rows < 0 || dim < 0 || rows > kMaxRows || dim > kMaxDim) return MUON_NS_ERR_INVALID_ARG;
  if (rows > 0 && dim == 0) return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

bool f32_aligned(const void* p) { return element_aligned(p, MUON_LM_F32); }

int run_norm(const void* x, int x_type, const void* residual, const void* weight, int w_type, long long rows, int dim,
             float eps, void* s, void* y, float* scales, float* rstd, bool out8, cudaStream_t stream) {
  int st = rms_check(rows, dim);
  if (st != MUON_NS_OK) return st;
  if (!type_ok(x_type) || !type_ok(w_type) || !(eps >= 0.0f) || !std::isfinite(eps)) return MUON_NS_ERR_INVALID_ARG;
  if (rows == 0) return MUON_NS_OK;
  if (!x || !weight || !y || (out8 && !scales)) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(x, x_type) || !element_aligned(residual, x_type) || !element_aligned(s, x_type) ||
      !element_aligned(weight, w_type) || (!out8 && !element_aligned(y, x_type)) || !f32_aligned(scales) || !f32_aligned(rstd))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t xb = static_cast<size_t>(rows) * dim * type_size(x_type), qb = static_cast<size_t>(rows) * dim;
  // Where the outputs may lie over the inputs they do so element by element.
  if (residual && s && overlap(s, xb, x, xb) && s != x) return MUON_NS_ERR_INVALID_ARG;
  if (residual && s && overlap(s, xb, residual, xb) && s != residual) return MUON_NS_ERR_INVALID_ARG;
  if (residual && s && overlap(s, xb, y, out8 ? qb : xb)) return MUON_NS_ERR_INVALID_ARG;
  if (out8 ? overlap(y, qb, x, xb) : overlap(y, xb, x, xb) && y != x) return MUON_NS_ERR_INVALID_ARG;
  if (residual && (out8 ? overlap(y, qb, residual, xb) : overlap(y, xb, residual, xb) && y != residual))
    return MUON_NS_ERR_INVALID_ARG;
  const size_t blocks = (static_cast<size_t>(dim) + kBlock8 - 1) / kBlock8;
  const Span rows_x = {x, xb}, rows_a = {residual, xb}, rows_s = {residual ? s : nullptr, xb}, rows_y = {y, out8 ? qb : xb},
             w = {weight, static_cast<size_t>(dim) * type_size(w_type)}, rs = {rstd, 4 * static_cast<size_t>(rows)},
             sc = {out8 ? scales : nullptr, 4 * blocks * rows};
  if (overlaps(w, {rows_s, rows_y, rs, sc}) || overlaps(rs, {rows_x, rows_a, rows_s, rows_y, sc}) ||
      overlaps(sc, {rows_x, rows_a, rows_s, rows_y}))
    return MUON_NS_ERR_INVALID_ARG;
  if ((st = muon_ns_device_supported(-1)) != MUON_NS_OK) return st;
  return with_type(x_type, [&](auto xt) {
    return with_type(w_type, [&](auto wt) {
      using T = decltype(xt);
      using TW = decltype(wt);
      RmsRows<T, TW> R = {};
      R.x = static_cast<const T*>(x);
      R.residual = static_cast<const T*>(residual);
      R.w = static_cast<const TW*>(weight);
      R.rows = rows;
      R.dim = dim;
      R.inv_dim = 1.0f / static_cast<float>(dim);
      R.eps = eps;
      R.s = static_cast<T*>(s);
      R.y = y;
      R.scales = scales;
      R.rstd = rstd;
      if (dim > kRowMax) {
        const unsigned grid = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
        return status_of(mns::launch_pdl(out8 ? rms_norm_fwd_long<T, TW, true> : rms_norm_fwd_long<T, TW, false>,
                                         dim3(grid), dim3(1024), 0, stream, R));
      }
      const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
      int width = row_width(dim, x_type, at(x) | at(residual) | at(s) | (out8 ? at(y) * type_size(x_type) : at(y)));
      // Weights are read 32 bytes at most, whatever the rows' type.
      while (width > 1 && at(weight) % (width * type_size(w_type) > 16 ? 32 : width * type_size(w_type)) != 0)
        width = width > 2 ? 2 : 1;
      const int g = row_group(dim), cta = g > kRowCta ? g : kRowCta;
      const unsigned grid = static_cast<unsigned>((rows + cta / g - 1) / (cta / g));
      return with_row_width<T>(width, [&](auto wc) {
        constexpr int kW = decltype(wc)::value;
        if (cta > kRowCta)
          return status_of(mns::launch_pdl(out8 ? rms_norm_fwd<T, TW, kW, true, true> : rms_norm_fwd<T, TW, kW, false, true>,
                                           dim3(grid), dim3(cta), 0, stream, R, g));
        return status_of(mns::launch_pdl(out8 ? rms_norm_fwd<T, TW, kW, true, false> : rms_norm_fwd<T, TW, kW, false, false>,
                                         dim3(grid), dim3(cta), 0, stream, R, g));
      });
    });
  });
}

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_rms_norm(const void* x, int x_type, const void* residual, const void* weight, int w_type, long long rows,
                  int dim, float eps, void* s, void* y, float* rstd, cudaStream_t stream) {
  return run_norm(x, x_type, residual, weight, w_type, rows, dim, eps, s, y, nullptr, rstd, false, stream);
}

int muon_rms_norm8(const void* x, int x_type, const void* residual, const void* weight, int w_type, long long rows,
                   int dim, float eps, void* s, void* y, float* scales, float* rstd, cudaStream_t stream) {
  return run_norm(x, x_type, residual, weight, w_type, rows, dim, eps, s, y, scales, rstd, true, stream);
}

}  // extern "C"
