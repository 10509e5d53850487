// Rows in blocks of 128 columns, the blocks of 8-bit storage: how a group of
// threads holds a row, and a block's way into e4m3 with a scale.  (Here and in the
// other kernels of a block with experts no pointer is __restrict__: they start beside
// the kernel before them, so what that one writes is not read-only while they run.)
#pragma once

#include "lm/common.cuh"

namespace mns {
namespace lm {

constexpr int kBlock8 = 128;     // columns that share a scale
constexpr float kTop8 = 448.0f;  // largest e4m3 value
constexpr int kRowPer = 16;      // elements of a row that a thread holds

// A block of 128 columns is taken by kLanes lanes in accesses of W elements: 16
// lanes for 8 elements (16 bytes of bf16), a warp for fewer.
template <int W>
struct Blk {
  static constexpr int kLanes = W == 8 ? 16 : 32;
  static constexpr int kU = kBlock8 / kLanes;  // elements a lane holds of it
  static constexpr int kP = kU / W;            // accesses
  static constexpr int kK = kRowPer / kU;      // blocks a thread holds, at most
  static constexpr int kH = kU / 2;            // pairs: arithmetic is on two at once
  static __device__ __forceinline__ int col(int block, int lane, int p) {
    return block * kBlock8 + p * kLanes * W + lane * W;
  }
  template <typename T>
  static __device__ __forceinline__ void load(const T* row, int block, int lane, int dim, Vec<T, W> (&v)[kP]) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const int c = col(block, lane, p);
      if (c < dim)
        v[p] = load_global<T, W>(row + c);
      else
        v[p] = Vec<T, W>{};
    }
  }
  template <typename T>
  static __device__ __forceinline__ void store(T* row, int block, int lane, int dim, const float2 (&f)[kH]) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const int c = col(block, lane, p);
      float o[W];
#pragma unroll
      for (int i = 0; i < W; ++i) o[i] = (p * W + i) & 1 ? f[(p * W + i) / 2].y : f[(p * W + i) / 2].x;
      if (c < dim) store_global<T, W>(row + c, o);
    }
  }
  // As it was loaded.
  template <typename T>
  static __device__ __forceinline__ void put(T* row, int block, int lane, int dim, const Vec<T, W> (&v)[kP]) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const int c = col(block, lane, p);
      if (c < dim) *reinterpret_cast<Vec<T, W>*>(row + c) = v[p];
    }
  }
  template <typename T>
  static __device__ __forceinline__ void widen(const Vec<T, W> (&v)[kP], float2 (&f)[kH]) {
#pragma unroll
    for (int j = 0; j < kH; ++j)
      f[j] = make_float2(to_f32(v[2 * j / W].v[2 * j % W]), to_f32(v[(2 * j + 1) / W].v[(2 * j + 1) % W]));
  }
  // Rounded to T.
  template <typename T>
  static __device__ __forceinline__ void narrow(const float2 (&f)[kH], Vec<T, W> (&v)[kP]) {
#pragma unroll
    for (int j = 0; j < kU; ++j) v[j / W].v[j % W] = from_f32<T>(j & 1 ? f[j / 2].y : f[j / 2].x);
  }
};

// Larger magnitude of two; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}

// Largest magnitude of a lane's part of a block.
template <int H>
__device__ __forceinline__ float top_of(const float2 (&f)[H]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < H; ++j) m = max_nan(max_nan(m, f[j].x), f[j].y);
  return m;
}

// Largest of LANES lanes' magnitudes.  As integers a NaN is above everything, so it
// is not lost.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(float m) {
  uint32_t v = __float_as_uint(m) & 0x7FFFFFFFu;
  if constexpr (LANES == 32) {
    return __reduce_max_sync(0xFFFFFFFFu, v);
  } else {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      const uint32_t w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
      v = w > v ? w : v;
    }
    return v;
  }
}

// Scale of a block whose largest magnitude has these bits: NaN where the block
// holds a NaN or an infinity, 1 where it is all zero.  A scale below the normal
// numbers is rounded up: to nearest it could be a few steps too small for the
// block's largest values, or 0, which makes NaN of its zeros.
__device__ __forceinline__ float scale_of(uint32_t bits) {
  if (bits >= 0x7F800000u) return __uint_as_float(0x7FFFFFFFu);
  if (bits == 0u) return 1.0f;
  const float top = __uint_as_float(bits), scale = top / kTop8;
  return scale < 1.1754944e-38f ? __fdiv_ru(top, kTop8) : scale;
}

// e4m3 of a pair, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float2 f) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(f.y), "f"(f.x));
  return r;
}

// A lane's part of a block, in units of its scale, to rows of bytes.
template <int W>
__device__ __forceinline__ void put8(uint8_t* row, int block, int lane, int dim, const float2 (&q)[Blk<W>::kH]) {
  using B = Blk<W>;
#pragma unroll
  for (int p = 0; p < B::kP; ++p) {
    const int c = B::col(block, lane, p);
    if (c >= dim) continue;
    if constexpr (W == 8) {
      *reinterpret_cast<uint2*>(row + c) =
          make_uint2(e4m3x2(q[0]) | e4m3x2(q[1]) << 16, e4m3x2(q[2]) | e4m3x2(q[3]) << 16);
    } else if constexpr (W == 4) {
      *reinterpret_cast<uint32_t*>(row + c) = e4m3x2(q[0]) | e4m3x2(q[1]) << 16;
    } else if constexpr (W == 2) {
      *reinterpret_cast<uint16_t*>(row + c) = static_cast<uint16_t>(e4m3x2(q[p]));
    } else {
      row[c] = static_cast<uint8_t>(e4m3x2(q[p / 2]) >> (8 * (p & 1)));
    }
  }
}

// A lane's part of a block, divided by its scale, to rows of bytes.  The quotient
// is a product with the reciprocal, corrected once by what it leaves over
// (Markstein, IBM J. Res. Dev. 34, 1990), so that as few values as with a division
// fall to the other side of a rounding boundary; a division where the reciprocal
// would overflow.
template <int W>
__device__ __forceinline__ void store8(uint8_t* row, int block, int lane, int dim, const float2 (&f)[Blk<W>::kH],
                                       float scale) {
  using B = Blk<W>;
  const float inv = 1.0f / scale;
  float2 q[B::kH];
  if (scale < 1.1754944e-38f) {
#pragma unroll
    for (int j = 0; j < B::kH; ++j) q[j] = make_float2(f[j].x / scale, f[j].y / scale);
  } else {
#pragma unroll
    for (int j = 0; j < B::kH; ++j) {
      q[j] = mul2(f[j], both(inv));
      q[j] = fma2(fma2(q[j], both(-scale), f[j]), both(inv), q[j]);
    }
  }
  put8<W>(row, block, lane, dim, q);
}

// Sum over the g threads of a group (a power of two from 32 to the CTA's size),
// the same value in each.  `red` holds a float a warp; callers alternate between
// two of them, so one barrier is enough.
__device__ __forceinline__ float group_total(float v, int g, float* red) {
  v = warp_sum(v);
  if (g == 32) return v;
  const int warp = threadIdx.x >> 5, n = g >> 5, first = warp / n * n;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < n; ++w) v += red[first + w];
  return v;
}

// ------------------------------------------------------------------- host --

constexpr int kRowCta = 256;              // CTA size for groups up to it
constexpr int kRowMax = 1024 * kRowPer;   // longest row that a group holds

// Threads a row takes, whole warps.  `per`: elements of it that each holds.
inline int row_group(int dim, int per = kRowPer) {
  int g = 32;
  while (g < 1024 && g * per < dim) g *= 2;
  return g;
}

// Width of accesses to rows of `type`: 16 bytes, 2 elements or one, as the row
// length and the pointers (their addresses or-ed) allow.
inline int row_width(int dim, int type, uintptr_t pointers) {
  const int wide = type == MUON_LM_F32 ? 4 : 8;
  if (dim % wide == 0 && pointers % 16 == 0) return wide;
  return dim % 2 == 0 && pointers % (2 * type_size(type)) == 0 ? 2 : 1;
}

template <typename T, typename F>
auto with_row_width(int w, F&& f) {
  if (w == 2) return f(std::integral_constant<int, 2>{});
  if (w == 1) return f(std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, (sizeof(T) == 2 ? 8 : 4)>{});
}

}  // namespace lm
}  // namespace mns
