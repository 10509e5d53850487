// Shared by layer norm's two passes: sums over the threads of a row, and how
// many threads a row takes.
#pragma once

#include "lm/common.cuh"

namespace mns {
namespace lm {

constexpr int kNormCta = 256;  // CTA size for groups up to it

// Sums of N values over the G threads of a group (a power of two from 8), the
// same values in each, in place.  `red` holds a float per value and warp of
// the CTA; callers alternate between two of them, so one barrier is enough.
template <int G, int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float (*red)[32]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (G <= 32) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][warp] = v[i];
  }
  __syncthreads();
  constexpr int kW = G > 32 ? G / 32 : 1;
  const int first = warp / kW * kW;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kW; ++w) v[i] += red[i][first + w];
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v, float (*red)[32]) {
  float a[1] = {v};
  group_sums<G, 1>(a, red);
  return a[0];
}

// The columns of a row that a thread of a group of G takes, in units of kU: the
// VEC elements of one access, or, where accesses are single, two elements G
// columns apart, so that arithmetic always has pairs.
template <int VEC, int G, int PER>
struct Cols {
  static constexpr int kU = VEC == 1 ? 2 : VEC;
  static constexpr int kK = PER / kU;  // units of a thread
  static constexpr int kP = kU / 2;    // pairs of a unit
  static __device__ __forceinline__ int first(int k, int tid) { return (VEC == 1 ? 2 * k * G : k * G * VEC) + (VEC == 1 ? tid : tid * VEC); }
  // Whether the unit's second single element is a column.
  static __device__ __forceinline__ bool second(int c, int dim) { return VEC > 1 || c + G < dim; }

  // From and to global memory, or (kShared) shared memory.
  template <bool kShared = false, typename T>
  static __device__ __forceinline__ Vec<T, kU> load(const T* row, int c, int dim) {
    if constexpr (VEC > 1) {
      return kShared ? load_vec<T, VEC>(row + c) : load_global<T, VEC>(row + c);
    } else {
      Vec<T, kU> v;
      v.v[0] = row[c];
      v.v[1] = second(c, dim) ? row[c + G] : T{};
      return v;
    }
  }
  template <bool kShared = false, typename T>
  static __device__ __forceinline__ void store(T* row, int c, int dim, const float2 (&f)[kP]) {
    if constexpr (VEC > 1) {
      float o[VEC];
      from_pairs<VEC>(f, o);
      if (kShared)
        store_vec<T, VEC>(row + c, o);
      else
        store_global<T, VEC>(row + c, o);
    } else {
      row[c] = from_f32<T>(f[0].x);
      if (second(c, dim)) row[c + G] = from_f32<T>(f[0].y);
    }
  }
  template <typename T>
  static __device__ __forceinline__ void copy(T* dst, const T* row, int c, int dim) {
    copy_async<VEC * sizeof(T)>(dst + c, row + c);
    if constexpr (VEC == 1) {
      if (second(c, dim)) copy_async<sizeof(T)>(dst + c + G, row + c + G);
    }
  }
};

// Rows of bf16 with an odd number of columns start on 2 bytes, less than
// cp.async can copy.  They are copied as the 4-byte words that cover them, by a
// group of G threads, to a buffer of word_pitch(dim) elements; the row then
// starts at element `row_shift` of it.  A word may hold an element of the row
// before or after; only the tensor's very last may lack its second half.
template <typename T, int VEC>
constexpr bool kByWords = VEC * sizeof(T) < 4;
MNS_HD int word_pitch(int dim) { return (dim + 3) & ~1; }
template <typename T>
__device__ __forceinline__ int row_shift(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 1u);
}
template <int G, typename T>
__device__ __forceinline__ void copy_words(T* dst, const T* base, long long row, long long rows, int dim, int tid) {
  const T* src = base + row * dim;
  const int shift = row_shift(src);
  const bool last = row == rows - 1;
  for (int i = 2 * tid; i < dim + shift; i += 2 * G) {
    if (last && i + 1 - shift >= dim)
      dst[i] = src[i - shift];
    else
      copy_async<4>(dst + i, src + i - shift);
  }
}
// Makes a group's copies (after its wait) visible to it, and its reads done.
template <int G>
__device__ __forceinline__ void group_barrier() {
  if (G > 32)
    __syncthreads();
  else
    __syncwarp();
}

// Threads a row takes with `per` elements each: 8 to 1024.
inline int group_of(int dim, int per) {
  int g = 8;
  while (g < 1024 && g * per < dim) g *= 2;
  return g;
}

template <typename F>
auto with_group(int g, F&& f) {
  switch (g) {
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 256: return f(std::integral_constant<int, 256>{});
    case 512: return f(std::integral_constant<int, 512>{});
    default: return f(std::integral_constant<int, 1024>{});
  }
}

// Widest vector for rows of x_type: 16 bytes, so that a warp's accesses are
// contiguous.
inline int norm_vec(int dim, const void* p, int x_type) {
  const int v = vec_of(dim, p, x_type);
  return x_type == MUON_LM_F32 && v > 4 ? 4 : v;
}

// Calls f with the vector widths that norm_vec gives rows of T.
template <typename T, typename F>
auto with_norm_vec(int vec, F&& f) {
  if constexpr (sizeof(T) == 2) {
    if (vec == 8) return f(std::integral_constant<int, 8>{});
  }
  switch (vec) {
    case 4: return f(std::integral_constant<int, 4>{});
    case 2: return f(std::integral_constant<int, 2>{});
    default: return f(std::integral_constant<int, 1>{});
  }
}

inline int norm_check(long long rows, int dim) {
  if (rows < 0 || dim < 0 || rows > kMaxRows || dim > kMaxDim) return MUON_NS_ERR_INVALID_ARG;
  if (rows > 0 && dim == 0) return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

}  // namespace lm
}  // namespace mns
