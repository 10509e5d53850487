// Shared by the memory-bound operators: element types, vectors of VEC
// elements (the widest that the row length and the pointers allow), rounding,
// and the host's choice between them.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gemm_launch.cuh"
#include "muon_lm.h"
#include "ptx.cuh"

namespace mns {
namespace lm {

using bf16 = uint16_t;  // raw bits, as muon_bf16

__device__ __forceinline__ float to_f32(bf16 v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// VEC consecutive elements, moved in one access (two for 8 fp32).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Vec {
  T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, VEC>*>(p);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  Vec<T, VEC> o;
#pragma unroll
  for (int j = 0; j < VEC; ++j) o.v[j] = from_f32<T>(f[j]);
  *reinterpret_cast<Vec<T, VEC>*>(p) = o;
}

// Token id at `t`, or -1 if it names no row of the table.
__device__ __forceinline__ long long load_id(const void* ids, int ids64, long long t, long long vocab) {
  const long long v = ids64 ? static_cast<const long long*>(ids)[t]
                            : static_cast<long long>(static_cast<const int*>(ids)[t]);
  return (v >= 0 && v < vocab) ? v : -1;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ------------------------------------------------------------------- host --

constexpr long long kMaxRows = 1LL << 30;
constexpr int kMaxDim = 1 << 20;

inline int type_size(int type) { return type == MUON_LM_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == MUON_LM_BF16 || type == MUON_LM_F32; }

inline bool element_aligned(const void* p, int type) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(type_size(type) - 1)) == 0;
}

// Widest vector (8, 4, 2 or 1 elements) with which rows of `dim` elements can
// be walked through `p`: dim a multiple of it, and p aligned to its bytes (to
// 16 where 8 fp32 take two accesses).
inline int vec_of(int dim, const void* p, int type) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  for (int v = 8; v > 1; v >>= 1) {
    int bytes = v * type_size(type);
    if (bytes > 16) bytes = 16;
    if (dim % v == 0 && (a & static_cast<uintptr_t>(bytes - 1)) == 0) return v;
  }
  return 1;
}

inline int min_vec(int a, int b) { return a < b ? a : b; }

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

inline int status_of(cudaError_t e) {
  if (e == cudaSuccess) return MUON_NS_OK;
  cudaGetLastError();
  return MUON_NS_ERR_CUDA;
}

// SMs of the current device (queried once per device).
int sm_count();

// Calls f with a std::integral_constant of the vector width.
template <typename F>
auto with_vec(int vec, F&& f) {
  switch (vec) {
    case 8: return f(std::integral_constant<int, 8>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 2: return f(std::integral_constant<int, 2>{});
    default: return f(std::integral_constant<int, 1>{});
  }
}

// Calls f with a value of the element type, as a tag.
template <typename F>
auto with_type(int type, F&& f) {
  return type == MUON_LM_F32 ? f(float{}) : f(bf16{});
}

}  // namespace lm
}  // namespace mns
