// Shared by the memory-bound operators: element types, vectors of VEC
// elements (the widest that the row length and the pointers allow), rounding,
// and the host's choice between them.
#pragma once

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

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

// VEC consecutive elements.
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

// The same in global memory, where 8 fp32 are one 32-byte access (sm_100 and
// later): as two of 16 bytes, lanes 32 bytes apart would use half of each line
// an instruction touches.
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_global(const T* p) {
  if constexpr (sizeof(T) * VEC == 32) {
    Vec<float, 8> v;
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v.v[0]), "=f"(v.v[1]), "=f"(v.v[2]), "=f"(v.v[3]), "=f"(v.v[4]), "=f"(v.v[5]), "=f"(v.v[6]),
                   "=f"(v.v[7])
                 : "l"(p));
    return v;
  } else {
    return load_vec<T, VEC>(p);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_global(T* p, const float (&f)[VEC]) {
  if constexpr (sizeof(T) * VEC == 32)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
  else
    store_vec<T, VEC>(p, f);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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

// Two fp32 operations in one instruction (sm_100 and later); each half rounds
// as the scalar operation does.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The vector as pairs.
template <typename T, int VEC>
__device__ __forceinline__ void to_pairs(const Vec<T, VEC>& v, float2 (&p)[VEC / 2]) {
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) p[j] = make_float2(to_f32(v.v[2 * j]), to_f32(v.v[2 * j + 1]));
}
template <int VEC>
__device__ __forceinline__ void from_pairs(const float2 (&f)[VEC / 2], float (&o)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) o[j] = (j & 1) ? f[j / 2].y : f[j / 2].x;
}

// cp.async of BYTES (4, 8, 16 or 32) to shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  constexpr int kOne = BYTES > 16 ? 16 : BYTES;
#pragma unroll
  for (int i = 0; i < BYTES; i += kOne)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(static_cast<uint8_t*>(dst) + i)),
                 "l"(static_cast<const uint8_t*>(src) + i), "n"(kOne)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------- host --

constexpr long long kMaxRows = 1LL << 30;
constexpr int kMaxDim = 1 << 20;
// SMs of a GB300, for what is settled without a device to ask: workspace sizes,
// the grids that fill them, and the head's splits.  Fewer SMs would take the same
// grids in more turns.
constexpr int kSms = 152;

inline int type_size(int type) { return type == MUON_LM_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type == MUON_LM_BF16 || type == MUON_LM_F32; }

inline bool element_aligned(const void* p, int type) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(type_size(type) - 1)) == 0;
}

// Widest vector (8, 4, 2 or 1 elements) with which rows of `dim` elements can
// be walked through `p`: dim a multiple of it, and p aligned to its bytes.
inline int vec_of(int dim, const void* p, int type) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  for (int v = 8; v > 1; v >>= 1)
    if (dim % v == 0 && (a & static_cast<uintptr_t>(v * type_size(type) - 1)) == 0) return v;
  return 1;
}

inline int min_vec(int a, int b) { return a < b ? a : b; }

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// An array of a call.  Null and empty ones overlap nothing.
struct Span {
  const void* p;
  size_t n;
};
inline bool overlaps(Span a, std::initializer_list<Span> others) {
  if (!a.p || a.n == 0) return false;
  for (const Span& b : others)
    if (b.p && b.n > 0 && overlap(a.p, a.n, b.p, b.n)) return true;
  return false;
}

inline int status_of(cudaError_t e) {
  if (e == cudaSuccess) return MUON_NS_OK;
  cudaGetLastError();
  return MUON_NS_ERR_CUDA;
}

// Allows `kernel` as much dynamic shared memory, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>* configured) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (configured->load() >> (dev & 63) & 1ull)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) configured->fetch_or(1ull << (dev & 63));
  return e;
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
