// The weighted sum that brings the experts' rows back to their tokens, and its
// gradient:
//   out[t] = sum_j gates[t][j] y[slots[t][j]]   (fp32, in the order of j),
//   dy[slots[t][j]] = gates[t][j] dout[t],  dgates[t][j] = <dout[t], y[slots[t][j]]>.
// A slot outside the rows is left out.  Without gates they are 1: then the sum is
// the gradient of the tokens' dispatch to their rows.  Gathers and scatters of
// whole rows, bound by HBM traffic; no row is named twice, so nothing is added in
// memory.
#include "lm/common.cuh"
#include "muon_moe.h"

namespace mns {
namespace lm {

namespace {

constexpr int kCombineMost = 32;  // rows of a token

struct Combine {
  const int* slots;
  const float* gates;  // or null
  long long tokens, rows;
  int k, dim;
};

__device__ __forceinline__ int slot_of(const Combine& C, long long i) {
  const int s = C.slots[i];
  return s >= 0 && s < C.rows ? s : -1;
}

// Threads x of a CTA take VEC columns each, y of them tokens.  KB rows of a token
// are on their way at once (a token's k of up to 8: with 8 whatever the k, 4 of
// 2048 columns held twice the registers and took 90 us for 55 at 16384 tokens).
template <typename T, int VEC, int KB>
__global__ void __launch_bounds__(256) combine_fwd(const Combine C, const T* y, T* out) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (c >= C.dim || t >= C.tokens) return;
  float o[VEC] = {};
  for (int j0 = 0; j0 < C.k; j0 += KB) {
    Vec<T, VEC> v[KB];
    float g[KB];
    int s[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      s[j] = j0 + j < C.k ? slot_of(C, t * C.k + j0 + j) : -1;
      g[j] = s[j] >= 0 && C.gates != nullptr ? C.gates[t * C.k + j0 + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (s[j] >= 0) v[j] = load_global<T, VEC>(y + static_cast<long long>(s[j]) * C.dim + c);
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (s[j] >= 0) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = fmaf(g[j], to_f32(v[j].v[i]), o[i]);
      }
  }
  store_global<T, VEC>(out + t * C.dim + c, o);
}

// SPLIT warps of a CTA share a token (few tokens), or each takes one.
template <typename T, int VEC, int SPLIT, int KB>
__global__ void __launch_bounds__(256)
    combine_bwd(const Combine C, const T* dout, const T* y, T* dy,
                float* dgates) {
  __shared__ float red[8][KB];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % SPLIT;
  const long long t = static_cast<long long>(blockIdx.x) * (8 / SPLIT) + warp / SPLIT;
  const bool live = t < C.tokens;
  if (SPLIT == 1 && !live) return;
  for (int j0 = 0; j0 < C.k; j0 += KB) {
    float g[KB], dot[KB];
    int s[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      s[j] = live && j0 + j < C.k ? slot_of(C, t * C.k + j0 + j) : -1;
      g[j] = s[j] >= 0 && C.gates != nullptr ? C.gates[t * C.k + j0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int c = (part * 32 + lane) * VEC; live && c < C.dim; c += SPLIT * 32 * VEC) {
      const Vec<T, VEC> d = load_global<T, VEC>(dout + t * C.dim + c);
      Vec<T, VEC> v[KB];
      if (dgates != nullptr) {
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (s[j] >= 0) v[j] = load_global<T, VEC>(y + static_cast<long long>(s[j]) * C.dim + c);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (s[j] < 0) continue;
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          o[i] = g[j] * to_f32(d.v[i]);
          if (dgates != nullptr) dot[j] = fmaf(to_f32(d.v[i]), to_f32(v[j].v[i]), dot[j]);
        }
        if (dy != nullptr) store_global<T, VEC>(dy + static_cast<long long>(s[j]) * C.dim + c, o);
      }
    }
    if (dgates == nullptr) continue;
#pragma unroll
    for (int j = 0; j < KB; ++j) dot[j] = warp_sum(dot[j]);
    if (SPLIT > 1) {
      __syncthreads();  // the last batch's sums have been read
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < KB; ++j) red[warp][j] = dot[j];
      }
      __syncthreads();
    }
    if (live && part == 0 && lane < KB && j0 + lane < C.k) {
      float v = 0.0f;
      if (SPLIT > 1) {
#pragma unroll
        for (int w = 0; w < SPLIT; ++w) v += red[warp + w][lane];
      } else {
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (lane == j) v = dot[j];
      }
      dgates[t * C.k + j0 + lane] = v;
    }
  }
}

int combine_check(long long tokens, int k, long long rows, int dim, int type) {
  if (tokens < 0 || tokens > kMaxRows || k < 1 || k > kCombineMost || rows < 0 || rows > kMaxRows || dim < 0 || dim > kMaxDim ||
      !type_ok(type))
    return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

// Rows in flight: those of a token, up to 8.
template <typename F>
auto with_batch(int k, F&& f) {
  if (k <= 2) return f(std::integral_constant<int, 2>{});
  if (k <= 4) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{});
}

bool f32_aligned(const void* p) { return element_aligned(p, MUON_LM_F32); }

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_combine(const void* y, int type, const int* slots, const float* gates, long long tokens, int k, long long rows,
                 int dim, void* out, cudaStream_t stream) {
  int st = combine_check(tokens, k, rows, dim, type);
  if (st != MUON_NS_OK) return st;
  if (tokens == 0 || dim == 0) return MUON_NS_OK;
  if ((rows > 0 && !y) || !slots || !out) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(y, type) || !element_aligned(out, type) || !f32_aligned(slots) || !f32_aligned(gates))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t yb = static_cast<size_t>(rows) * dim * type_size(type), ob = static_cast<size_t>(tokens) * dim * type_size(type);
  const size_t sb = 4 * static_cast<size_t>(tokens) * k;
  if (overlap(out, ob, y, yb) || overlap(out, ob, slots, sb) || (gates && overlap(out, ob, gates, sb)))
    return MUON_NS_ERR_INVALID_ARG;
  if ((st = muon_ns_device_supported(-1)) != MUON_NS_OK) return st;
  const Combine C = {slots, gates, tokens, rows, k, dim};
  return with_type(type, [&](auto tt) {
    using T = decltype(tt);
    return with_vec(min_vec(vec_of(dim, y, type), vec_of(dim, out, type)), [&](auto vc) {
      constexpr int V = decltype(vc)::value;
      const int vecs = (dim + V - 1) / V;
      int x = 8;
      while (x < 256 && x < vecs) x *= 2;
      const dim3 block(x, 256 / x);
      const dim3 grid(static_cast<unsigned>((tokens + block.y - 1) / block.y), static_cast<unsigned>((vecs + x - 1) / x));
      return with_batch(k, [&](auto bc) {
        return status_of(mns::launch_pdl(combine_fwd<T, V, decltype(bc)::value>, grid, block, 0, stream, C,
                                         static_cast<const T*>(y), static_cast<T*>(out)));
      });
    });
  });
}

int muon_combine_grad(const void* dout, const void* y, int type, const int* slots, const float* gates, long long tokens,
                      int k, long long rows, int dim, void* dy, float* dgates, cudaStream_t stream) {
  int st = combine_check(tokens, k, rows, dim, type);
  if (st != MUON_NS_OK) return st;
  if (tokens == 0 || (!dy && !dgates)) return MUON_NS_OK;
  if (!slots || (dim > 0 && !dout) || (dgates && rows > 0 && dim > 0 && !y)) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(dout, type) || !element_aligned(y, type) || !element_aligned(dy, type) || !f32_aligned(slots) ||
      !f32_aligned(gates) || !f32_aligned(dgates))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t yb = static_cast<size_t>(rows) * dim * type_size(type), ob = static_cast<size_t>(tokens) * dim * type_size(type);
  const size_t sb = 4 * static_cast<size_t>(tokens) * k;
  if (dy && (overlap(dy, yb, dout, ob) || (dgates && y && overlap(dy, yb, y, yb)) || overlap(dy, yb, slots, sb) ||
             (gates && overlap(dy, yb, gates, sb)) || (dgates && overlap(dy, yb, dgates, sb))))
    return MUON_NS_ERR_INVALID_ARG;
  if (overlaps({dgates, sb}, {{slots, sb}, {gates, sb}, {dout, ob}, {y, yb}})) return MUON_NS_ERR_INVALID_ARG;
  if ((st = muon_ns_device_supported(-1)) != MUON_NS_OK) return st;
  const Combine C = {slots, gates, tokens, rows, k, dim};
  return with_type(type, [&](auto tt) {
    using T = decltype(tt);
    const T *dp = static_cast<const T*>(dout), *yp = static_cast<const T*>(y);
    T* op = static_cast<T*>(dy);
    int vec = vec_of(dim, dout, type);
    if (dgates) vec = min_vec(vec, vec_of(dim, y, type));
    if (dy) vec = min_vec(vec, vec_of(dim, dy, type));
    return with_vec(vec, [&](auto vc) {
      constexpr int V = decltype(vc)::value;
      return with_batch(k, [&](auto bc) {
        constexpr int KB = decltype(bc)::value;
        // A warp a token would leave SMs without one.  (A CTA and a warp a token: 64
        // tokens, k 8, 2048 columns 3.2 us and 10.7; 608: 6.6 and 10.8; 2000: 26.0 and
        // 24.6; 4 of 7168 at 2000 tokens 41.7 and 50.9, but 2 of 768 5.0 and 4.0.)
        if (tokens < 16LL * sm_count())
          return status_of(mns::launch_pdl(combine_bwd<T, V, 8, KB>, dim3(static_cast<unsigned>(tokens)), dim3(256), 0, stream, C,
                                           dp, yp, op, dgates));
        return status_of(mns::launch_pdl(combine_bwd<T, V, 1, KB>, dim3(static_cast<unsigned>((tokens + 7) / 8)), dim3(256), 0,
                                         stream, C, dp, yp, op, dgates));
      });
    });
  });
}

}  // extern "C"
