// Rows and weight blocks into 8-bit storage: e4m3 values and fp32 scales, a scale
// for each 128 columns of a row or each 128 x 128 block of a matrix.  Bound by HBM
// traffic.
#include "lm/block8.cuh"
#include "muon_moe.h"

namespace mns {
namespace lm {

namespace {

// `rows` x dim in bands of BAND rows (1, or 128 that share their scales): a CTA
// takes 128 columns of a band, a warp every 8th of its rows.  With BAND 1 its rows
// are 64 bands.
template <typename T, int W, int BAND>
__global__ void __launch_bounds__(256)
    quantize8(const T* x, long long rows, int dim, uint8_t* q, float* scales) {
  using B = Blk<W>;
  constexpr int kTake = 32 / B::kLanes;  // rows a warp takes at once
  constexpr int kRows = BAND > 1 ? BAND : 64;
  constexpr int kTurns = kRows / (8 * kTake);
  __shared__ uint32_t red[8];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & (B::kLanes - 1), sub = (threadIdx.x & 31) / B::kLanes;
  const int block = blockIdx.x, blocks = gridDim.x;
  // Matrices of `rows` rows each along z; single rows are one matrix.
  const long long bands = (rows + kRows - 1) / kRows;
  const long long m = blockIdx.z, base = m * rows * dim;
  for (long long band = blockIdx.y; band < bands; band += gridDim.y) {
    Vec<T, W> v[kTurns][B::kP];
    float top[kTurns];
    float most = 0.0f;
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      const long long row = band * kRows + (t * 8 + warp) * kTake + sub;
#pragma unroll
      for (int p = 0; p < B::kP; ++p) v[t][p] = Vec<T, W>{};
      if (row < rows) B::load(x + base + row * dim, block, lane, dim, v[t]);
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      float2 f[B::kH];
      B::widen(v[t], f);
      top[t] = top_of(f);
      most = max_nan(most, top[t]);
    }
    uint32_t all = 0u;
    if (BAND > 1) {
      all = lanes_max<32>(most);
      if ((threadIdx.x & 31) == 0) red[warp] = all;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) all = red[w] > all ? red[w] : all;
      __syncthreads();
      if (threadIdx.x == 0) scales[(m * bands + band) * blocks + block] = scale_of(all);
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
      const long long row = band * kRows + (t * 8 + warp) * kTake + sub;
      const float scale = scale_of(BAND > 1 ? all : lanes_max<B::kLanes>(top[t]));
      if (row < rows) {
        float2 f[B::kH];
        B::widen(v[t], f);
        store8<W>(q + base + row * dim, block, lane, dim, f, scale);
        if (BAND == 1 && lane == 0) scales[row * blocks + block] = scale;
      }
    }
  }
}

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" int muon_quantize8(const void* x, int x_type, long long batch, long long rows, int dim, int square, void* q,
                              float* scales, cudaStream_t stream) {
  if (batch < 0 || rows < 0 || dim < 0 || batch > 65535 || rows > kMaxRows || dim > kMaxDim) return MUON_NS_ERR_INVALID_ARG;
  if (!type_ok(x_type) || (square != 0 && square != 1)) return MUON_NS_ERR_INVALID_ARG;
  if (batch == 0 || rows == 0 || dim == 0) return MUON_NS_OK;
  if (!x || !q || !scales) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(x, x_type) || !element_aligned(scales, MUON_LM_F32)) return MUON_NS_ERR_ALIGNMENT;
  const size_t n = static_cast<size_t>(batch) * rows * dim;
  const size_t lines = static_cast<size_t>(batch) * (square ? (rows + kBlock8 - 1) / kBlock8 : rows);
  const Span in = {x, n * type_size(x_type)}, sc = {scales, 4 * lines * ((static_cast<size_t>(dim) + kBlock8 - 1) / kBlock8)};
  if (overlaps({q, n}, {in, sc}) || overlaps(in, {sc})) return MUON_NS_ERR_INVALID_ARG;
  const int st = muon_ns_device_supported(-1);
  if (st != MUON_NS_OK) return st;
  // Single rows are one matrix whatever the stack.
  const long long all = square ? rows : batch * rows;
  const unsigned z = square ? static_cast<unsigned>(batch) : 1u;
  const long long bands = (all + (square ? 127 : 63)) / (square ? 128 : 64);
  const dim3 grid(static_cast<unsigned>((dim + kBlock8 - 1) / kBlock8), static_cast<unsigned>(bands < 65535 ? bands : 65535), z);
  return with_type(x_type, [&](auto xt) {
    using T = decltype(xt);
    const uintptr_t p = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(q) * type_size(x_type);
    return with_row_width<T>(row_width(dim, x_type, p), [&](auto wc) {
      constexpr int kW = decltype(wc)::value;
      return status_of(mns::launch_pdl(square ? quantize8<T, kW, 128> : quantize8<T, kW, 1>, grid, dim3(256), 0, stream,
                                       static_cast<const T*>(x), all, dim, static_cast<uint8_t*>(q), scales));
    });
  });
}
