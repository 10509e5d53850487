// The products grouped by expert: argument checks, tensor maps and launches of
// experts_gemm.cuh.  Compute-bound past about 300 rows an expert (2 rows flops a
// weight against 2 bytes of it); below that by reading W, and the gradient by
// writing dW.
#include <atomic>
#include <cmath>

#include <cudaTypedefs.h>

#include "lm/common.cuh"
#include "lm/experts_gemm.cuh"
#include "muon_moe.h"

namespace mns {
namespace lm {

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Map over batch x rows x inner contiguous elements, boxes with the 128-byte swizzle.
bool map3d(CUtensorMap* map, const void* base, CUtensorMapDataType type, int bytes, long long inner, long long rows,
           long long batch, int box_inner, int box_rows) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(mns::tensor_map_encoder());
  if (!fn) return false;
  const cuuint64_t line = static_cast<cuuint64_t>(inner) * bytes;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {line, line * rows};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_bf16(CUtensorMap* map, const void* base, long long inner, long long rows, long long batch, int box_rows) {
  return map3d(map, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, inner, rows, batch, 64, box_rows);
}
// The rows that are the MMA's N, K-major: boxes of 128, 64, 32 and 16 of them.
bool map_rows(CUtensorMap (&map)[kExpBoxes], const void* base, bool f8, long long inner, long long rows) {
  for (int i = 0; i < kExpBoxes; ++i)
    if (!(f8 ? map3d(&map[i], base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, inner, rows, 1, 128, 128 >> i)
             : map_bf16(&map[i], base, inner, rows, 1, 128 >> i)))
      return false;
  return true;
}

template <int MODE>
cudaError_t launch_experts(const ExpertsParam<MODE>& P, long long units, cudaStream_t stream) {
  constexpr int kSmem = ExpSmem<MODE>::kBytes;
  static std::atomic<int> resident[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int most = resident[dev & 63].load();
  if (most == 0) {
    e = cudaFuncSetAttribute(experts_gemm<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // A build that spills registers is not run.  TMEM loads write their registers some
    // time after they are issued, and a build of the 8-bit form that spilled around
    // them ended in a launch failure.  That the spilling was the cause is a suspicion:
    // the same build also issued MMAs from a lane that had not polled their barrier.
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, experts_gemm<MODE>);
    if (e != cudaSuccess) return e;
    if (a.localSizeBytes != 0) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(ExpSmem<MODE>::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&most, experts_gemm<MODE>, &cfg);
    if (e != cudaSuccess) return e;
    if (most < 1) return cudaErrorInvalidConfiguration;
    resident[dev & 63].store(most);
  }
  const unsigned n = static_cast<unsigned>(units < most ? units : most);
  return mns::launch_pdl_cluster(experts_gemm<MODE>, dim3(2 * n), dim3(ExpSmem<MODE>::kThreads), kSmem, stream, 2, P);
}

constexpr long long kMostUnits = 1LL << 30;  // 32-bit unit numbers in the kernel

long long tiles_of(long long n) { return (n + kExpTile - 1) / kExpTile; }

// Row tiles of all experts, at most.
template <int MODE>
long long row_tiles(long long rows, int experts) {
  return (rows + ExpSmem<MODE>::kRows - 1) / ExpSmem<MODE>::kRows + (experts < rows ? experts : rows);
}

int check(long long rows, int experts, int out_dim, int dim, int step) {
  if (rows < 0 || rows > kMaxRows || experts < 0 || experts > kExpMax || out_dim < 1 || out_dim > kMaxDim || dim < 1 ||
      dim > kMaxDim)
    return MUON_NS_ERR_INVALID_ARG;
  if (out_dim % 8 != 0 || dim % step != 0) return MUON_NS_ERR_ALIGNMENT;
  if (row_tiles<kExp8>(rows, experts) * tiles_of(out_dim) >= kMostUnits || row_tiles<kExp8>(rows, experts) * tiles_of(dim) >= kMostUnits ||
      experts * tiles_of(out_dim) * tiles_of(dim) >= kMostUnits)
    return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

Span offsets_of(const int* offsets, int experts) { return {offsets, 4 * (static_cast<size_t>(experts) + 1)}; }

template <typename Param = ExpertsGemm>
Param common(const int* offsets, long long rows, int experts, int* device_error) {
  Param P = {};
  P.offsets = offsets;
  P.experts = experts;
  P.rows = static_cast<int>(rows);
  P.err = device_error;
  P.budget = mns::wait_budget();
  return P;
}

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_experts(const muon_bf16* x, const muon_bf16* W, const int* offsets, long long rows, int experts, int out_dim,
                 int dim, muon_bf16* y, int* device_error, cudaStream_t stream) {
  int s = check(rows, experts, out_dim, dim, 8);
  if (s != MUON_NS_OK) return s;
  if (rows == 0 || experts == 0) return MUON_NS_OK;
  if (!x || !W || !offsets || !y) return MUON_NS_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(y, 16) || !aligned(offsets, 4) || !aligned(device_error, 4))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t xb = 2 * static_cast<size_t>(rows) * dim, yb = 2 * static_cast<size_t>(rows) * out_dim;
  const size_t wb = 2 * static_cast<size_t>(experts) * out_dim * dim;
  const Span rx = {x, xb}, ry = {y, yb}, w = {W, wb}, at = offsets_of(offsets, experts), word = {device_error, 4};
  if (overlaps(ry, {rx, w, at, word}) || overlaps(word, {rx, w, at})) return MUON_NS_ERR_INVALID_ARG;
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  ExpertsGemm P = common(offsets, rows, experts, device_error);
  P.m = out_dim;
  P.kdim = dim;
  P.out = y;
  if (!map_bf16(&P.tmA, W, dim, out_dim, experts, 128) || !map_rows(P.tmB, x, false, dim, rows)) return MUON_NS_ERR_CUDA;
  return status_of(launch_experts<kExpFwd>(P, row_tiles<kExpFwd>(rows, experts) * tiles_of(out_dim), stream));
}

int muon_experts_grad(const muon_bf16* dy, const muon_bf16* x, const muon_bf16* W, const int* offsets, long long rows,
                      int experts, int out_dim, int dim, muon_bf16* dx, void* dW, int dW_type, int accumulate,
                      int* device_error, cudaStream_t stream) {
  int s = check(rows, experts, out_dim, dim, 8);
  if (s != MUON_NS_OK) return s;
  if (!type_ok(dW_type) || (accumulate && dW_type != MUON_LM_F32)) return MUON_NS_ERR_INVALID_ARG;
  if (experts == 0 || (!dx && !dW)) return MUON_NS_OK;
  if (rows > 0 && (!offsets || !dy || (dx && !W) || (dW && !x))) return MUON_NS_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(W, 16) || !aligned(dx, 16) || !aligned(dW, 16) ||
      !aligned(offsets, 4) || !aligned(device_error, 4))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t gb = 2 * static_cast<size_t>(rows) * out_dim, xb = 2 * static_cast<size_t>(rows) * dim;
  const size_t n = static_cast<size_t>(experts) * out_dim * dim, db = n * type_size(dW_type);
  const Span rg = {dy, gb}, rx = {x, xb}, w = {W, 2 * n}, rdx = {dx, xb}, rdw = {dW, db}, at = offsets_of(offsets, experts),
             word = {device_error, 4};
  if (overlaps(rdx, {rg, rx, w, rdw, at, word}) || overlaps(rdw, {rg, rx, w, at, word}) || overlaps(word, {rg, rx, w, at}))
    return MUON_NS_ERR_INVALID_ARG;
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  if (rows == 0)
    return dW && !accumulate ? status_of(cudaMemsetAsync(dW, 0, db, stream)) : MUON_NS_OK;
  if (dx) {
    ExpertsGemm P = common(offsets, rows, experts, device_error);
    P.m = dim;
    P.kdim = out_dim;
    P.out = dx;
    if (!map_bf16(&P.tmA, W, dim, out_dim, experts, mns::kBlockK) || !map_rows(P.tmB, dy, false, out_dim, rows))
      return MUON_NS_ERR_CUDA;
    const cudaError_t e = launch_experts<kExpDx>(P, row_tiles<kExpDx>(rows, experts) * tiles_of(dim), stream);
    if (e != cudaSuccess) return status_of(e);
  }
  if (!dW) return MUON_NS_OK;
  ExpertsGemmDw P = common<ExpertsGemmDw>(offsets, rows, experts, device_error);
  P.m = out_dim;
  P.n = dim;
  P.out = dW;
  P.add = accumulate ? 1 : 0;
  P.sectors = dim % 16 == 0 && aligned(dW, 32) ? 1 : 0;
  if (!map_bf16(&P.tmA, dy, out_dim, rows, 1, mns::kBlockK) || !map_bf16(&P.tmB[0], x, dim, rows, 1, mns::kBlockK))
    return MUON_NS_ERR_CUDA;
  static constexpr int kTailRows[kExpTails] = {1, 2, 3, 4, 8, 12, 16, 32, 48};
  for (int i = 0; i < kExpTails; ++i)
    if (!map_bf16(&P.tail[0][i], dy, out_dim, rows, 1, kTailRows[i]) || !map_bf16(&P.tail[1][i], x, dim, rows, 1, kTailRows[i]))
      return MUON_NS_ERR_CUDA;
  const long long units = experts * tiles_of(out_dim) * tiles_of(dim);
  if (dW_type == MUON_LM_BF16) return status_of(launch_experts<kExpDwBf16>(P, units, stream));
  if (!map3d(&P.tmOut, dW, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, dim, out_dim, experts, 32, 32)) return MUON_NS_ERR_CUDA;
  return status_of(launch_experts<kExpDwF32>(P, units, stream));
}

int muon_experts8(const void* x, const float* x_scales, const void* W, const float* W_scales, const int* offsets,
                  long long rows, int experts, int out_dim, int dim, muon_bf16* y, int* device_error,
                  cudaStream_t stream) {
  int s = check(rows, experts, out_dim, dim, 16);
  if (s != MUON_NS_OK) return s;
  if (rows == 0 || experts == 0) return MUON_NS_OK;
  if (!x || !x_scales || !W || !W_scales || !offsets || !y) return MUON_NS_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(y, 16) || !aligned(x_scales, 4) || !aligned(W_scales, 4) ||
      !aligned(offsets, 4) || !aligned(device_error, 4))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t xb = static_cast<size_t>(rows) * dim, yb = 2 * static_cast<size_t>(rows) * out_dim;
  const size_t kb = (static_cast<size_t>(dim) + 127) / 128, mb = (static_cast<size_t>(out_dim) + 127) / 128;
  const Span rx = {x, xb}, ry = {y, yb}, w = {W, static_cast<size_t>(experts) * out_dim * dim}, xs = {x_scales, 4 * kb * rows},
             ws = {W_scales, 4 * kb * mb * experts}, at = offsets_of(offsets, experts), word = {device_error, 4};
  if (overlaps(ry, {rx, w, xs, ws, at, word}) || overlaps(word, {rx, w, xs, ws, at})) return MUON_NS_ERR_INVALID_ARG;
  if ((s = muon_ns_device_supported(-1)) != MUON_NS_OK) return s;
  ExpertsGemm P = common(offsets, rows, experts, device_error);
  P.m = out_dim;
  P.kdim = dim;
  P.out = y;
  P.xs = x_scales;
  P.ws = W_scales;
  if (!map3d(&P.tmA, W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, dim, out_dim, experts, 128, 128) ||
      !map_rows(P.tmB, x, true, dim, rows))
    return MUON_NS_ERR_CUDA;
  return status_of(launch_experts<kExp8>(P, row_tiles<kExp8>(rows, experts) * tiles_of(out_dim), stream));
}

}  // extern "C"
