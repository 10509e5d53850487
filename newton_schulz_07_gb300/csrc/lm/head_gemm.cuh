// The output head's three products on 2-SM tensor-core MMAs.
//
// With e = exp(h W^T - ref) of the live tokens (compact rows, `count` of them)
// and one piece of the vocabulary,
//   kLogits  z = h W^T (both operands K-major); the epilogue takes e, its row
//            sums and the rows' largest z, and stores e in bf16, all without
//            the rows' targets;
//   kDh      e W (e K-major, W MN-major) in fp32, split over the vocabulary
//            where there are few output tiles; splits go to rows of their own,
//            later pieces are added by bulk reductions;
//   kDw*     e^T hs (both MN-major), plus the targets' rows, in bf16 or fp32.
//
// A pair of CTAs computes a 256 x 256 tile: tcgen05.mma.cta_group::2 over
// 128-byte-swizzled operand tiles that TMA loads into a ring of 6 stages of 64
// K (each CTA its 128 rows of A and half of B), into one of two TMEM
// accumulators, while the epilogue warps drain the other.  Roles, barriers and
// their bounded waits are those of the Newton-Schulz products: warp 0 loads,
// warp 1 of the pair's first CTA issues the MMAs, warps 2 to 9 are the
// epilogue, two to a TMEM lane quarter.  A wait that runs out sets the error
// word; the roles leave, copies and MMAs in flight are waited for and TMEM is
// freed.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "gemm_tc.cuh"
#include "lm/common.cuh"

namespace mns {
namespace lm {

enum HeadMode : int { kLogits = 0, kDh = 1, kDwBf16 = 2, kDwF32 = 3 };

constexpr int kHeadStages = 6;
constexpr int kHeadStageBytes = kABytes + kBBytes / 2;  // A tile and half a B panel: 32 KB
constexpr int kHeadEpiWarps = 8;
constexpr int kHeadThreads = 64 + 32 * kHeadEpiWarps;
constexpr int kHeadStaging = 4096;  // an epilogue warp's box: 32 rows of 128 bytes
constexpr int kHeadSmem = kHeadStages * kHeadStageBytes + kHeadEpiWarps * kHeadStaging + 1024;
static_assert(kHeadSmem + 1024 <= 232448, "shared memory");
constexpr int kHeadRows = 256;      // rows and columns of a pair's tile
constexpr int kHeadHalf = 128;      // columns an epilogue warp takes: one statistic a row
// Waits on the way out, at least: what is in flight must land before the CTA
// may leave, however short the budget of the waits that gave up.
constexpr long long kHeadDrain = 4000000000LL;

// Control words at the start of the workspace.
enum HeadCtl : int { kCtlErr = 0, kCtlCount = 1, kCtlSplits = 2, kCtlRedo = 3, kCtlWords = 64 };

struct HeadGemm {
  CUtensorMap tmA, tmB, tmOut;
  int* ctl;
  int vp;   // vocabulary columns of the piece
  int dim;
  int group;  // pair rows walked together, column by column
  // kLogits (e) and kDwBf16 (dW): bf16 output, written from registers.
  void* out;
  long long ld;
  int rows;     // rows of the output
  int sectors;  // its rows start on 32 bytes
  // kLogits
  const float* ref;   // per row
  const int* target;  // per row: its column of the whole vocabulary
  float2* stat;       // [rows][stat_ld]: (largest z, sum of e) of 128 columns; may be null
  int stat_ld, stat0; // stat0: the piece's first
  int store;          // write e
  const int* redo;    // rows of tiles to compute again (per pair row); null: all of them
  // kDh, kDwF32: add to what is there
  int add;
  // kDw*
  const float* addend;         // fp32 [rows][dim], compact
  const int* slot;             // row of a vocabulary row's addend: one if sorted[slot] has its key
  const unsigned long long* sorted;
  // kLogits, kDw*
  long long v0;                // first vocabulary row of the piece
  long long budget;
};

// Pair rows of the live tokens.  With none, one tile of masked rows is
// computed all the same: it is what makes e and dW zero.
__device__ __forceinline__ int token_pairs(int count) {
  return count > kHeadRows ? (count + kHeadRows - 1) / kHeadRows : 1;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// As tma_store_3d, but fp32 values are added to global memory.
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// Arrival on a barrier of the pair's other CTA that orders no memory: it tells
// the MMA thread that an accumulator has been read, which tcgen05.wait::ld and
// the fence before it have made sure of.  (A release at cluster scope waits for
// every earlier write of the thread, about 2000 cycles a tile here.)
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 16 bf16 to a 32-byte aligned address: one whole sector a lane.
__device__ __forceinline__ void store_sector(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Division by a number known once per launch: a multiplication and at most two
// corrections in place of the hundreds of cycles of a 64-bit division, which
// each role would take between two tiles.
struct FastDiv {
  uint32_t d, m;
  __device__ __forceinline__ explicit FastDiv(uint32_t divisor) : d(divisor), m(0xFFFFFFFFu / divisor) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t n, uint32_t* rest) const {
    uint32_t q = __umulhi(n, m), r = n - q * d;
    if (r >= d) {
      ++q;
      r -= d;
    }
    if (r >= d) {
      ++q;
      r -= d;
    }
    *rest = r;
    return q;
  }
};

constexpr float kLog2e = 1.4426950408889634f;

template <int MODE>
__global__ void __launch_bounds__(kHeadThreads, 1) head_gemm(const __grid_constant__ HeadGemm P) {
  constexpr bool kAMn = MODE >= kDwBf16;
  constexpr bool kBMn = MODE != kLogits;
  using EC = ElemCfg<false>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kHeadStages + 5];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  // Stages this CTA has asked to be filled, and (in the pair's first CTA) the
  // stages and accumulators its MMAs have committed.
  __shared__ int fills_sh, stages_sh, units_sh;
  __shared__ int peer_abort_sh;  // the other CTA of the pair gave up

  ptx::griddep_launch_dependents();
  // Nothing to do again: the whole grid leaves before it sets anything up.
  if (MODE == kLogits && P.redo != nullptr) {
    ptx::griddep_wait();
    if (P.ctl[kCtlRedo] == 0) return;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = static_cast<int>(ptx::cluster_ctarank());
  const bool leader = crank == 0;
  volatile int* abort_flag = &abort_sh;
  int* err = P.ctl + kCtlErr;

  // Barriers: full[s], empty[s], tfull[2], tempty[2], mma_done.
  const uint32_t bar0 = ptx::smem_u32(&bars[0]);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kHeadStages + s); };
  auto tfull = [&](int i) { return bar0 + 8u * (2 * kHeadStages + i); };
  auto tempty = [&](int i) { return bar0 + 8u * (2 * kHeadStages + 2 + i); };
  const uint32_t mma_done = bar0 + 8u * (2 * kHeadStages + 4);
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kHeadStages; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(tfull(i), 1);
      ptx::mbar_init(tempty(i), 2 * kHeadEpiWarps);
    }
    ptx::mbar_init(mma_done, 1);
    *abort_flag = 0;
    fills_sh = stages_sh = units_sh = peer_abort_sh = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&P.tmA);
    ptx::prefetch_tensormap(&P.tmB);
    if (MODE == kDh || MODE == kDwF32) ptx::prefetch_tensormap(&P.tmOut);
  }
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 0) {
    ptx::tmem_alloc_pair(ptx::smem_u32(&tmem_base_sh), kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  // The set-up above touches this CTA's own memory alone and runs beside the
  // end of the kernel before.
  ptx::griddep_wait();
  const int4 ctl = *reinterpret_cast<const int4*>(P.ctl);
  static_assert(kCtlCount == 1 && kCtlSplits == 2, "control words");

  // The tile space: `splits` times pair rows x column tiles, split-major, so
  // that tiles running together read the same part of a split contraction.
  const int count = ctl.y;
  const int pr = MODE >= kDwBf16 ? (P.vp + kHeadRows - 1) / kHeadRows : token_pairs(count);
  const int tn = ((MODE == kLogits ? P.vp : P.dim) + kHeadRows - 1) / kHeadRows;
  const int kb_all = MODE == kLogits ? (P.dim + kBlockK - 1) / kBlockK
                     : MODE == kDh   ? (P.vp + kBlockK - 1) / kBlockK
                                     : (count > 0 ? (count + kBlockK - 1) / kBlockK : 1);
  const int splits = MODE == kDh ? ctl.z : 1;
  // (Fewer than 2^31 tiles: the host sees to it.)
  const uint32_t tiles = static_cast<uint32_t>(pr) * static_cast<uint32_t>(tn);
  const uint32_t total = tiles * static_cast<uint32_t>(splits);
  const uint32_t unit0 = ptx::cluster_id_x(), ustride = ptx::cluster_count_x();
  const FastDiv by_tiles(tiles), by_group(static_cast<uint32_t>(P.group) * static_cast<uint32_t>(tn));
  // A band of `group` pair rows is walked column by column; the last may hold
  // fewer.
  const FastDiv by_rows(P.group), by_last(pr % P.group ? pr % P.group : P.group);
  const uint32_t last_band = static_cast<uint32_t>((pr - 1) / P.group);
  struct Unit {
    int I, J, s, kb0, kb1;  // row tile of this CTA, column tile, split, its k-blocks
  };
  auto unit = [&](uint32_t u) {
    Unit t;
    uint32_t in_split = u, in_band, row;
    t.s = 0;
    t.kb0 = 0;
    t.kb1 = kb_all;
    if (MODE == kDh) {
      t.s = static_cast<int>(by_tiles(u, &in_split));
      t.kb0 = static_cast<int>(static_cast<long long>(kb_all) * t.s / splits);
      t.kb1 = static_cast<int>(static_cast<long long>(kb_all) * (t.s + 1) / splits);
    }
    const uint32_t band = by_group(in_split, &in_band);
    t.J = static_cast<int>(band == last_band ? by_last(in_band, &row) : by_rows(in_band, &row));
    t.I = 2 * static_cast<int>(band * P.group + row) + crank;
    return t;
  };
  auto skip = [&](const Unit& t) { return MODE == kLogits && P.redo != nullptr && P.redo[t.I >> 1] == 0; };

  const long long drain = P.budget > kHeadDrain ? P.budget : kHeadDrain;
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      // The operands were written by other kernels' ordinary stores.
      ptx::fence_proxy_async_global();
      int stage = 0, fills = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (uint32_t u = unit0; ok && u < total; u += ustride) {
        const Unit t = unit(u);
        if (skip(t)) continue;
        const int row0 = t.I * kTileM, col0 = t.J * kTileN + crank * (kTileN / 2);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!detail::wait_bounded<true>(empty(stage), phase ^ 1u, abort_flag, err, P.budget)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_base + stage * kHeadStageBytes, sb = sa + kABytes;
          const int k0 = kb * kBlockK;
          // All bytes of the pair are counted on CTA 0's barrier.
          const uint32_t fb = ptx::mapa(full(stage), 0);
          if (leader) ptx::mbar_arrive_expect_tx(full(stage), 2 * kHeadStageBytes);
          if (kAMn) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              ptx::tma_load_3d_pair(sa + c * EC::kMnChunkBytes, &P.tmA, fb, row0 + c * EC::kMnChunk, k0, 0);
          } else {
            ptx::tma_load_3d_pair(sa, &P.tmA, fb, k0, row0, 0);
          }
          if (kBMn) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              ptx::tma_load_3d_pair(sb + c * EC::kMnChunkBytes, &P.tmB, fb, col0 + c * EC::kMnChunk, k0, 0);
          } else {
            ptx::tma_load_3d_pair(sb, &P.tmB, fb, k0, col0, 0);
          }
          ++fills;
          if (++stage == kHeadStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      fills_sh = fills;
      // The last release of each stage is awaited here, so that after a full
      // run no commit is on its way to this CTA's barriers when it leaves.
      for (int i = fills > kHeadStages ? fills - kHeadStages : 0; ok && i < fills; ++i)
        ok = detail::wait_bounded<true>(empty(i % kHeadStages), (i / kHeadStages) & 1, abort_flag, err, P.budget);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc = ptx::idesc_bf16_f32(2 * kTileM, kTileN, kAMn, kBMn);
      int stage = 0, buf = 0, stages = 0, units = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (uint32_t u = unit0; ok && u < total; u += ustride) {
        const Unit t = unit(u);
        if (skip(t)) continue;
        if (!detail::wait_bounded<true>(tempty(buf), tphase ^ 1u, abort_flag, err, P.budget)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kTileN);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!detail::wait_bounded<true>(full(stage), phase, abort_flag, err, P.budget)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sa = smem_base + stage * kHeadStageBytes, sb = sa + kABytes;
#pragma unroll
          for (int kk = 0; kk < kBlockK / EC::kMmaK; ++kk) {
            const uint64_t ad = kAMn ? ptx::sw128_desc(sa + kk * EC::kMnStep, EC::kMnChunkBytes, 1024)
                                     : ptx::sw128_desc(sa + kk * 32, 16, 1024);
            const uint64_t bd = kBMn ? ptx::sw128_desc(sb + kk * EC::kMnStep, EC::kMnChunkBytes, 1024)
                                     : ptx::sw128_desc(sb + kk * 32, 16, 1024);
            ptx::mma_bf16_pair(d_tmem, ad, bd, idesc, (kb != t.kb0 || kk != 0) ? 1u : 0u);
          }
          ptx::mma_commit_pair(empty(stage), 0x3);
          ++stages;
          if (++stage == kHeadStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_pair(tfull(buf), 0x3);
        ++units;
        buf ^= 1;
        if (buf == 0) tphase ^= 1u;
      }
      ptx::mma_commit_pair(mma_done, 0x1);
      detail::drain_wait<true>(mma_done, 0, drain);
      stages_sh = stages;
      units_sh = units;
    }
  } else {
    // ------------------------------------------------------------- epilogue
    // Warp e reads TMEM lane quarter warp % 4 (32 rows, a row a lane) and 128
    // of the tile's 256 columns, in chunks of 32.
    const int e = warp - 2, q = warp & 3;
    const int c_begin = (e >> 2) * kHeadHalf;
    const uint32_t stg = smem_base + kHeadStages * kHeadStageBytes + static_cast<uint32_t>(e * kHeadStaging);
    int buf = 0;
    uint32_t tphase = 0;
    // kDw*: where the addend of this lane's row is, resolved a tile ahead: the
    // slot's load is issued two tiles ahead, that of the key it must have one.
    auto row_of = [&](uint32_t u) {
      const int row = u < total ? unit(u).I * kTileM + q * 32 + lane : P.vp;
      return row < P.vp ? row : -1;
    };
    auto slot_at = [&](int row) { return row >= 0 ? P.slot[P.v0 + row] : -1; };
    auto key_at = [&](int slot) {
      return static_cast<unsigned>(slot) < static_cast<unsigned>(count) ? P.sorted[slot] >> 32 : ~0ull;
    };
    int row1 = -1, slot1 = -1;          // next tile
    int slot0 = -1;                     // this tile
    unsigned long long key0 = ~0ull;
    if (MODE >= kDwBf16) {
      slot0 = slot_at(row_of(unit0));
      key0 = key_at(slot0);
      row1 = row_of(unit0 + ustride);
      slot1 = slot_at(row1);
    }
    for (uint32_t u = unit0; u < total; u += ustride) {
      const Unit t = unit(u);
      if (skip(t)) continue;
      const int row_w = t.I * kTileM + q * 32;  // first row of the warp
      const int row = row_w + lane;
      const int col0 = t.J * kTileN + c_begin;
      const int cols = MODE == kLogits ? P.vp : P.dim;
      // What the rows need besides the product, fetched before the wait.
      float cl = 0.0f;
      bool live = false;
      int target = -1;  // among the warp's columns, if it is there
      if (MODE == kLogits) {
        live = row < count;
        if (live) {
          cl = P.ref[row] * kLog2e;
          target = P.target[row] - static_cast<int>(P.v0) - col0;
        }
      }
      const float* addend = nullptr;
      if (MODE >= kDwBf16) {
        if (key0 == static_cast<unsigned long long>(P.v0 + row)) addend = P.addend + static_cast<long long>(slot0) * P.dim;
        slot0 = slot1;
        key0 = key_at(slot1);
        row1 = row_of(u + 2 * ustride);
        slot1 = slot_at(row1);
      }
      int ready = 0;
      if (lane == 0) ready = detail::wait_bounded<true>(tfull(buf), tphase, abort_flag, err, P.budget) ? 1 : 0;
      ready = __shfl_sync(0xFFFFFFFFu, ready, 0);
      if (!ready) break;
      __syncwarp();
      ptx::tc_fence_after();
      const uint32_t t_lane =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * kTileN + c_begin);
      // The pair's next MMAs write both CTAs' accumulators: one arrival a warp,
      // on CTA 0's barrier.
      auto release = [&] {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            ptx::mbar_arrive(tempty(buf));
          else
            arrive_remote_relaxed(ptx::mapa(tempty(buf), 0));
        }
      };
      float mx = -INFINITY, s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int cc = 0; cc < kHeadHalf / 32; ++cc) {
        const int gj = col0 + cc * 32;
        if (gj >= cols) break;  // warp-uniform
        uint32_t v[32];
        ptx::tmem_ld_32cols(t_lane + static_cast<uint32_t>(cc * 32), v);
        ptx::tmem_wait_ld();
        if (cc + 1 == kHeadHalf / 32 || gj + 32 >= cols) {
          // The warp's last read: its part of the accumulator may be written.
          release();
        }
        if (MODE == kLogits) {
          // Columns past the piece hold zero, not a logit: no part of the sums.
          const int n = cols - gj;
          // Nor is the target's: 1 - p is the sum of the others, and would be
          // lost in rounding beside it.  (Rows are sorted by target where there
          // is a gradient; few chunks hold any.)
          const int hit = target - cc * 32;
          if (__any_sync(0xFFFFFFFFu, static_cast<unsigned>(hit) < 32u)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (hit == j) v[j] = 0xFF800000u;  // -infinity
          }
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float z = j < n ? __uint_as_float(v[j]) : -INFINITY;
            mx = fmaxf(mx, z);
            // One fused multiply-add in the exponent: the rounding of cl moves
            // the whole row's reference by 2^-24 of itself, the target's
            // exponential (head_finish) with it, and cancels in their ratios.
            f[j] = exp2_approx(fmaf(z, kLog2e, -cl));
            s4[j & 3] += f[j];
          }
          if (P.store) {
            // e is rounded to bf16 here, the MMAs' operand type: a relative
            // error of up to 2^-8 in each term of sums over many; the target's
            // term, the sum of all others, is added in fp32.  Rows past the
            // live tokens are zero.
            if (row < P.rows) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = live ? detail::pack_bf16x2(f[2 * k], f[2 * k + 1]) : 0u;
              bf16* to = static_cast<bf16*>(P.out) + static_cast<long long>(row) * P.ld + gj;
              store_sector(to, w);
              store_sector(to + 16, w + 8);
            }
          }
        } else {
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
          if (MODE >= kDwBf16 && addend != nullptr) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              if (gj + 4 * g < cols) {
                const float4 a = *reinterpret_cast<const float4*>(addend + gj + 4 * g);
                f[4 * g] += a.x;
                f[4 * g + 1] += a.y;
                f[4 * g + 2] += a.z;
                f[4 * g + 3] += a.w;
              }
            }
          }
          if (MODE == kDwBf16) {
            if (row < P.rows) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = detail::pack_bf16x2(f[2 * k], f[2 * k + 1]);
              bf16* to = static_cast<bf16*>(P.out) + static_cast<long long>(row) * P.ld + gj;
              if (P.sectors && gj + 32 <= cols) {
                store_sector(to, w);
                store_sector(to + 16, w + 8);
              } else {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                  if (gj + 8 * g < cols) ptx::st_global_v4(to + 8 * g, w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
              }
            }
          } else {
            if (lane == 0) ptx::bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 8; ++g)
              ptx::st_shared_v4(stg + stage_off32(lane, 4 * g), __float_as_uint(f[4 * g]), __float_as_uint(f[4 * g + 1]),
                                __float_as_uint(f[4 * g + 2]), __float_as_uint(f[4 * g + 3]));
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int y = MODE == kDh ? t.s * pr * kHeadRows + row_w : row_w;
              if (P.add)
                tma_add_3d(&P.tmOut, stg, gj, y, 0);
              else
                ptx::tma_store_3d(&P.tmOut, stg, gj, y, 0);
              ptx::bulk_commit();
            }
          }
        }
      }
      if (col0 >= cols) release();  // nothing to read
      if (MODE == kLogits && P.stat != nullptr && live && col0 < cols)
        P.stat[static_cast<long long>(row) * P.stat_ld + P.stat0 + col0 / kHeadHalf] =
            make_float2(mx, (s4[0] + s4[1]) + (s4[2] + s4[3]));
      buf ^= 1;
      if (buf == 0) tphase ^= 1u;
    }
    // The staging boxes stay until the bulk stores are done.
    if (lane == 0) ptx::bulk_wait_all();
    __syncwarp();
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag)
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(
                     ptx::mapa(ptx::smem_u32(&peer_abort_sh), static_cast<uint32_t>(crank ^ 1))),
                 "r"(1)
                 : "memory");
  // Neither CTA leaves while the other may still address it.
  ptx::cluster_sync();
  // (The same in both CTAs: neither flag changes any more.)
  const bool gave_up = *abort_flag || *static_cast<volatile int*>(&peer_abort_sh);
  if (gave_up && warp == 0 && lane == 0) {
    // Nothing may be on its way to a CTA that leaves.  After a full run every
    // arrival has been awaited by the role that it was for; after a wait that
    // ran out the two CTAs may have asked for different numbers of fills.
    // Copies are counted on the first CTA's barriers: it expects the other's
    // bytes alone for fills of its own that are missing, and the other stands
    // in for its missing ones.
    auto remote = [](const int* p, int rank) {
      int v;
      asm volatile("ld.shared::cluster.s32 %0, [%1];"
                   : "=r"(v)
                   : "r"(ptx::mapa(ptx::smem_u32(p), static_cast<uint32_t>(rank)))
                   : "memory");
      return v;
    };
    const int mine = fills_sh, other = remote(&fills_sh, crank ^ 1);
    const int top = mine > other ? mine : other;
    if (leader) {
      for (int i = top > kHeadStages ? top - kHeadStages : 0; i < top; ++i) {
        const int s = i % kHeadStages;
        if (i >= mine) ptx::mbar_arrive_expect_tx(full(s), kHeadStageBytes);
        detail::drain_wait<true>(full(s), (i / kHeadStages) & 1, drain);
      }
    } else {
      for (int i = mine; i < top; ++i)
        asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(
                         ptx::mapa(full(i % kHeadStages), 0)),
                     "r"(kHeadStageBytes)
                     : "memory");
    }
    const int stages = remote(&stages_sh, 0), units = remote(&units_sh, 0);
    for (int i = stages > kHeadStages ? stages - kHeadStages : 0; i < stages; ++i)
      detail::drain_wait<true>(empty(i % kHeadStages), (i / kHeadStages) & 1, drain);
    for (int i = units > 2 ? units - 2 : 0; i < units; ++i) detail::drain_wait<true>(tfull(i & 1), (i >> 1) & 1, drain);
  }
  if (gave_up) {
    __syncthreads();
    ptx::cluster_sync();
  }
  if (warp == 0) {
    __syncwarp();
    ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

}  // namespace lm
}  // namespace mns
