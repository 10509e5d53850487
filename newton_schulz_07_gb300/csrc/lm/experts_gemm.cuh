// Products grouped by expert on 2-SM tensor-core MMAs.  Rows lo_e .. lo_e + len_e
// of x (and of y, dy, dx) are those of expert e, of any number:
//   kExpFwd   y  = x W_e^T
//   kExpDx    dx = dy W_e
//   kExpDw*   dW_e = dy_e^T x_e, in bf16 or fp32
//   kExp8     y  = x W_e^T on e4m3 operands with a scale for each 128 of the
//             contraction (and each 128 rows of W)
//
// In the first two and the last the features of W are the MMA's M (256 a CTA
// pair) and the expert's rows its N, any multiple of 32 up to 256: an expert with
// few rows, or a last tile, costs what it holds, and rows of the next expert that
// a tile's last box reads are columns of the accumulator that nobody stores (no
// masking, and nothing they hold can spread).  With rows as M a tile is 256 rows
// whatever it holds: a quarter more work at 512 rows an expert on average.  The
// accumulator is y^T, so the epilogue transposes 32 x 32 pieces on their way
// through shared memory (matrix-fragment TMEM loads, transposing matrix stores).
//
// dW's contraction runs over the expert's rows, and its last 16 may hold rows of
// others, which have to be zero in both operands.  The copies see to it: a stage that
// ends so is brought in up to three boxes that hold the expert's rows alone, and the
// rest of the 16 in a box that starts behind the last row of x, where a copy reads
// zeros.  Nothing but copies writes the stages, so the copies' own barrier orders all
// of it for the MMA, in both CTAs.  (Rows zeroed by a warp would have to be handed
// from one CTA to the other with a release at cluster scope, about 2000 cycles.  Boxes
// of the rows' binary digits took 379 us for 369 at 65536 rows of 128 experts, 1536 x
// 2048; without any ragged expert 344.)
//
// Roles: warp 0 loads A by TMA (each CTA its 128 rows) into a ring of 6 stages
// (kExp8: 3 of two k-blocks) and warp 3 its half of B (one thread that loaded both
// took longer over a stage than its MMAs), warp 1 of the pair's first CTA issues MMAs into one of two TMEM
// accumulators, 8 more are the epilogue, two to a TMEM lane quarter.  kExp8: warp 2
// loads scales, and 16 are the epilogue.
// The bytes of both CTAs are counted on the first one's barrier.  Waits are bounded;
// where one runs out the error word is set, the epilogue writes NaN in place of what
// it has not got, copies and MMAs in flight are waited for and TMEM is freed.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "gemm_tc.cuh"
#include "lm/common.cuh"

namespace mns {
namespace lm {

enum ExpMode : int { kExpFwd = 0, kExpDx = 1, kExpDwBf16 = 2, kExpDwF32 = 3, kExp8 = 4 };

constexpr int kExpTile = 256;      // features (rows and columns of dW) of a pair's tile
constexpr int kExpMax = 1024;      // experts
constexpr int kExpBand = 16;       // row tiles of an expert that are walked together
constexpr int kExpAhead = 16;      // units that a producer finds at once
constexpr int kExpBoxes = 4;       // B boxes: of 128, 64, 32 or 16 rows
constexpr int kExpTails = 9;       // dW's last rows: boxes of 1, 2, 3, 4, 8, 12, 16, 32 or 48 of them
constexpr long long kExpDrain = 4000000000LL;
constexpr uint32_t kExpNan = 0x7FFF7FFFu;  // NaN of fp32 and of bf16 alike

constexpr int kExpScales = 8;      // k-blocks whose scales are brought together (kExp8)

template <int MODE>
struct ExpSmem {
  static constexpr bool kDw = MODE == kExpDwBf16 || MODE == kExpDwF32;
  static constexpr int kRoles = 4;  // warps before the epilogue's
  // Of the epilogue: two to a TMEM lane quarter, or four (kExp8, which scales every
  // k-block: 353 us became 342, and 291 with two k-blocks to a wait; at 16384 rows of
  // 32 experts, 7168 x 2048).
  static constexpr int kEpi = MODE == kExp8 ? 16 : 8;
  static constexpr int kThreads = 32 * (kRoles + kEpi);
  // Rows of a tile, at most.  kExp8 takes 128: its epilogue holds their sums in
  // registers, and an accumulator holds two k-blocks.
  static constexpr int kRows = MODE == kExp8 ? 128 : 256;
  // k-blocks of a stage: kExp8 takes two, as many as an accumulator (8192^3: 580 us
  // became 561).
  static constexpr int kPer = MODE == kExp8 ? 2 : 1;
  static constexpr int kBBytes = kRows * 64;  // half a B panel
  static constexpr int kStageBytes = kPer * (kABytes + kBBytes);
  static constexpr int kStages = 6 / kPer;
  static constexpr int kStaging = kDw ? 4096 : 2048;  // an epilogue warp's
  static constexpr int kStagingAt = kStages * kStageBytes;
  static constexpr int kSpanAt = kStagingAt + kEpi * kStaging;      // int2 [experts]: first row, rows
  static constexpr int kUnitsAt = kSpanAt + (kDw ? 0 : 8 * kExpMax);        // int [experts + 1]: units before
  static constexpr int kScalesAt = kUnitsAt + (kDw ? 0 : 4 * kExpMax + 16);  // kExp8: float [2][kExpScales][kRows]
  static constexpr int kBytes = kScalesAt + (MODE == kExp8 ? 2 * kExpScales * kRows * 4 : 0) + 1024;
  // The static part: units of the next turns (lists of kExpAhead), barriers, words.
  static constexpr int kTurnLists = MODE == kExp8 ? 2 + kEpi : 2;
  static constexpr int kBars = 2 * kStages + 2 * 2 + 5;
  static constexpr int kStatic = 16 * kTurnLists * kExpAhead + 8 * kBars + 64;
  static_assert(kBytes + kStatic <= 232448, "shared memory");
};

struct ExpertsGemm {
  CUtensorMap tmA, tmB[kExpBoxes], tmOut;
  const int* offsets;  // [experts + 1]
  int experts;
  int rows;   // of x
  int m;      // features that are the MMA's M: of y (kExpFwd, kExp8, kExpDw*) or of dx
  int n;      // kExpDw*: columns of dW
  int kdim;   // contraction, but for kExpDw*
  void* out;
  int sectors;  // kExpDwBf16: rows of dW start on 32 bytes
  int add;      // kExpDwF32: add to what is there
  int* err;
  long long budget;
  // kExp8
  const float* xs;  // [rows][kblocks]
  const float* ws;  // [experts][ceil(m / 128)][kblocks]
};
// kExpDw*: the maps of the last rows of dy and x.
struct ExpertsGemmDw : ExpertsGemm {
  CUtensorMap tail[2][kExpTails];
};
template <int MODE>
using ExpertsParam = std::conditional_t<ExpSmem<MODE>::kDw, ExpertsGemmDw, ExpertsGemm>;

// One lane of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// After the wait for TMEM loads, of the registers that they loaded: nothing that
// uses these is moved before it.
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Whether a stage of dW with `left` rows to go ends in an MMA's 16 that are not all
// the expert's.
__device__ __forceinline__ bool others_rows(int left) { return left < kBlockK && (left & 15) != 0; }

// First row and rows of expert e, whatever the offsets hold: inside the rows.
__device__ __forceinline__ int2 expert_span(const int* offsets, int e, int rows) {
  const int a = offsets[e], b = offsets[e + 1];
  const int lo = a < 0 ? 0 : a > rows ? rows : a;
  const int hi = b < lo ? lo : b > rows ? rows : b;
  return make_int2(lo, hi - lo);
}

// Arrival on the barrier of the pair's first CTA at this CTA's offset `bar` that
// orders no memory: what it tells of, reads of TMEM, has been ordered by
// tcgen05.wait::ld and tcgen05.fence.
__device__ __forceinline__ void arrive_pair_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(ptx::mapa(bar, 0)) : "memory");
}

template <int MODE>
__global__ void __launch_bounds__(ExpSmem<MODE>::kThreads, 1) experts_gemm(const __grid_constant__ ExpertsParam<MODE> P) {
  using S = ExpSmem<MODE>;
  using EC = ElemCfg<false>;
  constexpr bool kDw = S::kDw;
  constexpr bool kAMn = MODE == kExpDx || kDw;
  constexpr bool kBMn = kDw;
  constexpr int kK = MODE == kExp8 ? 128 : kBlockK;  // contraction of a k-block
  constexpr int kStages = S::kStages, kBufs = 2, kPer = S::kPer;
  extern __shared__ uint8_t smem_raw[];
  // Barriers: full[s], empty[s], tfull[b], tempty[b], mma_done, sfull[2], sempty[2].
  __shared__ __align__(8) uint64_t bars[S::kBars];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  // Stages this CTA has asked to be filled (with A, with B) and, in the pair's
  // first CTA, the stages and accumulators its MMAs have committed.
  __shared__ int fills_sh[2], stages_sh, units_sh;
  __shared__ int peer_abort_sh;  // the other CTA of the pair gave up
  // Units of the next turns of a producer and (kExp8, to spare registers) of the
  // epilogue's warps: expert, tiles, first row, rows.
  __shared__ int4 turns_sh[S::kTurnLists][kExpAhead];

  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = static_cast<int>(ptx::cluster_ctarank());
  const bool leader = crank == 0;
  volatile int* abort_flag = &abort_sh;
  int* err = P.err;

  const uint32_t bar0 = ptx::smem_u32(&bars[0]);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tfull = [&](int i) { return bar0 + 8u * (2 * kStages + i); };
  auto tempty = [&](int i) { return bar0 + 8u * (2 * kStages + kBufs + i); };
  const uint32_t mma_done = bar0 + 8u * (2 * kStages + 2 * kBufs);
  auto sfull = [&](int i) { return mma_done + 8u * (1 + i); };
  auto sempty = [&](int i) { return mma_done + 8u * (3 + i); };
  const uint32_t smem_base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem_base - ptx::smem_u32(smem_raw));
  int2* span = reinterpret_cast<int2*>(smem + S::kSpanAt);
  int* before = reinterpret_cast<int*>(smem + S::kUnitsAt);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      ptx::mbar_init(tfull(i), 1);
      ptx::mbar_init(tempty(i), 2 * S::kEpi);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(sfull(i), 1);
      ptx::mbar_init(sempty(i), S::kEpi);
    }
    ptx::mbar_init(mma_done, 1);
    *abort_flag = 0;
    fills_sh[0] = fills_sh[1] = stages_sh = units_sh = peer_abort_sh = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tensormap(&P.tmA);
    ptx::prefetch_tensormap(&P.tmB[0]);
    if (MODE == kExpDwF32) ptx::prefetch_tensormap(&P.tmOut);
  }
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 0) {
    ptx::tmem_alloc_pair(ptx::smem_u32(&tmem_base_sh), kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  // The set-up above touches this CTA's own memory alone and runs beside the
  // end of the kernel before.
  ptx::griddep_wait();

  // The tile space.  A unit is a tile: for kExpDw* every expert has the same; else
  // as many row tiles as its rows take, of equal size up to 32 rows.
  const int mtiles = (P.m + kExpTile - 1) / kExpTile;
  const int ntiles = kDw ? (P.n + kExpTile - 1) / kExpTile : 1;
  if (!kDw) {
    for (int e = threadIdx.x; e < P.experts; e += S::kThreads) span[e] = expert_span(P.offsets, e, P.rows);
    __syncthreads();
    if (warp == 1) {
      int sum = 0, most = 0;
      for (int e0 = 0; e0 < P.experts; e0 += 32) {
        const int e = e0 + lane;
        // An expert starts behind all before it, so that no row is two experts'
        // (and the tiles stay as few as the host has counted) even where offsets
        // decrease.
        int2 s = e < P.experts ? span[e] : make_int2(0, 0);
        const int end = s.x + s.y;
        int top = end;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, top, o);
          if (lane >= o && v > top) top = v;
        }
        int behind = __shfl_up_sync(0xFFFFFFFFu, top, 1);
        if (lane == 0 || behind < most) behind = most;
        if (s.x < behind) s.x = behind;
        s.y = end > s.x ? end - s.x : 0;
        if (e < P.experts) span[e] = s;
        top = __shfl_sync(0xFFFFFFFFu, top, 31);
        most = top > most ? top : most;
        const int mine = (s.y + S::kRows - 1) / S::kRows * mtiles;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
          if (lane >= o) upto += v;
        }
        if (e < P.experts) before[e] = sum + upto - mine;
        sum += __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
      if (lane == 0) before[P.experts] = sum;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;

  // (Fewer than 2^30 units: the host sees to it.)
  const int total = kDw ? P.experts * mtiles * ntiles : before[P.experts];
  const int unit0 = static_cast<int>(ptx::cluster_id_x()), ustride = static_cast<int>(ptx::cluster_count_x());
  struct Unit {
    int e, I, J;     // expert, M tile of this CTA, N tile (kExpDw*)
    int row0, rows;  // rows of the tile (kExpDw*: of the expert)
    int half;        // MMA columns of a CTA's half of B
    int kbs;         // k-blocks
  };
  // The place of unit u, packed: expert and N tile, M tile of the pair, first row,
  // rows.  It takes several divisions, so each warp finds 32 of its units at once, a
  // lane one.
  auto place = [&](int u) {
    if (u >= total) return make_int4(0, 0, 0, 0);
    if (kDw) {
      const int each = mtiles * ntiles, e = u / each, in = u - e * each, n = in / mtiles;
      const int2 s = expert_span(P.offsets, e, P.rows);
      return make_int4(e | n << 12, in - n * mtiles, s.x, s.y);
    }
    int a = 0, b = P.experts;  // before[a] <= u < before[b]
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (before[mid] <= u)
        a = mid;
      else
        b = mid;
    }
    const int2 s = span[a];
    const int in = u - before[a], nt = (s.y + S::kRows - 1) / S::kRows;
    const int size = ((s.y + nt - 1) / nt + 31) & ~31;
    // A band of row tiles is walked feature tile by feature tile.
    const int band = in / (kExpBand * mtiles), rest = in - band * kExpBand * mtiles;
    const int wide = nt - band * kExpBand < kExpBand ? nt - band * kExpBand : kExpBand;
    const int m = rest / wide, at = (band * kExpBand + rest - m * wide) * size;
    return make_int4(a, m, s.x + at, s.y - at < size ? s.y - at : size);
  };
  const int kbs_all = kDw ? 0 : (P.kdim + kK - 1) / kK;
  auto unit_of = [&](int4 v) {
    Unit t;
    t.e = v.x & 4095;
    t.J = v.x >> 12;
    t.I = 2 * v.y + crank;
    t.row0 = v.z;
    t.rows = v.w;
    t.half = kDw ? kExpTile / 2 : ((v.w + 31) & ~31) / 2;
    t.kbs = kDw ? (v.w + kK - 1) / kK : kbs_all;
    return t;
  };
  const int turns = unit0 < total ? (total - unit0 + ustride - 1) / ustride : 0;
  struct Ahead {
    int4 v;
  };
  auto unit_at = [&](int turn, Ahead& a) {
    if ((turn & 31) == 0) a.v = place(turn + lane < turns ? unit0 + (turn + lane) * ustride : total);
    return unit_of(make_int4(__shfl_sync(0xFFFFFFFFu, a.v.x, turn & 31), __shfl_sync(0xFFFFFFFFu, a.v.y, turn & 31),
                             __shfl_sync(0xFFFFFFFFu, a.v.z, turn & 31), __shfl_sync(0xFFFFFFFFu, a.v.w, turn & 31)));
  };
  auto look_ahead = [&](int turn, int4* next) {
    if (turn % kExpAhead != 0) return;
    __syncwarp();
    if (lane < kExpAhead) next[lane] = place(turn + lane < turns ? unit0 + (turn + lane) * ustride : total);
    __syncwarp();
  };
  // A wait of the whole warp, by every lane.
  auto all_await = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, detail::wait_bounded<true>(bar, parity, abort_flag, err, P.budget)) != 0;
  };
  // The same, of which one lane polls.
  auto warp_await = [&](uint32_t bar, uint32_t parity) {
    int ready = 0;
    if (lane == 0) ready = detail::wait_bounded<true>(bar, parity, abort_flag, err, P.budget) ? 1 : 0;
    ready = __shfl_sync(0xFFFFFFFFu, ready, 0);
    // The other lanes see what the polling one acquired, and the warp is one again
    // for the instructions that ask for it (.aligned).
    __syncwarp();
    return ready != 0;
  };
  // Rows of the box that brings a half of B: the least of 16, 32, 64 and 128 that
  // hold it.  (Two boxes that hold just it cost the loading thread more than the
  // bytes do.)
  auto box_of = [&](const Unit& t) { return kDw || t.half > 64 ? 0 : t.half > 32 ? 1 : t.half > 16 ? 2 : 3; };
  auto b_bytes_of = [&](const Unit& t) { return 16384u >> box_of(t); };
  // Rows of zeros behind the `left` of a stage that ends in others': 16 in one box,
  // of which those past a multiple of 16 are not read, or as many as the stage has
  // room for.
  auto zeros_of = [](int left) { return left <= kBlockK - 16 ? 16 : kBlockK - left; };
  // Bytes of A in k-block kb of a unit, and of B.
  auto a_bytes = [&](const Unit& t, int kb) {
    const int left = t.rows - kb * kK;
    return kDw && others_rows(left) ? 256u * static_cast<uint32_t>(left + zeros_of(left)) : static_cast<uint32_t>(kABytes);
  };
  auto b_bytes = [&](const Unit& t, int kb) { return kDw ? a_bytes(t, kb) : b_bytes_of(t); };

  const long long drain = P.budget > kExpDrain ? P.budget : kExpDrain;
  if (warp < S::kRoles) {
    if (warp == 0 || warp == 3) {
      // ----------------------------------------------------------- producers
      const bool loads_a = warp == 0;
      // The operands were written by other kernels' ordinary stores.
      if (lane == 0) ptx::fence_proxy_async_global();
      int4* next = turns_sh[loads_a ? 0 : 1];
      int stage = 0, fills = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int turn = 0; turn < turns; ++turn) {
        look_ahead(turn, next);
        if (lane != 0 || !ok) continue;
        const Unit t = unit_of(next[turn % kExpAhead]);
        // Features or columns, or rows, that this CTA's part starts at.
        const int b_at = kDw ? t.J * kTileN + crank * (kTileN / 2) : t.row0 + crank * t.half;
        const int at = loads_a ? t.I * kTileM : b_at;
        const CUtensorMap* tm = loads_a ? &P.tmA : &P.tmB[box_of(t)];
        const int z = loads_a && !kDw ? t.e : 0;
        int k0 = kDw ? t.row0 : 0;
        for (int kb = 0; kb < t.kbs; kb += kPer, k0 += kPer * kK) {
          ok = detail::wait_bounded<true>(empty(stage), phase ^ 1u, abort_flag, err, P.budget);
          if (!ok) break;
          const uint32_t to = smem_base + stage * S::kStageBytes + (loads_a ? 0 : kPer * kABytes);
          const bool two = kPer == 2 && kb + 1 < t.kbs;
          const uint32_t fb = ptx::mapa(full(stage), 0);
          if (loads_a && leader) {
            const uint32_t bytes = a_bytes(t, kb) + b_bytes(t, kb);
            ptx::mbar_arrive_expect_tx(full(stage), two ? 4 * bytes : 2 * bytes);
          }
          bool tail = false;
          if constexpr (kDw) {
            const int left = t.rows - kb * kK;
            tail = others_rows(left);
            if (tail) {
              // To `row` on of the stage, from row `from` of x or dy on; zeros from behind
              // the last.  (A box may start at any row of the swizzle's pattern of 8, which
              // goes by the shared-memory address.)
              auto box = [&](int row, int map, int from) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  ptx::tma_load_3d_pair(to + c * EC::kMnChunkBytes + row * 128, &P.tail[loads_a ? 0 : 1][map], fb,
                                        at + c * EC::kMnChunk, from, 0);
              };
              auto few = [&](int row, int n, int from, bool zeros) {
                const int n4 = n & 12, n1 = n & 3;
                if (n4 != 0) box(row, 2 + n4 / 4, from);
                if (n1 != 0) box(row + n4, n1 - 1, zeros ? from : from + n4);
              };
              const int n16 = left & 48, zeros = zeros_of(left);
              if (n16 != 0) box(0, 5 + n16 / 16, k0);
              few(n16, left & 15, k0 + n16, false);
              if (zeros == 16)
                box(left, 6, P.rows);
              else
                few(left, zeros, P.rows, true);
            }
          }
          if (tail) {
          } else if (loads_a ? kAMn : kBMn) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              ptx::tma_load_3d_pair(to + c * EC::kMnChunkBytes, tm, fb, at + c * EC::kMnChunk, k0, z);
          } else {
            ptx::tma_load_3d_pair(to, tm, fb, k0, at, z);
            if (two) ptx::tma_load_3d_pair(to + (loads_a ? kABytes : S::kBBytes), tm, fb, k0 + kK, at, z);
          }
          ++fills;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (lane == 0) {
        fills_sh[loads_a ? 0 : 1] = fills;
        // The last release of each stage is awaited here, so that after a full
        // run no commit is on its way to this CTA's barriers when it leaves.
        for (int i = fills > kStages ? fills - kStages : 0; ok && i < fills; ++i)
          ok = detail::wait_bounded<true>(empty(i % kStages), (i / kStages) & 1, abort_flag, err, P.budget);
      }
    } else if (warp == 1) {
      if (leader) {
        // -------------------------------------------------------- MMA issuer
        // The whole warp walks the units and waits, so that what the loop uses is the
        // same in all lanes and stays in uniform registers, and one lane issues, which
        // has waited itself.  (As code of one lane, 4 MMAs and their commit took 275
        // to 470 cycles, so 125 to 143; the MMAs take 128 each at most.  8192^3: 1744
        // TFLOP/s, so 1870 to 1923.)
        const bool one = elect_one();
        // Operand descriptors of the first stage.
        const uint64_t ad0 = kAMn ? ptx::sw128_desc(smem_base, EC::kMnChunkBytes, 1024) : ptx::sw128_desc(smem_base, 16, 1024);
        const uint64_t bd0 = kBMn ? ptx::sw128_desc(smem_base + kABytes, EC::kMnChunkBytes, 1024)
                                  : ptx::sw128_desc(smem_base + kPer * kABytes, 16, 1024);
        constexpr int kAStep = (kAMn ? EC::kMnStep : 32) >> 4, kBStep = (kBMn ? EC::kMnStep : 32) >> 4;
        int stage = 0, buf = 0, stages = 0, units = 0;
        uint32_t phase = 0, tphase = 0;
        bool ok = true;
        auto next_buf = [&] {
          if (one) ptx::mma_commit_pair(tfull(buf), 0x3);
          ++units;
          if (++buf == kBufs) {
            buf = 0;
            tphase ^= 1u;
          }
        };
        Ahead ahead;
        for (int turn = 0; ok && turn < turns; ++turn) {
          const Unit t = unit_at(turn, ahead);
          if (kDw && t.kbs == 0) continue;
          const uint32_t idesc = MODE == kExp8 ? ptx::idesc_e4m3_f32(2 * kTileM, 2 * t.half)
                                               : ptx::idesc_bf16_f32(2 * kTileM, 2 * t.half, kAMn, kBMn);
          if (MODE != kExp8) ok = all_await(tempty(buf), tphase ^ 1u);
          for (int kb = 0; ok && kb < t.kbs; kb += kPer) {
            // kExp8: an accumulator's two parts are the two k-blocks of a stage, which
            // the epilogue scales.
            if (MODE == kExp8) ok = all_await(tempty(buf), tphase ^ 1u);
            ok = ok && all_await(full(stage), phase);
            if (!ok) break;
            ptx::tc_fence_after();
            if (one) {
              const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kTileN);
              const uint64_t ad = ad0 + static_cast<uint32_t>(stage * (S::kStageBytes >> 4));
              const uint64_t bd = bd0 + static_cast<uint32_t>(stage * (S::kStageBytes >> 4));
              const int left = t.rows - kb * kK;
              if (MODE == kExp8) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                  if (j > 0 && kb + j >= t.kbs) break;
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_f8_pair(d_tmem + j * S::kRows, ad + j * (kABytes >> 4) + kk * kAStep,
                                     bd + j * (S::kBBytes >> 4) + kk * kBStep, idesc, kk != 0 ? 1u : 0u);
                }
              } else if (kDw && left < kK) {
                for (int kk = 0; kk * EC::kMmaK < left; ++kk)
                  ptx::mma_bf16_pair(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, (kb != 0 || kk != 0) ? 1u : 0u);
              } else {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  ptx::mma_bf16_pair(d_tmem, ad + kk * kAStep, bd + kk * kBStep, idesc, (kb != 0 || kk != 0) ? 1u : 0u);
              }
              ptx::mma_commit_pair(empty(stage), 0x3);
            }
            ++stages;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
            if (MODE == kExp8) next_buf();
          }
          if (MODE != kExp8 && ok) next_buf();
        }
        if (one) {
          ptx::mma_commit_pair(mma_done, 0x1);
          detail::drain_wait<true>(mma_done, 0, drain);
          stages_sh = stages;
          units_sh = units;
        }
      }
    } else if (warp == 2) {
      if (MODE == kExp8) {
        // ----------------------------------------------------------- scales
        // Of the tile's rows, times that of the CTA's 128 rows of W, 8 k-blocks
        // together: a row's are next to one another.  (A k-block at a time, and by
        // each of the epilogue's warps for itself, the gathers of 4 bytes a row took
        // the SM's whole L1: 436 to 530 us.)
        const int mblocks = (P.m + 127) / 128;
        float* to = reinterpret_cast<float*>(smem + S::kScalesAt) + lane;
        int half = 0;
        uint32_t phase = 0;
        bool ok = true;
        Ahead ahead;
        for (int turn = 0; ok && turn < turns; ++turn) {
          const Unit t = unit_at(turn, ahead);
          // (A tile's upper half may lie past the features: any scale will do.)
          const int mb = t.I < mblocks ? t.I : mblocks - 1;
          const float* ws = P.ws + (static_cast<long long>(t.e) * mblocks + mb) * t.kbs;
          const float* xs = P.xs + static_cast<long long>(t.row0 + lane) * t.kbs;
          for (int kb0 = 0; kb0 < t.kbs; kb0 += kExpScales) {
            // All loads at once, before the wait: one latency for the lot.
            float v[S::kRows / 32][kExpScales];
#pragma unroll
            for (int r = 0; r < S::kRows / 32; ++r)
#pragma unroll
              for (int j = 0; j < kExpScales; ++j)
                v[r][j] = 32 * r + lane < t.rows && kb0 + j < t.kbs ? xs[static_cast<long long>(32 * r) * t.kbs + kb0 + j] : 0.0f;
            const float w = lane < kExpScales && kb0 + lane < t.kbs ? ws[kb0 + lane] : 0.0f;
            ok = warp_await(sempty(half), phase ^ 1u);
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < kExpScales; ++j) {
              const float wj = __shfl_sync(0xFFFFFFFFu, w, j);
#pragma unroll
              for (int r = 0; r < S::kRows / 32; ++r) to[(half * kExpScales + j) * S::kRows + 32 * r] = v[r][j] * wj;
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sfull(half));
            half ^= 1;
            if (half == 0) phase ^= 1u;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    // Warp e reads TMEM lane quarter warp % 4 (32 features) and half of the
    // tile's columns.
    const int e = warp - S::kRoles, q = warp & 3, h = e >> 2;
    const uint32_t stg = smem_base + S::kStagingAt + static_cast<uint32_t>(e * S::kStaging);
    int buf = 0, shalf = 0;
    uint32_t tphase = 0, sphase = 0;
    bool failed = false;
    // The pair's next MMAs write both CTAs' accumulators: one arrival a warp, on
    // CTA 0's barrier: tcgen05.wait::ld and the fence have made sure that the
    // accumulator has been read.  (Not on CTA 0's own with a release either: 8192^3 in
    // 8 bits took 561 us for 549.)
    auto release = [&] {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_pair_relaxed(tempty(buf));
    };
    auto await = [&](uint32_t bar, uint32_t parity) {
      if (failed) return;
      // (All lanes of kExp8's poll, whose epilogue bounds it: 475 us became 436.)
      failed = MODE == kExp8 ? !all_await(bar, parity) : !warp_await(bar, parity);
      __syncwarp();
      ptx::tc_fence_after();
    };
    auto next_buf = [&] {
      if (++buf == kBufs) {
        buf = 0;
        tphase ^= 1u;
      }
    };
    // What the bulk stores add to or write over was written by other kernels' ordinary
    // stores.
    if (MODE == kExpDwF32 && lane == 0) ptx::fence_proxy_async_global();
    Ahead ahead;
    for (int turn = 0; turn < turns; ++turn) {
      if (MODE == kExp8) look_ahead(turn, turns_sh[MODE == kExp8 ? 2 + e : 0]);
      const Unit t = MODE == kExp8 ? unit_of(turns_sh[MODE == kExp8 ? 2 + e : 0][turn % kExpAhead]) : unit_at(turn, ahead);
      const int feature0 = t.I * kTileM + q * 32;
      const uint32_t t_warp = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      if constexpr (!kDw) {
        const int width = 2 * t.half / (S::kEpi / 4), c0 = h * width;  // the warp's columns
        // 32 columns of the accumulator (c on, of this warp's half), whose 8-column
        // groups g are the fragments f(i, 4 g ..): rows of y through the staging
        // box, 64 bytes a row.
        auto put = [&](int c, const auto& word) {
          __syncwarp();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            // Thread 8 m + j addresses column j of the 8 features m.
            const int tok = 8 * g + (lane & 7), m = lane >> 3;
            ptx::st_matrix_trans(stg + tok * 64 + ((m ^ ((tok >> 1) & 3)) << 4), word(0, 4 * g), word(0, 4 * g + 2),
                                 word(1, 4 * g), word(1, 4 * g + 2));
          }
          __syncwarp();
          const int f = feature0 + (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = 8 * i + (lane >> 2);
            if (c + tok < width && c0 + c + tok < t.rows && f < P.m) {
              uint32_t w[4];
              ptx::ld_shared_v4(stg + tok * 64 + (((lane & 3) ^ ((tok >> 1) & 3)) << 4), w);
              ptx::st_global_v4(static_cast<bf16*>(P.out) + static_cast<long long>(t.row0 + c0 + c + tok) * P.m + f, w[0], w[1],
                                w[2], w[3]);
            }
          }
        };
        if constexpr (MODE != kExp8) {
          await(tfull(buf), tphase);
          const uint32_t t_at = t_warp + static_cast<uint32_t>(buf * kTileN + c0);
#pragma unroll 1
          for (int c = 0; c < width; c += 32) {
            uint32_t v[2][16];
            if (!failed) {
              ptx::tmem_ld_16x32cols(t_at + c, v[0]);
              ptx::tmem_ld_16x32cols(t_at + (16u << 16) + c, v[1]);
              ptx::tmem_wait_ld();
              loaded(v[0]);
              loaded(v[1]);
              if (c + 32 >= width) release();
            }
            put(c, [&](int i, int k) {
              return failed ? kExpNan : detail::pack_bf16x2(__uint_as_float(v[i][k]), __uint_as_float(v[i][k + 1]));
            });
          }
          next_buf();
        } else {
          // Each k-block's products are sums of e4m3 products in fp32; they are
          // scaled and added here, in fp32 registers.
          const float* scales = reinterpret_cast<const float*>(smem + S::kScalesAt) + c0 + 2 * (lane & 3);
          float2 acc[2][8];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[i][k] = both(0.0f);
#pragma unroll 1
          for (int kb = 0; kb < t.kbs; kb += 2) {
            if (kb % kExpScales == 0) await(sfull(shalf), sphase);
            await(tfull(buf), tphase);
            if (failed) break;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (kb + b == t.kbs) break;
              const float* of = scales + (shalf * kExpScales + kb % kExpScales + b) * S::kRows;
              // 32 columns, whatever the tile holds, so that no load is conditional.
              uint32_t v[2][16];
              const uint32_t t_at = t_warp + static_cast<uint32_t>(buf * kTileN + b * S::kRows + c0);
              ptx::tmem_ld_16x32cols(t_at, v[0]);
              ptx::tmem_ld_16x32cols(t_at + (16u << 16), v[1]);
              ptx::tmem_wait_ld();
              loaded(v[0]);
              loaded(v[1]);
              if (b == 1 || kb + 1 == t.kbs) release();
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const float2 sc = *reinterpret_cast<const float2*>(of + 8 * g);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int k = 2 * g; k < 2 * g + 2; ++k)
                    acc[i][k] = fma2(make_float2(__uint_as_float(v[i][2 * k]), __uint_as_float(v[i][2 * k + 1])), sc, acc[i][k]);
              }
            }
            next_buf();
            if ((kb + 2) % kExpScales == 0 || kb + 2 >= t.kbs) {
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(sempty(shalf));
              shalf ^= 1;
              if (shalf == 0) sphase ^= 1u;
            }
          }
          put(0, [&](int i, int k) { return failed ? kExpNan : detail::pack_bf16x2(acc[i][k >> 1].x, acc[i][k >> 1].y); });
        }
      } else {
        const int row = feature0 + lane, col0 = t.J * kTileN + h * (kTileN / 2);
        const bool none = t.kbs == 0;  // no rows: zero, or nothing to add
        if (none && P.add) continue;
        if (!none) await(tfull(buf), tphase);
        const uint32_t t_at = t_warp + static_cast<uint32_t>(buf * kTileN + h * (kTileN / 2));
        if (!none && !failed && col0 >= P.n) release();  // nothing to read
#pragma unroll 1
        for (int c = 0; c < kTileN / 2; c += 32) {
          const int gj = col0 + c;
          if (gj >= P.n) break;  // warp-uniform
          uint32_t v[32];
          if (none || failed) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = failed ? kExpNan : 0u;
          } else {
            ptx::tmem_ld_32cols(t_at + c, v);
            ptx::tmem_wait_ld();
            loaded(v);
            if (c + 32 == kTileN / 2 || gj + 32 >= P.n) release();
          }
          if (MODE == kExpDwBf16) {
            if (row < P.m) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 16; ++k)
                w[k] = failed ? kExpNan : detail::pack_bf16x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
              bf16* to = static_cast<bf16*>(P.out) + (static_cast<long long>(t.e) * P.m + row) * P.n + gj;
              if (P.sectors && gj + 32 <= P.n) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
                  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 16 * g),
                               "r"(w[8 * g]), "r"(w[8 * g + 1]), "r"(w[8 * g + 2]), "r"(w[8 * g + 3]), "r"(w[8 * g + 4]),
                               "r"(w[8 * g + 5]), "r"(w[8 * g + 6]), "r"(w[8 * g + 7])
                               : "memory");
              } else {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                  if (gj + 8 * g < P.n) ptx::st_global_v4(to + 8 * g, w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
              }
            }
          } else {
            if (lane == 0) ptx::bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 8; ++g)
              ptx::st_shared_v4(stg + stage_off32(lane, 4 * g), v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && feature0 < P.m) {
              if (P.add)
                asm volatile(
                    "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                        reinterpret_cast<uint64_t>(&P.tmOut)),
                    "r"(gj), "r"(feature0), "r"(t.e), "r"(stg)
                    : "memory");
              else
                ptx::tma_store_3d(&P.tmOut, stg, gj, feature0, t.e);
              ptx::bulk_commit();
            }
          }
        }
        if (!none) next_buf();
      }
    }
    // The staging boxes stay until the bulk stores are done.
    if (kDw) {
      if (lane == 0) ptx::bulk_wait_all();
      __syncwarp();
    }
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
    // arrival has been awaited by the role that it was for; after a wait that ran
    // out the loading threads may have asked for different numbers of fills.
    // Copies of a fill are counted on the first CTA's barrier, which expects those
    // of both CTAs once its own A is asked for; the first CTA stands in for what is
    // missing.
    auto remote = [](const int* p, int rank) {
      int v;
      asm volatile("ld.shared::cluster.s32 %0, [%1];"
                   : "=r"(v)
                   : "r"(ptx::mapa(ptx::smem_u32(p), static_cast<uint32_t>(rank)))
                   : "memory");
      return v;
    };
    auto stand_in = [](uint32_t bar, uint32_t bytes) {
      if (bytes > 0)
        asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
    };
    const int fills[4] = {fills_sh[0], fills_sh[1], remote(&fills_sh[0], crank ^ 1), remote(&fills_sh[1], crank ^ 1)};
    int top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fills[i] > top ? fills[i] : top;
    int turn = 0, before_turn = 0;  // the turn of fill i, and the fills before it
    Unit t = unit_of(place(unit0));
    for (int i = top > kStages ? top - kStages : 0; i < top; ++i) {
      while (i - before_turn >= (t.kbs + kPer - 1) / kPer) {
        before_turn += (t.kbs + kPer - 1) / kPer;
        t = unit_of(place(unit0 + ++turn * ustride));
      }
      const int s = i % kStages;
      const uint32_t n = kPer == 2 && 2 * (i - before_turn) + 1 < t.kbs ? 2 : 1;  // k-blocks of the fill
      const int kb = kPer * (i - before_turn);
      const uint32_t A = n * a_bytes(t, kb), B = n * b_bytes(t, kb);
      const uint32_t own = (i < fills[0] ? A : 0) + (i < fills[1] ? B : 0);
      const uint32_t peer = (i < fills[2] ? A : 0) + (i < fills[3] ? B : 0);
      if (leader) {
        if (i < fills[0])
          stand_in(ptx::mapa(full(s), 0), 2 * (A + B) - own - peer);
        else
          ptx::mbar_arrive_expect_tx(full(s), own + peer);
        detail::drain_wait<true>(full(s), (i / kStages) & 1, drain);
      }
    }
    const int stages = remote(&stages_sh, 0), units = remote(&units_sh, 0);
    for (int i = stages > kStages ? stages - kStages : 0; i < stages; ++i)
      detail::drain_wait<true>(empty(i % kStages), (i / kStages) & 1, drain);
    for (int i = units > kBufs ? units - kBufs : 0; i < units; ++i)
      detail::drain_wait<true>(tfull(i % kBufs), (i / kBufs) & 1, drain);
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
