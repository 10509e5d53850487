// The router's choice, its plan, and its gradient.
//
// A token takes the k experts of largest logit z (ties to the lower index; one of
// -inf or NaN is not to be had).  Its gates are softmax(z) at them, over all
// experts or, renormalised, over the chosen ones.  The plan sorts the choices by
// expert, then by token: offsets[e] is the first row of expert e, slots[t][j] the
// row of a choice, tokens[row] its token.
//
// A warp holds a token's logits, E / 32 a lane, and takes the largest k times (two
// integer reductions a time).  A CTA's tokens (32 or 128, or up to 256 in one CTA) mark
// their bit in a mask for each expert, so a choice's place among its expert's in
// the tile is a count of lower bits: no sort, and no atomics whose order shows.
// Many tokens: tiles leave their counts of each expert, a second kernel adds those
// of the tiles before, a third places the choices.  Bound by latency for few
// tokens, for many by the k reductions of the choice.
#include "lm/common.cuh"
#include "muon_moe.h"

namespace mns {
namespace lm {

namespace {

constexpr int kRouteExperts = 1024;
constexpr int kRouteMost = 32;    // choices of a token
// Tokens that one CTA takes alone.  (One CTA and three launches: 64 tokens of 128
// experts, k 8, 6.6 us and 7.6, 256 of them 20.7 and 7.9; of 320 experts 64 tokens
// 16.5 and 13.1, 256 57 and 13.7.  256 stands because up to as many are promised to
// need no workspace.)
constexpr int kOneTile = 256;

struct Route {
  const void* logits;
  long long tokens;
  int experts, k, renormalize;
  float* gates;
  int* chosen;
  int* slots;
  int* token_of;
  int* offsets;
  int* counts;  // [tiles][experts], then of the tiles before
  int* totals;  // [experts]
};

// Order of logits as integers: 0 for one that is not to be had.  -0 is 0.
__device__ __forceinline__ uint32_t order_of(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// The choice of one token, by a warp, of its logits z: lane j < k <= KM gets the
// expert (or -1) and the gate of choice j.
template <typename T, int J, int KM>
__device__ __forceinline__ int choose(const T* z, int experts, int k, bool renormalize, float* gate) {
  const int lane = threadIdx.x & 31;
  float v[J];
  uint32_t o[J], e[J];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    e[j] = lane + 32 * j;
    v[j] = static_cast<int>(e[j]) < experts ? to_f32(z[e[j]]) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    bad |= v[j] != v[j];
    o[j] = order_of(v[j]);
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  // Up to 4 a lane are put in order once, so that its largest is always at hand;
  // more are searched every time.
  constexpr bool kSorted = J <= 4;
  if (kSorted) {
    // (Insertion: only neighbours change places, so equal ones keep their order.)
#pragma unroll
    for (int n = 1; n < J; ++n)
#pragma unroll
      for (int a = n; a > 0; --a) {
        const bool up = o[a] > o[a - 1];
        const uint32_t x = up ? o[a] : o[a - 1], y = up ? o[a - 1] : o[a];
        const uint32_t f = up ? e[a] : e[a - 1], g = up ? e[a - 1] : e[a];
        o[a - 1] = x;
        o[a] = y;
        e[a - 1] = f;
        e[a] = g;
      }
  }
  int mine = -1;
  uint32_t mine_o = 0u, first = 0u;
#pragma unroll
  for (int i = 0; i < KM; ++i) {
    if (i >= k) break;
    uint32_t best = o[0], of = e[0];
    if (!kSorted) {
#pragma unroll
      for (int j = 1; j < J; ++j)
        if (o[j] > best) {
          best = o[j];
          of = e[j];
        }
    }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    if (top == 0u) break;  // none left
    const uint32_t taken = __reduce_min_sync(0xFFFFFFFFu, best == top ? of : ~0u);
    if (i == 0) first = top;
    if (lane == i) {
      mine = static_cast<int>(taken);
      mine_o = top;
    }
    // (An expert is in one lane's list, so its number alone tells whose it was.)
    if (kSorted) {
      const bool was = of == taken;
#pragma unroll
      for (int j = 1; j < J; ++j) {
        o[j - 1] = was ? o[j] : o[j - 1];
        e[j - 1] = was ? e[j] : e[j - 1];
      }
      o[J - 1] = was ? 0u : o[J - 1];
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (e[j] == taken) o[j] = 0u;
    }
  }
  const float top = value_of(first);
  const float p = mine >= 0 ? expf(value_of(mine_o) - top) : 0.0f;
  float sum = p;
  if (!renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) sum += first != 0u && lane + 32 * j < experts ? expf(v[j] - top) : 0.0f;
  }
  sum = warp_sum(sum);
  *gate = bad ? __uint_as_float(0x7FFFFFFFu) : mine >= 0 ? p / sum : 0.0f;
  return mine;
}

// Tokens of the tile before bit b whose mask of WORDS words says so.
template <int WORDS>
__device__ __forceinline__ int bits_below(const uint32_t* mask, int b) {
  int n = 0;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    const int left = b - 32 * w;
    if (left > 0) n += __popc(left >= 32 ? mask[w] : mask[w] & ((1u << left) - 1u));
  }
  return n;
}

// Exclusive sums of n <= 1024 counts, by one warp; `total` after them.
__device__ __forceinline__ void offsets_of(const int* counts, int n, int* before) {
  const int lane = threadIdx.x & 31;
  int sum = 0;
  for (int e0 = 0; e0 < n; e0 += 32) {
    const int mine = e0 + lane < n ? counts[e0 + lane] : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (e0 + lane < n) before[e0 + lane] = sum + upto - mine;
    sum += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  if (lane == 0) before[n] = sum;
}

// ONE: all tokens, by one CTA, and the whole plan.  Else the choices of a tile of
// TILE tokens and how many each expert has of it.
template <typename T, int J, bool ONE, int TILE>
__global__ void __launch_bounds__(ONE ? 1024 : 512) route_choose(const Route R) {
  constexpr int kTokens = TILE, kWords = TILE / 32;
  extern __shared__ uint32_t mask[];  // [experts][kWords], then (ONE) int [experts] and [experts + 1]
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x / 32;
  for (int i = threadIdx.x; i < R.experts * kWords; i += blockDim.x) mask[i] = 0u;
  __syncthreads();
  const long long t0 = static_cast<long long>(blockIdx.x) * kTokens;
  const int n = R.tokens - t0 < kTokens ? static_cast<int>(R.tokens - t0) : kTokens;
  for (int i = warp; i < n; i += warps) {
    float gate;
    const T* z = static_cast<const T*>(R.logits) + (t0 + i) * R.experts;
    const bool renormalize = R.renormalize != 0;
    const int e = R.k <= 8 ? choose<T, J, 8>(z, R.experts, R.k, renormalize, &gate)
                           : choose<T, J, kRouteMost>(z, R.experts, R.k, renormalize, &gate);
    if (lane < R.k) {
      R.gates[(t0 + i) * R.k + lane] = gate;
      R.chosen[(t0 + i) * R.k + lane] = e;
      if (e >= 0) atomicOr(&mask[e * kWords + (i >> 5)], 1u << (i & 31));
    }
  }
  __syncthreads();
  int* count = ONE ? reinterpret_cast<int*>(mask + R.experts * kWords)
                   : R.counts + static_cast<long long>(blockIdx.x) * R.experts;
  for (int e = threadIdx.x; e < R.experts; e += blockDim.x) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) c += __popc(mask[e * kWords + w]);
    count[e] = c;
  }
  if (!ONE) return;
  __syncthreads();
  int* before = count + R.experts;
  if (warp == 0) offsets_of(count, R.experts, before);
  __syncthreads();
  for (int e = threadIdx.x; e <= R.experts; e += blockDim.x) R.offsets[e] = before[e];
  for (int i = threadIdx.x; i < n * R.k; i += blockDim.x) {
    const int t = i / R.k, e = R.chosen[i];
    int slot = -1;
    if (e >= 0) {
      slot = before[e] + bits_below<kWords>(mask + e * kWords, t);
      R.token_of[slot] = t;
    }
    R.slots[i] = slot;
    if (i >= before[R.experts]) R.token_of[i] = -1;
  }
}

// Counts of the tiles before, in place, and of all: a CTA takes 32 experts, its
// warps consecutive parts of the tiles.
__global__ void __launch_bounds__(1024) route_scan(int* counts, int tiles, int experts, int* totals) {
  __shared__ int part[32][33];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
  const int i0 = static_cast<int>(static_cast<long long>(tiles) * warp / 32), i1 = static_cast<int>(static_cast<long long>(tiles) * (warp + 1) / 32);
  int sum = 0;
  if (e < experts) {
#pragma unroll 8
    for (int i = i0; i < i1; ++i) sum += counts[static_cast<long long>(i) * experts + e];
  }
  part[warp][lane] = sum;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += part[w][lane];
  if (e < experts) {
#pragma unroll 8
    for (int i = i0; i < i1; ++i) {
      const int c = counts[static_cast<long long>(i) * experts + e];
      counts[static_cast<long long>(i) * experts + e] = at;
      at += c;
    }
    if (warp == 31) totals[e] = at;
  }
}

// Places a tile's choices.
template <int TILE>
__global__ void __launch_bounds__(512) route_place(const Route R) {
  constexpr int kWords = TILE / 32;
  extern __shared__ uint32_t mask[];  // [experts][kWords], then int [experts + 1]
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5;
  int* before = reinterpret_cast<int*>(mask + R.experts * kWords);
  for (int i = threadIdx.x; i < R.experts * kWords; i += blockDim.x) mask[i] = 0u;
  ptx::griddep_wait();
  __syncthreads();
  const long long t0 = static_cast<long long>(blockIdx.x) * TILE;
  const int n = R.tokens - t0 < TILE ? static_cast<int>(R.tokens - t0) : TILE;
  const int* chosen = R.chosen + t0 * R.k;
  if (warp == 0) offsets_of(R.totals, R.experts, before);
  for (int i = threadIdx.x; i < n * R.k; i += blockDim.x) {
    const int e = chosen[i], t = i / R.k;
    if (e >= 0) atomicOr(&mask[e * kWords + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  const int* tile = R.counts + static_cast<long long>(blockIdx.x) * R.experts;
  for (int i = threadIdx.x; i < n * R.k; i += blockDim.x) {
    const int e = chosen[i], t = i / R.k;
    int slot = -1;
    if (e >= 0) {
      slot = before[e] + tile[e] + bits_below<kWords>(mask + e * kWords, t);
      R.token_of[slot] = static_cast<int>(t0 + t);
    }
    R.slots[t0 * R.k + i] = slot;
    if (t0 * R.k + i >= before[R.experts]) R.token_of[t0 * R.k + i] = -1;
  }
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= R.experts; e += blockDim.x) R.offsets[e] = before[e];
}

// Gradient of the gates.  With inner = sum_j dg_j g_j over the choices, dz at
// choice j is g_j (dg_j - inner), and elsewhere -p inner, p the softmax over all
// experts; 0 where the gates are renormalised.
//
// Where one gate is nearly 1, inner is nearly its dg, and what is left of the
// difference would be rounding.  So at the choices, with m that of the largest gate,
// d_j = dg_j - dg_m and `rest` the sum of p elsewhere,
//   dz_j = g_j (d_j - sum_i g_i d_i + dg_m rest):
// at m the first term is 0 and what remains are the small terms themselves.
//
// Over all experts a warp takes a token (J logits a lane).  (65536 tokens of 128
// experts, k 8: 23.3 us; with dg - inner, as first written, 19.9.)
template <typename T, int J>
__global__ void __launch_bounds__(256)
    route_grad(const float* dgates, const T* logits, const int* chosen,
               long long tokens, int experts, int k, T* dlogits) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  for (long long t = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < tokens; t += gridDim.x * 8LL) {
    const T* z = logits + t * experts;
    int e = lane < k ? chosen[t * k + lane] : -1;
    if (e >= experts) e = -1;
    const float dg = e >= 0 ? dgates[t * k + lane] : 0.0f;
    const float c = e >= 0 ? to_f32(z[e]) : -INFINITY;
    float p[J];
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = lane + 32 * j < experts ? to_f32(z[lane + 32 * j]) : -INFINITY;
    float top = p[0];
#pragma unroll
    for (int j = 1; j < J; ++j) top = fmaxf(top, p[j]);
    top = warp_max(top);
    const float own = e >= 0 ? expf(c - top) : 0.0f;
    float rest = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      // (A token without any expert to be had has no gradient.)
      p[j] = lane + 32 * j < experts && top != -INFINITY ? expf(p[j] - top) : 0.0f;
      const uint32_t chosen_of = __reduce_or_sync(0xFFFFFFFFu, e >= 0 && e >> 5 == j ? 1u << (e & 31) : 0u);
      if (!(chosen_of >> lane & 1u)) rest += p[j];
    }
    const uint32_t bits = __float_as_uint(own), most = __reduce_max_sync(0xFFFFFFFFu, bits);
    const uint32_t at_top = __ballot_sync(0xFFFFFFFFu, e >= 0 && bits == most);
    const float ref = __shfl_sync(0xFFFFFFFFu, dg, at_top != 0u ? __ffs(at_top) - 1 : 0);
    const float d = e >= 0 ? dg - ref : 0.0f;
    // In units of 1 / sum, sum = have + rest.
    const float have = warp_sum(own), left = warp_sum(d * own);
    rest = warp_sum(rest);
    const float sum = have + rest, inner = left + ref * have;
    const float factor = sum == 0.0f ? 0.0f : -(inner / sum) / sum;
    T* out = dlogits + t * experts;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane + 32 * j < experts) out[lane + 32 * j] = from_f32<T>(p[j] * factor);
    __syncwarp();  // the choices' places are written again, by other lanes
    if (e >= 0) out[e] = from_f32<T>(own / sum * (d - left / sum + ref * (rest / sum)));
  }
}

// Over the choices alone G >= k lanes take a token, and its row is zeroed by the
// warp in accesses of V elements.
template <typename T, int G, int V>
__global__ void __launch_bounds__(256)
    route_grad_chosen(const float* dgates, const T* logits, const int* chosen,
                      long long tokens, int experts, int k, T* dlogits) {
  constexpr int kTokens = 32 / G;  // of a warp
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, j = lane & (G - 1);
  const long long t0 = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kTokens;
  const long long t = t0 + lane / G;
  const bool live = t < tokens && j < k;
  int e = live ? chosen[t * k + j] : -1;
  if (e >= experts) e = -1;
  const float dg = e >= 0 ? dgates[t * k + j] : 0.0f;
  const float c = e >= 0 ? to_f32(logits[t * experts + e]) : -INFINITY;
  // The rows of the warp's tokens lie next to one another.
  const long long n = (t0 + kTokens < tokens ? kTokens : tokens > t0 ? tokens - t0 : 0) * experts;
  T* out = dlogits + t0 * experts;
  const float none[V] = {};
  for (long long i = lane * V; i < n; i += 32 * V) store_global<T, V>(out + i, none);
  float top = c;
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float own = e >= 0 ? expf(c - top) : 0.0f;
  auto total = [](float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  };
  const float sum = total(own);
  const float g = e >= 0 ? own / sum : 0.0f;
  const uint32_t group = (G == 32 ? 0xFFFFFFFFu : (1u << (G & 31)) - 1u) << (lane & ~(G - 1));
  const uint32_t at_top = __ballot_sync(0xFFFFFFFFu, e >= 0 && c == top) & group;
  const float ref = __shfl_sync(0xFFFFFFFFu, dg, at_top != 0u ? __ffs(at_top) - 1 : lane);
  const float d = e >= 0 ? dg - ref : 0.0f;
  const float left = total(d * g);
  __syncwarp();  // the choices' places are written again, by other lanes
  if (e >= 0) dlogits[t * experts + e] = from_f32<T>(g * (d - left));
}

template <typename F>
auto with_lanes(int experts, F&& f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>{});
  if (experts <= 64) return f(std::integral_constant<int, 2>{});
  if (experts <= 128) return f(std::integral_constant<int, 4>{});
  if (experts <= 256) return f(std::integral_constant<int, 8>{});
  if (experts <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

int route_check(long long tokens, int experts, int k, int type) {
  if (tokens < 0 || experts < 1 || experts > kRouteExperts || k < 1 || k > kRouteMost || k > experts)
    return MUON_NS_ERR_INVALID_ARG;
  // Rows of choices are 32-bit numbers.
  if (tokens > kMaxRows || tokens * k > kMaxRows || !type_ok(type)) return MUON_NS_ERR_INVALID_ARG;
  return MUON_NS_OK;
}

// Tokens of a tile: 32, or 128 for many, whose counts are then fewer.  (Of 128
// experts, k 8, in tiles of 32 and of 128: 4000 tokens 12.1 us and 18.0, 16385 16.3
// and 30.9, 30000 26.9 and 36.2, 65536 49.0 and 44.0; of 512 21.5 and 39, 36.6 and 61,
// 62 and 66, 124 and 120.)
int route_tile(long long tokens) { return tokens <= 1024 * 32 ? 32 : 128; }
long long route_tiles(long long tokens) {
  const int tile = route_tile(tokens);
  return tokens <= kOneTile ? 0 : (tokens + tile - 1) / tile;
}

}  // namespace

}  // namespace lm
}  // namespace mns

using namespace mns::lm;

extern "C" {

int muon_route_workspace_size(long long tokens, int experts, int k, size_t* bytes) {
  const int st = route_check(tokens, experts, k, MUON_LM_F32);
  if (st != MUON_NS_OK) return st;
  if (!bytes) return MUON_NS_ERR_INVALID_ARG;
  const long long tiles = route_tiles(tokens);
  *bytes = tiles == 0 ? 0 : align_up(sizeof(int) * static_cast<size_t>(tiles + 1) * experts, 256);
  return MUON_NS_OK;
}

int muon_route(const void* logits, int type, long long tokens, int experts, int k, int renormalize, float* gates,
               int* chosen, int* slots, int* token_of, int* offsets, void* workspace, size_t workspace_bytes,
               cudaStream_t stream) {
  int st = route_check(tokens, experts, k, type);
  if (st != MUON_NS_OK) return st;
  if (!offsets || (tokens > 0 && (!logits || !gates || !chosen || !slots || !token_of))) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(logits, type)) return MUON_NS_ERR_ALIGNMENT;
  for (const void* p : {static_cast<const void*>(gates), static_cast<const void*>(chosen), static_cast<const void*>(slots),
                        static_cast<const void*>(token_of), static_cast<const void*>(offsets)})
    if (!element_aligned(p, MUON_LM_F32)) return MUON_NS_ERR_ALIGNMENT;
  size_t need = 0;
  muon_route_workspace_size(tokens, experts, k, &need);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return MUON_NS_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MUON_NS_ERR_ALIGNMENT;
  }
  const size_t zb = static_cast<size_t>(tokens) * experts * type_size(type), gb = 4 * static_cast<size_t>(tokens) * k;
  const void* arrays[] = {logits, workspace, gates, chosen, slots, token_of, offsets};
  const size_t bytes[] = {zb, need, gb, gb, gb, gb, 4 * (static_cast<size_t>(experts) + 1)};
  for (int i = 1; i < 7; ++i)
    for (int j = 0; j < i; ++j)
      if (bytes[i] > 0 && bytes[j] > 0 && overlap(arrays[i], bytes[i], arrays[j], bytes[j])) return MUON_NS_ERR_INVALID_ARG;
  if ((st = muon_ns_device_supported(-1)) != MUON_NS_OK) return st;
  if (tokens == 0) return status_of(cudaMemsetAsync(offsets, 0, sizeof(int) * (experts + 1), stream));
  Route R = {};
  R.logits = logits;
  R.tokens = tokens;
  R.experts = experts;
  R.k = k;
  R.renormalize = renormalize ? 1 : 0;
  R.gates = gates;
  R.chosen = chosen;
  R.slots = slots;
  R.token_of = token_of;
  R.offsets = offsets;
  const long long tiles = route_tiles(tokens);
  R.totals = static_cast<int*>(workspace);
  R.counts = R.totals + (tiles > 0 ? experts : 0);
  const int tile = route_tile(tokens);
  const unsigned ctas = static_cast<unsigned>(tiles);
  st = with_type(type, [&](auto tt) {
    using T = decltype(tt);
    return with_lanes(experts, [&](auto jc) {
      constexpr int J = decltype(jc)::value;
      if (tiles == 0) {
        const size_t smem = sizeof(int) * (static_cast<size_t>(experts) * (kOneTile / 32 + 2) + 1);
        const unsigned warps = static_cast<unsigned>(tokens < 4 ? 4 : tokens < 32 ? tokens : 32);
        return status_of(mns::launch_pdl(route_choose<T, J, true, kOneTile>, dim3(1), dim3(32 * warps), smem, stream, R));
      }
      const size_t smem = sizeof(int) * static_cast<size_t>(experts) * (tile / 32);
      if (tile == 32) return status_of(mns::launch_pdl(route_choose<T, J, false, 32>, dim3(ctas), dim3(512), smem, stream, R));
      return status_of(mns::launch_pdl(route_choose<T, J, false, 128>, dim3(ctas), dim3(512), smem, stream, R));
    });
  });
  if (st != MUON_NS_OK || tiles == 0) return st;
  st = status_of(mns::launch_pdl(route_scan, dim3(static_cast<unsigned>((experts + 31) / 32)), dim3(1024), 0, stream,
                                 R.counts, static_cast<int>(tiles), experts, R.totals));
  if (st != MUON_NS_OK) return st;
  const size_t smem = sizeof(int) * (static_cast<size_t>(experts) * (tile / 32 + 1) + 1);
  if (tile == 32) return status_of(mns::launch_pdl(route_place<32>, dim3(ctas), dim3(512), smem, stream, R));
  return status_of(mns::launch_pdl(route_place<128>, dim3(ctas), dim3(512), smem, stream, R));
}

int muon_route_grad(const float* dgates, const void* logits, int type, const int* chosen, long long tokens, int experts,
                    int k, int renormalize, void* dlogits, cudaStream_t stream) {
  int st = route_check(tokens, experts, k, type);
  if (st != MUON_NS_OK) return st;
  if (tokens == 0) return MUON_NS_OK;
  if (!dgates || !logits || !chosen || !dlogits) return MUON_NS_ERR_INVALID_ARG;
  if (!element_aligned(logits, type) || !element_aligned(dlogits, type) || !element_aligned(dgates, MUON_LM_F32) ||
      !element_aligned(chosen, MUON_LM_F32))
    return MUON_NS_ERR_ALIGNMENT;
  const size_t zb = static_cast<size_t>(tokens) * experts * type_size(type), gb = 4 * static_cast<size_t>(tokens) * k;
  if (overlap(dlogits, zb, logits, zb) || overlap(dlogits, zb, dgates, gb) || overlap(dlogits, zb, chosen, gb))
    return MUON_NS_ERR_INVALID_ARG;
  if ((st = muon_ns_device_supported(-1)) != MUON_NS_OK) return st;
  return with_type(type, [&](auto tt) {
    using T = decltype(tt);
    const T* z = static_cast<const T*>(logits);
    T* dz = static_cast<T*>(dlogits);
    if (!renormalize) {
      const long long need = (tokens + 7) / 8, most = 64LL * sm_count();
      const dim3 grid(static_cast<unsigned>(need < most ? need : most));
      return with_lanes(experts, [&](auto jc) {
        constexpr int J = decltype(jc)::value;
        return status_of(mns::launch_pdl(route_grad<T, J>, grid, dim3(256), 0, stream, dgates, z, chosen, tokens, experts, k, dz));
      });
    }
    // (The rows of a warp's tokens start as aligned as the first where a row is a
    // multiple of the access.)
    return with_vec(vec_of(experts, dlogits, type), [&](auto vc) {
      constexpr int V = decltype(vc)::value;
      auto launch = [&](auto gc) {
        constexpr int G = decltype(gc)::value;
        const long long ctas = (tokens + 8 * (32 / G) - 1) / (8 * (32 / G));
        return status_of(mns::launch_pdl(route_grad_chosen<T, G, V>, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, stream,
                                         dgates, z, chosen, tokens, experts, k, dz));
      };
      if (k <= 8) return launch(std::integral_constant<int, 8>{});
      if (k <= 16) return launch(std::integral_constant<int, 16>{});
      return launch(std::integral_constant<int, 32>{});
    });
  });
}

}  // extern "C"
