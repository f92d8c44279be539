// The whole layer for a few tokens (T <= 64, one token tile), with bf16, fp32
// or 4-bit expert weights, and products of single rows with 4-bit weights.
//
// With few tokens nothing is computed often enough to matter: the layer is the
// read of the chosen experts' matrices, 3 d d_ff elements each, once for every
// 16 (or 32) of an expert's copies. So the weights go from memory straight into
// the matrix instructions' operand registers: the weight tile is the A operand
// (16 output features by 32 columns), up to 16 of the expert's tokens are the 16
// columns of B, and no weight passes through LDS; what every wave needs of x and
// of the scales does, in the wave's own part of it, without barriers.
//
// Four launches: the router's scores (matrix cores, fp64 sums), the choice of
// experts with the lists of their copies (one work-group), the gate and up
// products with h = silu(g) u, and the down product with the combine. With one
// token of a DeepSeek-V3-shaped layer (d = 7168, d_ff = 2048, 8 of 256 experts)
// they take 5.8, 8.1, 75 and 45 us in bf16 (705 MB of weights at 5.9 TB/s in the
// two products), and 5.8, 8.1, 27 and 17 us in u4 (184 MB at 4.2).
//
// Nothing here depends on the order in which work-groups run: every sum has a
// fixed order, and the expert lists are built by ranks, not by arrival.
#include "common.h"
#include "few.h"
#include "q4.h"

#include <algorithm>
#include <climits>
#include <cmath>

namespace moe {
namespace {

constexpr int kRouterWaves = 8, kRouterThreads = 64 * kRouterWaves;

enum WKind { kDenseBf16, kDenseF32, kU4, kE2m1 };

// ---------------------------------------------------------------------------
// Router scores. Block (expert tile, token tile, K slice); its waves split the
// slice. Products and sums are taken in fp64 on the matrix cores, where products
// of bf16 or fp32 numbers are exact: a score is off by at most (d + 16) 2^-53
// times the sum of its products' magnitudes, so the scores' order is decided far
// below fp32's rounding, and sums in another order pick the same experts unless
// their scores are that close. Bound by latency: W_router (3.7 MB at E = 256, d =
// 7168) over 128 work-groups and then 32 products of four columns a wave, one
// after the other, 5.8 us for one token; 9.0 us and 56 products for 64 tokens.
// (Four waves a work-group, with twice as many products each: 1 us more.)
// ---------------------------------------------------------------------------
typedef double f64x4 __attribute__((ext_vector_type(4)));

// The numbers of a 16-byte piece.
template <bool BF16>
__device__ inline double piece_value(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (BF16) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  return __uint_as_float(w[i]);
}

template <bool BF16>
__global__ __launch_bounds__(kRouterThreads) void few_router_kernel(const void* xv, const void* wv, int T, int E, int64_t d,
                                                              int S, double* __restrict__ part,
                                                              bf16_t* __restrict__ parts) {
  __shared__ double red[kRouterWaves][64][4];
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16, s = blockIdx.z;
  const int64_t block = (static_cast<int64_t>(s) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t nthreads = static_cast<int64_t>(gridDim.x) * gridDim.y * gridDim.z * kRouterThreads;
  if (!BF16 && parts) split_rows(static_cast<const float*>(xv), T * d, parts, block * kRouterThreads + threadIdx.x, nthreads);
  constexpr int kStep = BF16 ? 32 : 16, kVec = BF16 ? 8 : 4;
  const int64_t steps = ceil_div(d, kStep);
  const int64_t j0 = steps * (s * kRouterWaves + wave) / (S * kRouterWaves), j1 = steps * (s * kRouterWaves + wave + 1) / (S * kRouterWaves);
  const int64_t er = std::min(e0 + col, E - 1), tr = std::min(t0 + col, T - 1);
  const char* wr = static_cast<const char*>(wv) + er * d * (16 / kVec);
  const char* xr = static_cast<const char*>(xv) + tr * d * (16 / kVec);
  f64x4 acc = {0, 0, 0, 0};
  constexpr int U = 8;  // steps whose loads are in flight together
  for (int64_t j = j0; j < j1; j += U) {
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past the end the last piece again, and 0 for x (d is a multiple of kVec)
      const int64_t c = (j + u) * kStep + kVec * quad;
      const int64_t at = std::min(c, d - kVec) * (16 / kVec);
      a[u] = *reinterpret_cast<const uint4*>(wr + at);
      b[u] = *reinterpret_cast<const uint4*>(xr + at);
      if (j + u >= j1 || c >= d) a[u] = b[u] = uint4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u >= j1) break;
#pragma unroll
      for (int i = 0; i < kVec; ++i)  // lane: column c + i of expert row lane % 16 and of token lane % 16
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64(piece_value<BF16>(a[u], i), piece_value<BF16>(b[u], i), acc, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][lane][i] = acc[i];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  // thread: element i of lane l, i.e. expert row 4 i + l / 16 and token l % 16
  const int l = threadIdx.x >> 2, i = threadIdx.x & 3;
  double v = 0;
#pragma unroll
  for (int w = 0; w < kRouterWaves; ++w) v += red[w][l][i];
  const int e = e0 + 4 * i + (l >> 4), t = t0 + (l & 15);
  if (e < E && t < T) part[(static_cast<int64_t>(s) * T + t) * E + e] = v;
}

// ---------------------------------------------------------------------------
// Top-k, gates, slots and the experts' token lists: one work-group, a wave a
// token, so that the lists need no second launch. Bound by latency, k rounds of
// a maximum over a wave in a row (each by register shifts; scores loaded
// together): 5 us (4 tokens, E = 8) to 27 us (64 tokens, E = 256, k = 8, where
// the products after it take 3 ms). With more than 256 experts a lane holds 16
// scores, and the kernel spills about 80 registers (330 bytes a lane).
// ---------------------------------------------------------------------------

// Monotone map of a double to uint64 and back; NaN sorts below every number
// (its choice is unspecified, but stays a distinct expert), and 0 is below NaN.
__device__ inline uint64_t order_key(double v) {
  if (v != v) return 1;
  v += 0.0;  // -0.0 -> +0.0
  const uint64_t u = __double_as_longlong(v);
  return (u >> 63) ? ~u : (u | (uint64_t{1} << 63));
}
__device__ inline double key_value(uint64_t k) {
  return __longlong_as_double((k >> 63) ? (k & ~(uint64_t{1} << 63)) : ~k);
}

// The largest of a wave's 64 values, in every lane: partial maxima move up the
// lanes by register shifts (within 16, then across rows), without LDS.
__device__ inline uint32_t wave_max(uint32_t v) {
  v = std::max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true)));  // by 1
  v = std::max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true)));  // by 2
  v = std::max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true)));  // by 4
  v = std::max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true)));  // by 8
  v = std::max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xf, 0xf, true)));  // lane 15 on
  v = std::max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xf, 0xf, true)));  // lane 31 on
  return __builtin_amdgcn_readlane(v, 63);
}

// The best (key, then lowest expert) of a wave's candidates, one a lane; *win is
// the lane that holds it. Two candidates seldom share the key's upper half.
__device__ inline void wave_best(uint64_t key, int e, uint64_t* best_key, int* best_e, int* win) {
  const uint32_t hi = key >> 32, lo = static_cast<uint32_t>(key);
  const uint32_t mh = wave_max(hi);
  unsigned long long c = __ballot(hi == mh);
  uint32_t ml;
  if (__popcll(c) == 1) {
    ml = __builtin_amdgcn_readlane(lo, __ffsll(c) - 1);
  } else {
    ml = wave_max(hi == mh ? lo : 0u);
    c = __ballot(hi == mh && lo == ml);
    if (__popcll(c) > 1) {
      const bool mine = hi == mh && lo == ml;
      const uint32_t first = ~wave_max(mine ? ~static_cast<uint32_t>(e) : 0u);
      c = __ballot(mine && static_cast<uint32_t>(e) == first);
    }
  }
  *win = __ffsll(c) - 1;
  *best_e = __builtin_amdgcn_readlane(e, *win);
  *best_key = (static_cast<uint64_t>(mh) << 32) | ml;
}

struct RouteOut {
  int32_t* idx;     // [T, k]
  float* w;         // [T, k]
  int32_t* slot;    // [T, k] or NULL
  int32_t* routed;  // [E] or NULL
  int32_t* kept;    // [E] or NULL
  int32_t* send;    // [P] or NULL
  int64_t* totals;  // or NULL
};

struct Scores {
  const double* part;  // [S][T][E]
  int S;
  const float* bias;
  int T, E, k, P, M;
};

// Token t's experts and gates, by one wave: lane j < k gets the j-th best
// expert and its gate. rbest: the wave's LDS for 64 ranks' best scores.
template <int NE>  // scores a lane holds: E <= 64 NE
__device__ inline void choose(const Scores& a, int t, unsigned long long* rbest, int* expert, float* gate) {
  const int lane = threadIdx.x & 63, T = a.T, E = a.E, k = a.k, P = a.P, M = a.M, S = a.S, per = E / P;
  const double* __restrict__ part = a.part;
  const float* __restrict__ bias = a.bias;
  uint64_t key[NE];
  constexpr int G = NE < 4 ? NE : 4;  // experts a lane whose partial scores are fetched together
#pragma unroll
  for (int i0 = 0; i0 < NE; i0 += G) {
    double v[kFewMaxSplits][G];
#pragma unroll
    for (int s = 0; s < kFewMaxSplits; ++s)
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int e = lane + 64 * (i0 + i);
        v[s][i] = 0;
        if (s < S && e < E) v[s][i] = part[(static_cast<int64_t>(s) * T + t) * E + e];
      }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int e = lane + 64 * (i0 + i);
      double sum = v[0][i];
#pragma unroll
      for (int s = 1; s < kFewMaxSplits; ++s) sum += v[s][i];
      if (bias && e < E) sum += static_cast<double>(bias[e]);
      key[i0 + i] = e < E ? order_key(sum) : 0;
    }
  }
  if (M > 0 && M < P) {  // P <= 64: lane p holds rank p's best score
    rbest[lane] = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane + 64 * i < E) atomicMax(&rbest[(lane + 64 * i) / per], static_cast<unsigned long long>(key[i]));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    const uint64_t mine = rbest[lane];
    int ahead = 0;  // ranks ahead of mine: better score, or equal score and lower index
    for (int p = 0; p < P; ++p) {
      const uint64_t q = rbest[p];
      ahead += (q > mine || (q == mine && p < lane)) ? 1 : 0;
    }
    const uint64_t allowed = __ballot(lane < P && ahead < M);
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane + 64 * i < E && !((allowed >> ((lane + 64 * i) / per)) & 1)) key[i] = 0;
  }
  uint64_t sel = 0, top = 0;
  int sel_e = 0;
  for (int r = 0; r < k; ++r) {
    uint64_t mine = key[0], best;
    int me = lane, e, win;
#pragma unroll
    for (int i = 1; i < NE; ++i)
      if (key[i] > mine) {
        mine = key[i];
        me = lane + 64 * i;
      }
    wave_best(mine, me, &best, &e, &win);
    if (r == 0) top = best;
    if (lane == r) {
      sel = best;
      sel_e = e;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (e == lane + 64 * i) key[i] = 0;
  }
  const double z = lane < k ? exp(key_value(sel) - key_value(top)) : 0.0;
  double sum = z;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  *expert = sel_e;
  *gate = static_cast<float>(z / sum);
}

template <int NE>
__global__ __launch_bounds__(1024) void few_route_kernel(Scores sc, int64_t C, int64_t row_bytes, RouteOut o,
                                                         FewLists ls) {
  __shared__ int cnt[kFewMaxE], ecp[kFewMaxCopies], rank[kFewMaxCopies], scratch[kRankChunkInts];
  __shared__ unsigned long long rbest[16][64];
  __shared__ int wsum[17], send_s[64], dropped_tokens;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int T = sc.T, E = sc.E, k = sc.k, P = sc.P, per = E / P;
  for (int e = tid; e < E; e += 1024) cnt[e] = 0;
  if (tid == 0) dropped_tokens = 0;
  for (int i = tid; i < ls.n_done; i += 1024) ls.done[i] = 0;
  for (int t = wave; t < T; t += 16) {
    int e;
    float w;
    choose<NE>(sc, t, rbest[wave], &e, &w);
    if (lane < k) {
      o.idx[t * k + lane] = e;
      o.w[t * k + lane] = w;
      ecp[t * k + lane] = e;
    }
  }
  __syncthreads();

  const int n = T * k;
  if (tile_ranks_by_waves(k, E)) {
    rank_tile_waves(ecp, n, E, cnt, scratch, rank);
  } else if (wave == 0) {
    rank_tile(ecp, n, E, cnt, rank);
  }
  __syncthreads();

  // exclusive scan over the experts of (has kept copies, kept copies)
  const int routed = tid < E ? cnt[tid] : 0;
  const int kept = static_cast<int>(std::min<int64_t>(routed, C));
  const int mine = ((kept > 0) << 16) | kept;
  int inc = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(inc, off);
    if (lane >= off) inc += up;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < 16; ++w) {
    if (w < wave) before += wsum[w];
    all += wsum[w];
  }
  const int excl = before + inc - mine;
  if (tid < E) {
    cnt[tid] = excl & 0xffff;  // now the expert's first position
    if (kept > 0) {
      ls.act_e[excl >> 16] = tid;
      ls.act_off[excl >> 16] = excl & 0xffff;
    }
    if (o.routed) o.routed[tid] = routed;
    if (o.kept) o.kept[tid] = kept;
  }
  const int total = all & 0xffff;
  if (tid == 0) {
    *ls.n_act = all >> 16;
    ls.act_off[all >> 16] = total;
  }
  // kept copies of each rank's send buffer: order-free integer sums
  if (o.send || o.totals) {
    if (P <= 64) {
      if (tid < P) send_s[tid] = 0;
      __syncthreads();
      if (tid < E && kept) atomicAdd(&send_s[tid / per], kept);
      __syncthreads();
      if (o.send && tid < P) o.send[tid] = send_s[tid];
    } else {  // then a rank holds at most 16 experts
      scratch[tid] = kept;
      __syncthreads();
      if (tid < P) {
        int c = 0;
        for (int q = 0; q < per; ++q) c += scratch[tid * per + q];
        if (o.send) o.send[tid] = c;
        if (tid == 0) send_s[0] = c;
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += 1024) {
    const int r = rank[i];
    const bool keep = r < C;
    const int pos = keep ? cnt[ecp[i]] + r : -1;
    if (keep) {
      ls.token[pos] = i / k;
      ls.gate[pos] = o.w[i];  // written by this work-group before the barriers above
    }
    if (o.slot) o.slot[i] = keep ? r : -1;
  }
  if (o.totals) {
    for (int t = tid; t < T; t += 1024) {
      bool any = false;
      for (int j = 0; j < k; ++j) any |= rank[t * k + j] < C;
      if (!any) atomicAdd(&dropped_tokens, 1);
    }
    __syncthreads();
    if (tid == 0) {
      o.totals[0] = n - total;
      o.totals[1] = dropped_tokens;
      o.totals[2] = E * C - total;
      o.totals[3] = static_cast<int64_t>(total - send_s[0]) * row_bytes;
    }
  }
}

// The same for at most 64 copies (T k <= 64) and 64 ranks: one wave holds all
// copies and takes an expert's copies at a time, by a ballot, in place of the
// larger kernel's scans and their barriers (4 tokens, E = 8: 6.5 -> 4.9 us; one
// token, E = 256: 8.5 -> 7.9 us).
template <int NE>
__global__ __launch_bounds__(1024) void few_route_small_kernel(Scores sc, int64_t C, int64_t row_bytes, RouteOut o,
                                                               FewLists ls) {
  __shared__ int ecp[64], send_s[64];
  __shared__ float gate[64];
  __shared__ unsigned long long rbest[16][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int T = sc.T, E = sc.E, k = sc.k, P = sc.P, n = T * k;
  for (int e = tid; e < E; e += blockDim.x) {
    if (o.routed) o.routed[e] = 0;
    if (o.kept) o.kept[e] = 0;
  }
  if (tid < 64) send_s[tid] = 0;
  for (int i = tid; i < ls.n_done; i += blockDim.x) ls.done[i] = 0;
  for (int t = wave; t < T; t += waves) {
    int e;
    float w;
    choose<NE>(sc, t, rbest[wave], &e, &w);
    if (lane < k) {
      o.idx[t * k + lane] = e;
      o.w[t * k + lane] = w;
      ecp[t * k + lane] = e;
      gate[t * k + lane] = w;
    }
  }
  __syncthreads();
  if (wave > 0) return;
  const bool in = lane < n;
  const int e = in ? ecp[lane] : -1;
  const unsigned long long below = (1ull << lane) - 1ull;
  int experts = 0, total = 0;  // experts listed so far (by their first copies), and their kept copies
  for (unsigned long long left = __ballot(in); left;) {
    const int its = __builtin_amdgcn_readlane(e, __ffsll(left) - 1);
    const unsigned long long mine = __ballot(e == its);
    const int rank = __popcll(mine & below), copies = __popcll(mine);
    const int kept = static_cast<int>(std::min<int64_t>(copies, C));  // C >= 1: an expert with copies keeps its first
    if (e == its) {
      if (rank < kept) {
        ls.token[total + rank] = lane / k;
        ls.gate[total + rank] = gate[lane];
      }
      if (o.slot) o.slot[lane] = rank < kept ? rank : -1;
      if (rank >= kept) ecp[lane] = -1;  // dropped
      if (rank == 0) {
        ls.act_e[experts] = e;
        ls.act_off[experts] = total;
        if (o.routed) o.routed[e] = copies;
        if (o.kept) o.kept[e] = kept;
        atomicAdd(&send_s[e / (E / P)], kept);  // order-free
      }
    }
    ++experts;
    total += kept;
    left &= ~mine;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  if (o.send && lane < P) o.send[lane] = send_s[lane];
  // tokens none of whose k copies is kept
  bool lost = lane < T;
  if (lost)
    for (int j = 0; j < k; ++j) lost &= ecp[lane * k + j] < 0;
  const int lost_tokens = __popcll(__ballot(lost));
  if (lane == 0) {
    *ls.n_act = experts;
    ls.act_off[experts] = total;
    if (o.totals) {
      o.totals[0] = n - total;
      o.totals[1] = lost_tokens;
      o.totals[2] = E * C - total;
      o.totals[3] = static_cast<int64_t>(total - send_s[0]) * row_bytes;
    }
  }
}

// ---------------------------------------------------------------------------
// Products of NS strips of 16 weight rows with NT tiles of 16 rows of x over a
// range of the contraction: acc[r][t] += W_r x_t^T, one 16 x 16 tile in the
// matrix instructions' layout (lane: token lane % 16, features 4 (lane / 16) + i).
// The range is in units of a strip's memory: 128-byte lines of dense rows,
// 128-column tiles of 4-bit ones.
// ---------------------------------------------------------------------------

constexpr bool is_dense(WKind k) { return k == kDenseBf16 || k == kDenseF32; }

// Waves a SIMD that the registers are cut for: as many as fit with at most a few
// spilled words (20 bytes a lane). A spill's own loads and stores make every wait
// one for all loads in flight.
constexpr int waves_per_simd(int parts, bool wide) { return parts == 3 ? 2 : wide ? 3 : 4; }

template <WKind KIND>
using XType = std::conditional_t<KIND == kDenseF32, float, bf16_t>;

// Units of a contraction of K columns.
template <WKind KIND>
__host__ __device__ inline int units_of(int64_t K) {
  return static_cast<int>(KIND == kDenseBf16 ? ceil_div(K, 64) : KIND == kDenseF32 ? ceil_div(K, 32) : ceil_div(K, 128));
}

// One matrix stack [E, N, K] as the kernels take it.
struct WMat {
  int64_t E;            // matrices
  const void* w;        // dense rows, or code tiles
  const bf16_t* scale;  // 4-bit only
  const uint8_t* zero;  // u4 only; NULL: 8
};

// The zero points of u4 weights that have none: read like others, over and
// over (a branch around the reads instead made the compiler copy whole tiles'
// work and spill).
__device__ const uint8_t kEights[16] __attribute__((aligned(16))) = {8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8, 8};

// A value that is the same in every lane, in a scalar register.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The lane's number, computed again where it is used: what follows from it is
// then not kept in registers from one use to the next.
__device__ inline int lane_here() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// Memory from `base` on, `bytes` long, for loads at a common base (in scalar
// registers) plus a lane's 32-bit offset. A lane past the end gets 0 and touches
// nothing, which also stands in for loads under a condition.
struct Span {
  const char* base;
  uint32_t bytes;

  __device__ inline uint32_t load4(uint32_t lane_off, uint32_t off) const {
    const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), static_cast<short>(0),
                                                     static_cast<int>(bytes), 0x00020000);
    return __builtin_amdgcn_raw_buffer_load_b32(r, static_cast<int>(lane_off), static_cast<int>(off), 0);
  }
  template <bool ONCE>  // read once: not to be kept in the caches
  __device__ inline auto load16(uint32_t lane_off, uint32_t off) const {
    const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), static_cast<short>(0),
                                                     static_cast<int>(bytes), 0x00020000);
    return __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(lane_off), static_cast<int>(off), ONCE ? 2 : 0);
  }
};
__device__ inline Span span(const void* base, int64_t bytes) {
  return Span{static_cast<const char*>(base), static_cast<uint32_t>(std::min<int64_t>(bytes, 0x7ffffff0ll))};
}
constexpr uint32_t kNowhere = 0x80000000u;  // a lane's offset past every span

// One strip: its weights from their first line or tile to the end of the
// matrices, and each lane's offset there (dense: of its pieces of rows 0 - 7
// and, `hi` further, of rows 8 - 15); the scales and zero points of its groups.
template <WKind KIND>
struct Strip {
  Span w, scale, zero;
  int zstep;             // bytes from one group's zero points to the next group's
  uint32_t lo, hi;
  int last;              // dense: the row's last line,
  bool past;             // and whether the lane's piece of that is past the row's end
};

// n rows of x (at most 64), and in lane c row c's offset.
struct Rows {
  Span first;
  int64_t part;  // bytes from one bf16 part of fp32 rows to the next
  uint32_t off;
  int n;
  __device__ inline Span of_part(int p) const { return Span{first.base + p * part, first.bytes}; }
};

// n rows of `stride` bytes in x, row `row` in lane c for c < n. The rows'
// numbers may still be on their way when the weights are asked for.
struct RowList {
  Span x;
  int64_t stride, part;
  int n, row;
  __device__ inline Rows rows() const {
    return Rows{x, part, static_cast<uint32_t>(row) * static_cast<uint32_t>(stride), n};
  }
};

// Dense strips are read in whole 128-byte lines, eight rows an instruction:
// lane l takes piece (l / 16) + 4 (l / 8 % 2) of row l % 8. Loads that take
// half lines of all 16 rows, as the operand layout has them, must leave the
// line in the cache for the other half and reach 5.9 TB/s; whole lines can
// stream past it (non-temporal) at 6.6 - 6.9 TB/s. Two such loads hold the
// operands of two steps, up to a rotation by eight lanes (operands()).
__device__ inline int piece_of(int lane) { return (lane >> 4) + 4 * ((lane >> 3) & 1); }

// Rows r0 .. r0 + 15 of matrix e (both the same for all lanes). What lies past
// the matrix is not stored, whatever is read there: the next matrix or, past
// the last one, 0.
template <WKind KIND, int GPT>
__device__ inline Strip<KIND> strip_of(const WMat& m, int64_t e, int64_t r0, int64_t N, int64_t K) {
  const int lane = threadIdx.x & 63;
  Strip<KIND> s = {};
  if constexpr (is_dense(KIND)) {
    const int64_t row = K * sizeof(XType<KIND>), at = (e * N + r0) * row;
    s.w = span(static_cast<const char*>(m.w) + at, m.E * N * row - at);
    s.lo = (lane & 7) * static_cast<uint32_t>(row) + piece_of(lane) * 16;
    s.last = static_cast<int>(ceil_div(row, 128)) - 1;
    s.past = s.last * 128 + piece_of(lane) * 16 >= row;
    // without rows 8 - 15 rows 0 - 7 again: a common offset past the span's end is no test of its end
    s.hi = r0 + 8 < N ? 8 * static_cast<uint32_t>(row) : 0;
  } else {
    const int64_t nt = ceil_div(N, 16), kt = ceil_div(K, 128), t = (e * nt + r0 / 16) * kt;
    s.w = span(static_cast<const char*>(m.w) + t * 1024, kt * 1024);
    s.lo = lane * 16;
    s.scale = span(m.scale + t * GPT * 16, kt * GPT * 32);
    s.zstep = m.zero ? 16 : 0;
    s.zero = span(m.zero ? m.zero + t * GPT * 16 : kEights, m.zero ? kt * GPT * 16 : 16);
  }
  return s;
}

// Groups of a tile between two marks of multiply().
template <WKind KIND, int NS>
constexpr int kMarkEvery = NS == 1 ? (KIND == kU4 ? 2 : 4) : 1;

__device__ inline u32x4 load_once(const Span& s, uint32_t lane_off, uint32_t off) {
  return __builtin_bit_cast(u32x4, s.load16<true>(lane_off, off));
}
__device__ inline u32x4 load_kept(const Span& s, uint32_t lane_off, uint32_t off = 0) {
  return __builtin_bit_cast(u32x4, s.load16<false>(lane_off, off));
}

template <WKind KIND>
__device__ inline f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (KIND == kDenseF32) {
    const f32x4 av = __builtin_bit_cast(f32x4, a), bv = __builtin_bit_cast(f32x4, b);
#pragma unroll  // the four columns go to four instructions: any order of k will do
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(av[i], bv[i], c, 0, 0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
}

// 4-bit strips: the codes enter the matrix instruction as 16 + q (u4) or as
// their value (e2m1), exact in bf16; each group's sum is scaled in fp32:
//   sum_k s (q - z) x = s (sum (16 + q) x - (16 + z) sum x),
// the last sum by one more instruction with a tile of ones. The offset is 16
// and not larger because the difference loses as many bits as it exceeds q.
// PARTS = 3: fp32 x as the exact sum of three bf16 arrays.

// One unit's weights, as loaded. Past the end of a dense row that ends inside
// its last line they are 0, as x is: what follows in memory may be NaN.
template <WKind KIND, int NS>
struct UnitW {
  u32x4 w[NS][is_dense(KIND) ? 2 : 1];
};

template <WKind KIND, int NS>
__device__ inline void load_weights(const Strip<KIND> (&a)[NS], int j, UnitW<KIND, NS>& u) {
#pragma unroll
  for (int r = 0; r < NS; ++r)
    if constexpr (is_dense(KIND)) {
      const uint32_t lo = j == a[r].last && a[r].past ? kNowhere : a[r].lo;
      u.w[r][0] = load_once(a[r].w, lo, j * 128);
      u.w[r][1] = load_once(a[r].w, lo, j * 128 + a[r].hi);
    } else {
      u.w[r][0] = load_once(a[r].w, a[r].lo, j * 1024);
    }
}

// x and the scales of a run of units, staged in the wave's own LDS: one wave's
// loads of x from the caches would otherwise pace it (x takes four times the
// registers that the 4-bit codes it meets do, so it cannot be asked for as far
// ahead, and a load takes about 1 us when all of them wait for memory). The
// next run's loads wait in registers while this one is multiplied.
// LDS of a wave: x [PARTS][rows][run bytes + 16] (the 16 bytes shift each row's
// banks), then fp32 scales [NS][units][GPT][16] and, for u4, -(16 + z) alike:
// converted here once, not by each of the 16 token columns.
//
// A run is up to 4 KiB of x (a part), for ROWS = 1, 4, 16 or (NT = 2) 32 rows: 16,
// 4 or 1 tiles, 32, 8, 2 or 1 lines; one tile (8 KiB) of 32 rows.
// Nothing here is loaded under a condition (lanes past the rows, the units and
// the groups load from nowhere): a load that some path leaves out makes the
// wait for any older one a wait for all of them.
template <WKind KIND, int GPT, int PARTS, int NS, int NT, int ROWS>
struct Stage {
  static constexpr bool kDense = is_dense(KIND);
  static constexpr int kUnitBytes = kDense ? 128 : 256;       // of a row of x (a part)
  static constexpr int kRows = ROWS;
  // no more groups in a run than the lanes hold zero points of
  static constexpr int kUnits = kDense ? 32 / ROWS : std::max(1, std::min(16 / GPT, 16 / ROWS));
  static constexpr int kLoads = (kUnits * kUnitBytes * ROWS + 1023) / 1024;  // 1 KiB each, a part
  static constexpr int kRow = kUnits * kUnitBytes;            // bytes of a row in a run
  static constexpr int kStride = kRow + 16;
  static constexpr int kXBytes = PARTS * kRows * kStride;
  static constexpr int kScale = kUnits * GPT * 64;            // bytes of a strip's scales
  static constexpr int kOff = NS * kScale;
  static constexpr int kBytes = kXBytes + (kDense ? 0 : KIND == kU4 ? 2 * kOff : kOff);
  // words of a strip's scales (two each) and zero points (four each) in a run, a lane
  static constexpr int kScaleWords = (kUnits * GPT * 8 + 63) / 64;
  static_assert(kDense || kUnits * GPT * 4 <= 64, "a lane for each four zero points of a run");

  char* lds;
  uint32_t from[kLoads];  // where this lane's pieces of x are in the first run
  u32x4 x[PARTS][kLoads];
  uint32_t scale[kDense ? 1 : NS][kScaleWords], zero[kDense ? 1 : NS];
  uint32_t at[NT];        // this lane's rows (and piece) in the staged x

  static __device__ inline int row_of(int lane, int u) { return (u * 64 + lane) / (kRow / 16); }
  static __device__ inline int piece(int lane, int u) { return (u * 64 + lane) % (kRow / 16) * 16; }

  __device__ inline void init(char* wave_lds, const Rows& r) {
    const int lane = threadIdx.x & 63;
    lds = wave_lds;
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const uint32_t row = __shfl(r.off, row_of(lane, u) & 63);
      from[u] = row_of(lane, u) < r.n ? row + piece(lane, u) : kNowhere;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)  // columns past n repeat the last row; their results are not stored
      at[t] = std::min(t * 16 + (lane & 15), r.n - 1) * kStride + (lane >> 4) * 16;
  }

  // Asks for units j .. j + kUnits - 1; x and the scales are 0 from unit j1 and
  // from the end of the contraction on.
  __device__ inline void ask(const Strip<KIND> (&a)[NS], const Rows& r, int64_t K, int j, int j1) {
    const int lane = lane_here();
    const int jj = std::min(j, j1 - 1);  // offsets stay inside, also where nothing is wanted
    const int64_t left = K * static_cast<int64_t>(sizeof(XType<KIND>)) - static_cast<int64_t>(j) * kUnitBytes;
    const int bytes = static_cast<int>(std::min<int64_t>(left, static_cast<int64_t>(j1 - j) * kUnitBytes));
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const uint32_t off = piece(lane, u) < bytes ? from[u] : kNowhere;
#pragma unroll
      for (int p = 0; p < PARTS; ++p) x[p][u] = load_kept(r.of_part(p), off, jj * kUnitBytes);
    }
    if constexpr (!kDense) {
      // groups that begin past the end are padding: 0, whatever the arrays hold
      const int groups = static_cast<int>(
          std::min<int64_t>(static_cast<int64_t>(j1 - j) * GPT, ceil_div(K, 128 / GPT) - static_cast<int64_t>(j) * GPT));
#pragma unroll
      for (int r2 = 0; r2 < NS; ++r2) {
#pragma unroll
        for (int k = 0; k < kScaleWords; ++k)
          scale[r2][k] = a[r2].scale.load4(lane + 64 * k < 8 * groups ? (lane + 64 * k) * 4 : kNowhere, jj * GPT * 32);
        if constexpr (KIND == kU4)
          zero[r2] = a[r2].zero.load4(lane < 4 * groups ? (lane & 3) * 4 + (lane >> 2) * a[r2].zstep : kNowhere,
                                      jj * GPT * a[r2].zstep);
      }
    }
  }

  // Puts what was asked for into LDS; the wave's reads of the run before are
  // done (a wave's LDS accesses keep their order).
  __device__ inline void put() {
    const int lane = lane_here();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        *reinterpret_cast<u32x4*>(lds + (p * kRows + row_of(lane, u)) * kStride + piece(lane, u)) = x[p][u];
    if constexpr (!kDense) {
#pragma unroll
      for (int r2 = 0; r2 < NS; ++r2) {
        float2* s = reinterpret_cast<float2*>(lds + kXBytes + r2 * kScale) + lane;
#pragma unroll
        for (int k = 0; k < kScaleWords; ++k)
          if (lane + 64 * k < kUnits * GPT * 8)
            s[64 * k] = float2{__uint_as_float(scale[r2][k] << 16), __uint_as_float(scale[r2][k] & 0xffff0000u)};
        if (KIND == kU4 && lane < kUnits * GPT * 4) {
          f32x4 z;
#pragma unroll
          for (int c = 0; c < 4; ++c) z[c] = -16.f - static_cast<float>((zero[r2] >> (8 * c)) & 0xffu);
          reinterpret_cast<f32x4*>(lds + kXBytes + kOff + r2 * kScale)[lane] = z;
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  }

  // 64 bytes' worth (step q) of unit i of the run, part p, of the row at `at`.
  __device__ inline u32x4 get(int i, uint32_t at, int p, int q) const {
    return *reinterpret_cast<const u32x4*>(lds + p * kRows * kStride + at + i * kUnitBytes + q * 64);
  }
  // Scales, and -(16 + z), of rows 4 quad .. 4 quad + 3 in group g of unit i, strip r.
  __device__ inline f32x4 get_scale(int i, int r, int g, int quad) const {
    return reinterpret_cast<const f32x4*>(lds + kXBytes + r * kScale + (i * GPT + g) * 64)[quad];
  }
  __device__ inline f32x4 get_off(int i, int r, int g, int quad) const {
    return reinterpret_cast<const f32x4*>(lds + kXBytes + kOff + r * kScale + (i * GPT + g) * 64)[quad];
  }
};

// LDS bytes of a wave: the larger of its kinds of run.
template <WKind KIND, int GPT, int PARTS, int NS, bool WIDE>
constexpr int kWaveLds =
    std::max({Stage<KIND, GPT, PARTS, NS, 1, 1>::kBytes, Stage<KIND, GPT, PARTS, NS, 1, 4>::kBytes,
              Stage<KIND, GPT, PARTS, NS, 1, 8>::kBytes, Stage<KIND, GPT, PARTS, NS, 1, 16>::kBytes,
              WIDE ? Stage<KIND, GPT, PARTS, NS, 2, 32>::kBytes : 0});

// acc += unit i of the staged run times its weights.
template <WKind KIND, int GPT, int PARTS, int NS, int NT, int ROWS>
__device__ inline void multiply(const UnitW<KIND, NS>& u, const Stage<KIND, GPT, PARTS, NS, NT, ROWS>& in, int i,
                                f32x4 (&acc)[NS][NT]) {
  if constexpr (is_dense(KIND)) {
    u32x4 x[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q) x[t][q] = in.get(i, in.at[t], 0, q);
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      u32x4 a0, a1;
      operands(u.w[r][0], u.w[r][1], a0, a1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc[r][t] = mma<KIND>(a0, x[t][0], acc[r][t]);
        acc[r][t] = mma<KIND>(a1, x[t][1], acc[r][t]);
      }
    }
  } else {
    constexpr bool kU = KIND == kU4;
    constexpr int kSteps = 4 / GPT;  // 32-column steps of a group
    bf16x8 ones;
#pragma unroll
    for (int c = 0; c < 8; ++c) ones[c] = static_cast<__bf16>(1.0f);
#pragma unroll
    for (int g = 0; g < GPT; ++g) {
      // One group after the other: with these marks neither its LDS reads nor its
      // sums move past its neighbours', which would keep all groups' in registers.
      uint32_t at[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        at[t] = in.at[t];
        if (g % kMarkEvery<KIND, NS> == 0) asm volatile("" : "+v"(at[t]));
      }
      const int quad = g % kMarkEvery<KIND, NS> == 0 ? lane_here() >> 4 : (threadIdx.x & 63) >> 4;
      f32x4 sum[NS][NT] = {}, sx[NT] = {};
#pragma unroll
      for (int st = g * kSteps; st < (g + 1) * kSteps; ++st) {
        bf16x8 v[NS];
#pragma unroll
        for (int r = 0; r < NS; ++r) v[r] = q4_decode<kU>(u.w[r][0][st]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            const bf16x8 xv = __builtin_bit_cast(bf16x8, in.get(i, at[t], p, st));
#pragma unroll
            for (int r = 0; r < NS; ++r)
              sum[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[r], xv, sum[r][t], 0, 0, 0);
            if constexpr (kU) sx[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xv, sx[t], 0, 0, 0);
          }
      }
#pragma unroll
      for (int r = 0; r < NS; ++r) {
        const f32x4 s = in.get_scale(i, r, g, quad);
        f32x4 off = {};
        if constexpr (kU) off = in.get_off(i, r, g, quad);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float v = kU ? fmaf(off[c], sx[t][c], sum[r][t][c]) : sum[r][t][c];
            acc[r][t][c] = fmaf(s[c], v, acc[r][t][c]);
          }
        if ((g + 1) % kMarkEvery<KIND, NS> == 0)
#pragma unroll
          for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(acc[r][t]));
      }
    }
  }
}

// Units j0 .. j1 - 1 of the strips. 4 KiB (4-bit) or 8 KiB (dense) of weights a
// wave are in flight all the time: each place of the ring is asked for again as
// soon as its unit is multiplied (past the range the last unit, from the cache).
// 16 waves a CU keep 64 KiB of 4-bit weights in flight; a ring of 8 KiB spilled
// registers (one token, u4: 75 us for 58; 16 tokens, e2m1: 210 for 168).
template <WKind KIND, int GPT, int PARTS, int NS, int NT, int ROWS>
__device__ inline void mac_run(const Strip<KIND> (&a)[NS], const RowList& list, int64_t K, int j0, int j1, char* lds,
                               f32x4 (&acc)[NS][NT]) {
  using Run = Stage<KIND, GPT, PARTS, NS, NT, ROWS>;
  constexpr int U = 4 / NS, kUnits = Run::kUnits;
  UnitW<KIND, NS> w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load_weights(a, std::min(j0 + u, j1 - 1), w[u]);
  Run in;
  const Rows x = list.rows();
  in.init(lds, x);
  in.ask(a, x, K, j0, j1);
  int i = 0;  // unit of the staged run, where a run has several rounds of the ring
  for (int j = j0; j < j1; j += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kUnits >= U ? u == 0 && i == 0 : u % kUnits == 0) {
        in.put();
        in.ask(a, x, K, j + u + kUnits, j1);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (j + u < j1) multiply<KIND, GPT, PARTS>(w[u], in, kUnits >= U ? i + u : u % kUnits, acc);
      __builtin_amdgcn_sched_barrier(0);
      load_weights(a, std::min(j + u + U, j1 - 1), w[u]);
    }
    if (kUnits > U) i = (i + U) % kUnits;
  }
}

template <WKind KIND, int GPT, int PARTS, int NS, int NT>
__device__ inline void mac(const Strip<KIND> (&a)[NS], const RowList& list, int64_t K, int j0, int j1, char* lds,
                           f32x4 (&acc)[NS][NT]) {
  if (j0 >= j1) return;
  if constexpr (NT == 1) {
    if (list.n > (is_dense(KIND) ? 4 : 8))
      mac_run<KIND, GPT, PARTS, NS, NT, 16>(a, list, K, j0, j1, lds, acc);
    else if constexpr (is_dense(KIND))
      mac_run<KIND, GPT, PARTS, NS, NT, 4>(a, list, K, j0, j1, lds, acc);
    else {
      if (list.n == 1)
        mac_run<KIND, GPT, PARTS, NS, NT, 1>(a, list, K, j0, j1, lds, acc);
      else if (list.n <= 4)
        mac_run<KIND, GPT, PARTS, NS, NT, 4>(a, list, K, j0, j1, lds, acc);
      else
        mac_run<KIND, GPT, PARTS, NS, NT, 8>(a, list, K, j0, j1, lds, acc);
    }
  } else {
    mac_run<KIND, GPT, PARTS, NS, NT, 32>(a, list, K, j0, j1, lds, acc);
  }
}

// The W waves' sums of both strips, joined in wave order in the first wave's
// registers; true for that wave.
template <int W, int NT>
__device__ inline bool join(f32x4 (&acc)[2][NT], f32x4* red) {
  if constexpr (W > 1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();  // every wave is done with its staged x
    if (wave > 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[((wave * 2 + r) * NT + t) * 64 + lane] = acc[r][t];
    }
    __syncthreads();
    if (wave > 0) return false;
#pragma unroll
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] += red[((w * 2 + r) * NT + t) * 64 + lane];
  }
  return true;
}

// Two strips, rows r0 of matrix m0 and r1 of m1 (expert e), times the x rows
// given over the whole contraction, K long, which the work-group's W waves
// split. True for the wave that gets the sums.
template <WKind KIND, int GPT, int PARTS, int W, int NT>
__device__ inline bool strip_pair(const WMat& m0, const WMat& m1, int64_t e, int64_t r0, int64_t r1, int64_t N,
                                  int64_t K, const RowList& x, f32x4 (&acc)[2][NT], char* lds) {
  const int wave = W > 1 ? uniform(threadIdx.x >> 6) : 0;
  const int units = units_of<KIND>(K);
  const Strip<KIND> a[2] = {strip_of<KIND, GPT>(m0, e, r0, N, K), strip_of<KIND, GPT>(m1, e, r1, N, K)};
  if constexpr (W > 1) __syncthreads();  // the sums of the pass before have been read
  mac<KIND, GPT, PARTS>(a, x, K, units * wave / W, units * (wave + 1) / W,
                        lds + wave * kWaveLds<KIND, GPT, PARTS, 2, (NT > 1)>, acc);
  return join<W, NT>(acc, reinterpret_cast<f32x4*>(lds));
}

struct FewArgs {
  int T, E, k;
  int64_t d, f;
  const void* x;         // x as the experts read it: [T, d], or its bf16 parts [PARTS][T][d]
  const void* x_res;     // the residual, [T, d] in the layer's type
  WMat gate, up, down;
  FewLists ls;
  void* h;               // [PARTS][T k][ldh], by position in the lists
  int64_t ldh;
  float* sums;           // [strips][shares][T][16]
  void* out;
};

// h = silu(g) u of 16 features for an expert's tokens.
template <WKind KIND, int GPT, int PARTS, int W, int NT>
__device__ inline void gate_up_tile(const FewArgs& a, int64_t e, int p0, int n, int64_t f0, char* lds) {
  constexpr int kElem = sizeof(XType<KIND>);
  const int lane = threadIdx.x & 63;
  const RowList x = {span(a.x, a.T * a.d * kElem), a.d * kElem, a.T * a.d * kElem, n,
                     a.ls.token[p0 + std::min(lane, n - 1)]};
  f32x4 v[2][NT] = {};
  if (!strip_pair<KIND, GPT, PARTS, W, NT>(a.gate, a.up, e, f0, f0, a.f, a.d, x, v, lds)) return;
  const int64_t feat = f0 + 4 * (lane >> 4);  // of this lane's four; d_ff is a multiple of 4
  if (feat >= a.f) return;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + (lane & 15);
    if (c >= n) continue;
    f32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float g = v[0][t][i];
      h[i] = g / (1.f + expf(-g)) * v[1][t][i];
    }
    const int64_t at = (p0 + c) * a.ldh + feat;
    if constexpr (KIND == kDenseF32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.h) + at) = h;
    } else if constexpr (PARTS == 1) {
      // Rounded as moe_layer_forward rounds h between its two products, so that the down product takes one matrix
      // instruction a step: out's relative error (root mean square, against 64 bits) grows from 1.64 - 1.66e-3, the
      // rounding of out alone, to 1.67 - 1.79e-3. Two bf16 parts would take twice the products and staged h.
      uint2 b;
      b.x = f32_to_bf16(h[0]) | static_cast<uint32_t>(f32_to_bf16(h[1])) << 16;
      b.y = f32_to_bf16(h[2]) | static_cast<uint32_t>(f32_to_bf16(h[3])) << 16;
      *reinterpret_cast<uint2*>(static_cast<bf16_t*>(a.h) + at) = b;
    } else {
      const int64_t part = static_cast<int64_t>(a.T) * a.k * a.ldh;
      bf16_t q[4][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) split3(h[i], q[i]);
#pragma unroll
      for (int j = 0; j < 3; ++j)
        *reinterpret_cast<uint2*>(static_cast<bf16_t*>(a.h) + j * part + at) =
            uint2{q[0][j] | static_cast<uint32_t>(q[1][j]) << 16, q[2][j] | static_cast<uint32_t>(q[3][j]) << 16};
    }
  }
}

// CALL for an expert's copies p .. p + n - 1, 16 at a time or (WIDE) 32. More
// copies read the weights again, past the caches as the first time, and each
// pass costs nearly what the first does: the layer with one chosen expert,
// d = d_ff = 4096 (101 MB in bf16), with 1, 16, 32 and 64 copies takes 47, 49, 74
// and 124 us in bf16 and 31, 41, 59 and 96 us in u4. Loads that leave the
// weights in the caches took 114 and 88 us for 64 copies, but 50 us in bf16 for one.
#define MOE_BY_TOKENS(first, count, CALL)                                        \
  do {                                                                           \
    constexpr int kMost = WIDE ? 32 : 16;                                        \
    for (int p = (first), left = (count); left > 0; p += kMost, left -= kMost) { \
      const int n = std::min(left, kMost);                                       \
      if (WIDE && n > 16) {                                                      \
        constexpr int NT = WIDE ? 2 : 1;                                         \
        CALL;                                                                    \
      } else {                                                                   \
        constexpr int NT = 1;                                                    \
        CALL;                                                                    \
      }                                                                          \
    }                                                                            \
  } while (0)

// LDS words of a work-group of W waves that works on a pair of strips.
template <WKind KIND, int GPT, int PARTS, bool WIDE, int W>
constexpr int kPairLds = W * kWaveLds<KIND, GPT, PARTS, 2, WIDE> / 16;

template <WKind KIND, int GPT, int PARTS, bool WIDE, int W>
__global__ __launch_bounds__(W * 64, waves_per_simd(PARTS, WIDE)) void few_gate_up_kernel(FewArgs a) {
  __shared__ f32x4 lds[kPairLds<KIND, GPT, PARTS, WIDE, W>];
  const int64_t ft = ceil_div(a.f, 16);
  const int64_t i = blockIdx.x / ft;
  const int n_act = *a.ls.n_act;  // the four loads together: past n_act the lists hold anything
  const int e = uniform(a.ls.act_e[i]), p0 = uniform(a.ls.act_off[i]), p1 = uniform(a.ls.act_off[i + 1]);
  if (i >= n_act) return;
  MOE_BY_TOKENS(p0, p1 - p0, (gate_up_tile<KIND, GPT, PARTS, W, NT>(a, e, p, n, (blockIdx.x % ft) * 16,
                                                                    reinterpret_cast<char*>(lds))));
}

// out for 16 of its columns: x plus the gate-weighted sums of all experts'
// down products. A work-group reads the strip's rows of every expert with
// copies; the units of all of them, expert after expert, are dealt to the
// waves in equal runs. A wave adds each expert's part of its run, times the
// gates, to its own sums of the T tokens in LDS, and these are joined in wave
// order: no y goes to memory. With few strips several work-groups share one: each
// leaves its sums in memory and counts itself, and the last to come adds them up
// in their order. Nothing waits for another work-group.
template <WKind KIND, int GPT, int PARTS, int NT>
__device__ inline void down_run(const FewArgs& a, int64_t e, int p0, int n, int64_t c0, int j0, int j1, char* lds,
                                float* sums) {
  const int lane = threadIdx.x & 63;
  const int64_t row = a.ldh * sizeof(XType<KIND>);
  const RowList x = {span(static_cast<const char*>(a.h) + p0 * row, n * row), row, a.T * a.k * row, n,
                     std::min(lane, n - 1)};
  int token[NT];
  float gate[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {  // on their way while the products are taken
    const int c = p0 + std::min(t * 16 + (lane & 15), n - 1);
    token[t] = a.ls.token[c];
    gate[t] = a.ls.gate[c];
  }
  f32x4 acc[1][NT] = {};
  const Strip<KIND> s[1] = {strip_of<KIND, GPT>(a.down, e, c0, a.d, a.f)};
  mac<KIND, GPT, PARTS>(s, x, a.f, j0, j1, lds, acc);
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (t * 16 + (lane & 15) < n) {
      f32x4* o = reinterpret_cast<f32x4*>(sums + token[t] * 16) + (lane >> 4);
      *o += gate[t] * acc[0][t];
    }
}

// Sums between work-groups, which may run on dies whose L2s do not see each
// other's writes: stored and loaded past these, one by one. (A fence instead
// would write back and drop a whole L2; with one in each wave the kernel took
// 100 us, with one a work-group as long as with unshared strips, 16 - 19 us.)
__device__ inline void to_chip(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline float from_chip(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void wait_for_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// SHARED: gridDim.y > 1 work-groups a strip.
template <WKind KIND, int GPT, int PARTS, bool WIDE, int WAVES, bool SHARED>
__global__ __launch_bounds__(WAVES * 64, waves_per_simd(PARTS, WIDE)) void few_down_kernel(
    FewArgs a) {
  constexpr int kStage = kWaveLds<KIND, GPT, PARTS, 1, WIDE>;
  static_assert(WAVES * (kStage + kFewMaxT * 64) <= 160 * 1024, "a CU's LDS");
  __shared__ f32x4 staged[WAVES * kStage / 16];
  extern __shared__ f32x4 all_sums_[];  // [WAVES][T][16] floats
  float* all_sums = reinterpret_cast<float*>(all_sums_);
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int strip = blockIdx.x, share = SHARED ? blockIdx.y : 0, shares = SHARED ? gridDim.y : 1;
  float* sums = all_sums + wave * a.T * 16;
  char* lds = reinterpret_cast<char*>(staged) + wave * kStage;
  // the first 64 experts of the list, on their way together with its length
  const int first_e = a.ls.act_e[std::min(lane, a.E - 1)], first_p = a.ls.act_off[std::min(lane, a.E)];
  const int after_p = a.ls.act_off[std::min(lane + 1, a.E)];
  for (int i = lane; i < a.T * 16; i += 64) sums[i] = -0.f;  // stays so for a token without copies
  const int64_t c0 = strip * 16ll;
  const int units = units_of<KIND>(a.f), nth = share * WAVES + wave, of = shares * WAVES;
  const int64_t total = static_cast<int64_t>(units) * uniform(*a.ls.n_act);  // below 2^31: 2^18 units of 1024 experts
  const int end = static_cast<int>(total * (nth + 1) / of);
  for (int u = static_cast<int>(total * nth / of); u < end;) {
    const int i = u / units, j0 = u % units, j1 = std::min(units, j0 + end - u);
    int e, p0, p1;
    if (i < 64) {
      e = __builtin_amdgcn_readlane(first_e, i);
      p0 = __builtin_amdgcn_readlane(first_p, i);
      p1 = __builtin_amdgcn_readlane(after_p, i);
    } else {
      e = uniform(a.ls.act_e[i]);
      p0 = uniform(a.ls.act_off[i]);
      p1 = uniform(a.ls.act_off[i + 1]);
    }
    MOE_BY_TOKENS(p0, p1 - p0, (down_run<KIND, GPT, PARTS, NT>(a, e, p, n, c0, j0, j1, lds, sums)));
    u += j1 - j0;
  }
  __syncthreads();
  float* shared = a.sums + strip * static_cast<int64_t>(shares) * a.T * 16;
  if constexpr (SHARED) {
    for (int i = threadIdx.x; i < a.T * 16; i += WAVES * 64) {
      float v = all_sums[i];
      for (int w = 1; w < WAVES; ++w) v += all_sums[w * a.T * 16 + i];
      to_chip(shared + share * a.T * 16 + i, v);
    }
    __shared__ int before;
    wait_for_stores();  // this wave's sums are there before thread 0 counts the work-group
    __syncthreads();
    if (threadIdx.x == 0)
      before = __hip_atomic_fetch_add(a.ls.done + strip, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (before + 1 < shares) return;
  }
  constexpr bool kBf16 = KIND == kDenseBf16 || (!is_dense(KIND) && PARTS == 1);
  for (int i = threadIdx.x; i < a.T * 16; i += WAVES * 64) {
    const int64_t col = c0 + (i & 15), at = (i >> 4) * a.d + col;
    if (col >= a.d) continue;
    float v;
    if constexpr (!SHARED) {
      v = all_sums[i];
      for (int w = 1; w < WAVES; ++w) v += all_sums[w * a.T * 16 + i];
    } else {
      float part[kFewMaxShares];  // asked for together
#pragma unroll
      for (int w = 0; w < kFewMaxShares; ++w) part[w] = w < shares ? from_chip(shared + w * a.T * 16 + i) : -0.f;
      v = part[0];
#pragma unroll
      for (int w = 1; w < kFewMaxShares; ++w) v += part[w];
    }
    const bool as_it_is = __float_as_uint(v) == 0x80000000u;  // x + -0: x's bits, also of NaN
    if constexpr (kBf16) {
      const bf16_t x = static_cast<const bf16_t*>(a.x_res)[at];
      static_cast<bf16_t*>(a.out)[at] = as_it_is ? x : f32_to_bf16(bf16_to_f32(x) + v);
    } else {
      const float x = static_cast<const float*>(a.x_res)[at];
      static_cast<float*>(a.out)[at] = as_it_is ? x : x + v;
    }
  }
}

// ---------------------------------------------------------------------------
// out[r] = W[expert[r]] x[r] with 4-bit weights.
// ---------------------------------------------------------------------------
struct MatvecArgs {
  int R, E;
  int64_t N, K;
  const bf16_t* x;  // [PARTS][R][K]
  const int32_t* expert;
  WMat w;
  void* out;        // [R, N] bf16 (PARTS = 1) or fp32
};

// The rows of one expert: rows with the same expert are a group, in the order of
// their first rows; row c of this one in lane c < n. Rows with an expert outside
// [0, E) are in none.
struct RowGroup {
  int e, n, row;  // n = 0: there are not so many groups
};

// Group i, by one wave in registers: lanes with the same expert find each other
// by one ballot a bit of its number. (Every wave for itself: the weights' loads,
// which only need the expert, then wait for no barrier.)
__device__ inline RowGroup row_group(const int32_t* expert, int R, int E, int i) {
  const int lane = threadIdx.x & 63;
  int e = -1;
  if (lane < R) e = expert ? expert[lane] : 0;
  const bool valid = e >= 0 && e < E;
  unsigned long long mates = __ballot(valid);
  for (int bit = 0; (E - 1) >> bit; ++bit) {
    const unsigned long long set = __ballot((e >> bit) & 1);
    mates &= (e >> bit) & 1 ? set : ~set;
  }
  const unsigned long long below = (1ull << lane) - 1ull;
  const bool leads = valid && !(mates & below);
  const unsigned long long leaders = __ballot(leads);
  if (i >= __popcll(leaders)) return {0, 0, 0};
  const int first = __ffsll(__ballot(leads && __popcll(leaders & below) == i)) - 1;
  const int its = __builtin_amdgcn_readlane(e, first);
  const unsigned long long mine = __ballot(e == its);
  const int n = __popcll(mine);
  // lane to lane: the group's rows first, then the others
  const int to = e == its ? __popcll(mine & below) : n + __popcll(~mine & below);
  return {its, n, __builtin_amdgcn_ds_permute(4 * to, lane)};
}

template <WKind KIND, int GPT, int PARTS, int W, int NT>
__device__ inline void matvec_tile(const MatvecArgs& a, const RowGroup& g, int p, int n, int64_t n0, char* lds) {
  const int lane = threadIdx.x & 63;
  const RowList x = {span(a.x, a.R * a.K * 2), a.K * 2, a.R * a.K * 2, n, __shfl(g.row, p + std::min(lane, n - 1))};
  // the last 16 rows of a matrix may have no 16 after them: they are read twice
  const int64_t n1 = n0 + 16 < a.N ? n0 + 16 : n0;
  f32x4 v[2][NT] = {};
  if (!strip_pair<KIND, GPT, PARTS, W, NT>(a.w, a.w, g.e, n0, n1, a.N, a.K, x, v, lds)) return;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + (lane & 15);
    const int64_t row = __shfl(g.row, (p + c) & 63) * a.N;
    if (c >= n) continue;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t col = n0 + 16 * r + 4 * (lane >> 4) + i;
        if (col >= a.N) continue;
        if constexpr (PARTS == 1)
          static_cast<bf16_t*>(a.out)[row + col] = f32_to_bf16(v[r][t][i]);
        else
          static_cast<float*>(a.out)[row + col] = v[r][t][i];
      }
  }
}

template <WKind KIND, int GPT, int PARTS, bool WIDE, int W>
__global__ __launch_bounds__(W * 64, waves_per_simd(PARTS, WIDE)) void matvec_kernel(MatvecArgs a) {
  __shared__ f32x4 lds[kPairLds<KIND, GPT, PARTS, WIDE, W>];
  const int64_t nt = ceil_div(a.N, 32);
  const RowGroup g = row_group(a.expert, a.R, a.E, static_cast<int>(blockIdx.x / nt));
  MOE_BY_TOKENS(0, g.n, (matvec_tile<KIND, GPT, PARTS, W, NT>(a, g, p, n, (blockIdx.x % nt) * 32,
                                                              reinterpret_cast<char*>(lds))));
}

__global__ __launch_bounds__(256) void split_kernel(const float* x, int64_t n, bf16_t* parts) {
  split_rows(x, n, parts, blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll);
}

// g(kind, groups per tile, parts, wide) with compile-time arguments.
template <typename F>
hipError_t by_weights(const FewWeights& w, bool bf16, bool wide, F&& g) {
  using std::integral_constant;
  auto f = [&](auto kind, auto gpt, auto parts) {
    // fp32 x in three parts fills the LDS with one token tile
    if constexpr (decltype(parts)::value == 1) {
      if (wide) return g(kind, gpt, parts, std::true_type{});
    }
    return g(kind, gpt, parts, std::false_type{});
  };
  if (w.kind < 0) {
    if (bf16) return f(integral_constant<WKind, kDenseBf16>{}, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    return f(integral_constant<WKind, kDenseF32>{}, integral_constant<int, 1>{}, integral_constant<int, 1>{});
  }
  auto parts = [&](auto kind, auto gpt) {
    if (bf16) return f(kind, gpt, integral_constant<int, 1>{});
    return f(kind, gpt, integral_constant<int, 3>{});
  };
  auto group = [&](auto kind) {
    if (w.group == 32) return parts(kind, integral_constant<int, 4>{});
    if (w.group == 64) return parts(kind, integral_constant<int, 2>{});
    return parts(kind, integral_constant<int, 1>{});
  };
  if (w.kind == kQ4U4) return group(integral_constant<WKind, kU4>{});
  return group(integral_constant<WKind, kE2m1>{});
}

// Experts that T tokens with k of E each hit, if each choice were as likely.
double expected_distinct(int E, int k, int T) { return E * (1 - std::pow(1 - static_cast<double>(k) / E, T)); }

// f(waves of a work-group) for about `items` pairs of strips over K columns. The
// chip holds 4096 waves: with few items and long rows more waves share one, so
// that the memory has enough to do; short rows leave eight waves a few units each
// and the joining to pay. Eight and four waves, one row of 128, 256 and 448 items:
// u4 row product, K = 14336: 14.6, 15.8, 23.2 and 17.6, 21.0, 24.7 us; K = 8192:
// 10.3, 11.8, 16.0 and 11.0, 12.3, 15.9; K = 5632 (44 units): 9.0, 10.2, 13.9 and
// 9.2, 10.9, 13.0; K = 4096 (32): 8.3, 10.6, 12.6 and 7.8, 8.8, 11.0; K = 2048: 6.4,
// 7.2, 9.4 and 6.0, 6.4, 8.1. The layer with one chosen expert, bf16, d = 8192 (128
// units): 46, 57, 85 and 47, 64, 95 us; d = 4096 (64): 36, 40, 53 and 36, 39, 51;
// d = 2048: 27, 35, 41 and 26, 32, 38; fp32, d = 4096 (128): 46, 58, 85 and 47, 59,
// 83. Two waves instead of four put 1024 - 2048 items on the chip at once (e2m1,
// 64 rows: 16.2 us, 19.0 with four). With very many, one wave alone spares the
// joining (64 tokens of a DeepSeek-V3-shaped layer: bf16 3.03 ms, 3.24 with four);
// below, its long items would leave the last round's waves alone with the memory
// (1.2 rounds of single waves: 254 us instead of 219 with four).
template <WKind KIND, int PARTS, typename F>
void by_waves(double items, int64_t K, F&& f) {
  if (PARTS == 1 && items <= 512 && units_of<KIND>(K) >= (is_dense(KIND) ? 80 : 40))
    f(std::integral_constant<int, 8>{});
  else if (items > 1024 && items <= 2048)
    f(std::integral_constant<int, 2>{});
  else if (items <= 16384)
    f(std::integral_constant<int, 4>{});
  else
    f(std::integral_constant<int, 1>{});
}

}  // namespace

// Slices of d for the router scores: enough work-groups to spread W_router
// over the chip, slices of 512 columns at least, and few enough partial scores
// to add up.
int few_router_splits(int64_t T, int64_t d, int E) {
  const int64_t tiles = std::max<int64_t>(1, ceil_div(E, 16) * ceil_div(T, 16));
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kFewMaxSplits, d / 512, 256 / tiles})));
}

// Enough work-groups for the chip (a CU holds two), but 16 units in each. The
// layer without sharing and with it: fp32, 7 tokens, d = 500 (32 strips) 37.2 and
// 28.6 us; u4, 3 tokens, d = 2048 (128 strips) 43.0 and 40.1 us; e2m1, 16 tokens,
// d = 4096 (256 strips) 180 and 167 us.
int few_down_splits(int64_t T, int64_t d, int64_t f, int E, int k, int unit_cols) {
  const int64_t units = std::min<int64_t>(E, T * k) * ceil_div(f, unit_cols);
  return static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>({kFewMaxShares, 512 / ceil_div(d, 16), units / 16})));
}

hipError_t launch_few_layer(const FewLayer& L, hipStream_t s) {
  const bool bf16 = L.bf16;
  const int S = few_router_splits(L.T, L.d, L.E);
  const dim3 rgrid(static_cast<unsigned>(ceil_div(L.E, 16)), static_cast<unsigned>(ceil_div(L.T, 16)), S);
  if (bf16)
    few_router_kernel<true><<<rgrid, dim3(kRouterThreads), 0, s>>>(L.x, L.wr, L.T, L.E, L.d, S, L.part, nullptr);
  else
    few_router_kernel<false><<<rgrid, dim3(kRouterThreads), 0, s>>>(L.x, L.wr, L.T, L.E, L.d, S, L.part, L.xparts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const RouteOut ro{L.idx, L.w, L.slot, L.routed, L.kept, L.send, L.totals};
  const int64_t row = L.d * (bf16 ? 2 : 4);
  const Scores sc{L.part, S, L.bias, L.T, L.E, L.k, L.P, L.M};
  const bool small = L.T * L.k <= 64 && L.P <= 64;
  auto route = [&](auto ne) {
    constexpr int NE = decltype(ne)::value;
    if (small)
      few_route_small_kernel<NE><<<dim3(1), dim3(64 * std::min(L.T, 16)), 0, s>>>(sc, L.C, row, ro, L.ls);
    else
      few_route_kernel<NE><<<dim3(1), dim3(1024), 0, s>>>(sc, L.C, row, ro, L.ls);
  };
  if (L.E <= 64)
    route(std::integral_constant<int, 1>{});
  else if (L.E <= 256)
    route(std::integral_constant<int, 4>{});
  else
    route(std::integral_constant<int, 16>{});
  if ((e = hipGetLastError()) != hipSuccess) return e;
  FewArgs a;
  a.T = L.T;
  a.E = L.E;
  a.k = L.k;
  a.d = L.d;
  a.f = L.f;
  a.x = L.xparts ? static_cast<const void*>(L.xparts) : L.x;
  a.x_res = L.x;
  a.gate = {L.E, L.wt.w[0], static_cast<const bf16_t*>(L.wt.scale[0]), static_cast<const uint8_t*>(L.wt.zero[0])};
  a.up = {L.E, L.wt.w[1], static_cast<const bf16_t*>(L.wt.scale[1]), static_cast<const uint8_t*>(L.wt.zero[1])};
  a.down = {L.E, L.wt.w[2], static_cast<const bf16_t*>(L.wt.scale[2]), static_cast<const uint8_t*>(L.wt.zero[2])};
  a.ls = L.ls;
  a.h = L.h;
  a.ldh = few_ld_h(L.f);
  a.sums = L.sums;
  a.out = L.out;
  const int64_t act = std::min<int64_t>(L.E, static_cast<int64_t>(L.T) * L.k);  // experts with copies, at most
  const int64_t strips = ceil_div(L.d, 16);
  // two token tiles at a time where experts have more than half of one on average: 64 tokens, k = 2 of 8, d = 4096,
  // d_ff = 14336: bf16 629 us, 788 with one; e2m1 291 and 307. With fewer copies the registers are better spent on waves.
  const bool wide = static_cast<int64_t>(L.T) * L.k > 8 * static_cast<int64_t>(L.E);
  return by_weights(L.wt, bf16, wide, [&](auto kind, auto gpt, auto parts, auto two) {
    constexpr WKind kKind = decltype(kind)::value;
    constexpr int kGpt = decltype(gpt)::value, kParts = decltype(parts)::value;
    constexpr bool kWide = decltype(two)::value;
    const int64_t ft = ceil_div(L.f, 16);
    by_waves<kKind, kParts>(expected_distinct(L.E, L.k, L.T) * ft, L.d, [&](auto waves) {
      constexpr int W = decltype(waves)::value;
      few_gate_up_kernel<kKind, kGpt, kParts, kWide, W>
          <<<dim3(static_cast<unsigned>(act * ft)), dim3(W * 64), 0, s>>>(a);
    });
    auto down = [&](auto shared) {
      constexpr int W = 2 * waves_per_simd(kParts, kWide);  // two work-groups a CU
      few_down_kernel<kKind, kGpt, kParts, kWide, W, decltype(shared)::value>
          <<<dim3(static_cast<unsigned>(strips), L.splits), dim3(W * 64), W * L.T * 64, s>>>(a);
    };
    if (L.splits > 1)
      down(std::true_type{});
    else
      down(std::false_type{});
    return hipGetLastError();
  });
}

hipError_t launch_q4_matvec(const void* x, bool bf16, const int32_t* expert, const FewWeights& w, int R, int E,
                            int64_t N, int64_t K, bf16_t* parts, void* out, hipStream_t s) {
  if (!bf16) {
    split_kernel<<<dim3(static_cast<unsigned>(std::min<int64_t>(1024, ceil_div(R * K, 256)))), dim3(256), 0, s>>>(
        static_cast<const float*>(x), R * K, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  MatvecArgs a;
  a.R = R;
  a.E = E;
  a.N = N;
  a.K = K;
  a.x = bf16 ? static_cast<const bf16_t*>(x) : parts;
  a.expert = expert;
  a.w = {E, w.w[0], static_cast<const bf16_t*>(w.scale[0]), static_cast<const uint8_t*>(w.zero[0])};
  a.out = out;
  const int64_t groups = expert ? std::min(E, R) : 1;
  return by_weights(w, bf16, R > 8 * groups, [&](auto kind, auto gpt, auto parts_, auto two) {
    constexpr WKind kKind = decltype(kind)::value;
    if constexpr (kKind == kU4 || kKind == kE2m1) {
      constexpr int kGpt = decltype(gpt)::value, kParts = decltype(parts_)::value;
      constexpr bool kWide = decltype(two)::value;
      const int64_t nt = ceil_div(N, 32);
      by_waves<kKind, kParts>((expert ? expected_distinct(E, 1, R) : 1) * nt, K, [&](auto waves) {
        constexpr int W = decltype(waves)::value;
        matvec_kernel<kKind, kGpt, kParts, kWide, W>
            <<<dim3(static_cast<unsigned>(groups * nt)), dim3(W * 64), 0, s>>>(a);
      });
      return hipGetLastError();
    } else {
      return hipErrorInvalidValue;
    }
  });
}

}  // namespace moe
