// The whole layer for a few tokens (T <= 64, one token tile), with bf16, fp32
// or 4-bit expert weights, and products of single rows with 4-bit weights.
//
// With few tokens nothing is computed often enough to matter: the layer is the
// read of the chosen experts' matrices, 3 d d_ff elements each, once. So the
// weights go from memory straight into the matrix instructions' operand
// registers: the weight tile is the A operand (16 output features by 32
// columns), up to 16 of the expert's tokens are the 16 columns of B, and no
// tile passes through LDS. A work-group of 4 waves takes two such 16-row tiles
// (gate and up rows of the same features, or 32 neighbouring rows of W_down)
// over the whole contraction; its waves split the contraction and join their
// sums through LDS, in wave order.
//
// Nothing here depends on the order in which work-groups run: every sum has a
// fixed order, and the expert lists are built by ranks, not by arrival.
#include "common.h"
#include "q4.h"

#include <algorithm>
#include <climits>

namespace moe {
namespace {

constexpr int kWaves = 4;            // waves of an expert work-group
constexpr int kThreads = kWaves * 64;

enum WKind { kDenseBf16, kDenseF32, kU4, kE2m1 };

// ---------------------------------------------------------------------------
// Router scores. Block (expert tile, token tile, K slice); its waves split the
// slice. Every MFMA starts from zero and its fp32 sums of 32 (fp32 inputs: 16)
// products are added up in fp64, so that the scores' order is decided well
// below fp32's rounding: sums of different order pick the same experts.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(kThreads) void few_router_kernel(const void* xv, const void* wv, int T, int E, int64_t d,
                                                              int S, double* __restrict__ part,
                                                              bf16_t* __restrict__ parts, int32_t* __restrict__ clear,
                                                              int n_clear) {
  __shared__ double red[kWaves][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, quad = lane >> 4;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16, s = blockIdx.z;
  const int64_t block = (static_cast<int64_t>(s) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t nthreads = static_cast<int64_t>(gridDim.x) * gridDim.y * gridDim.z * kThreads;
  for (int64_t i = block * kThreads + threadIdx.x; i < n_clear; i += nthreads) clear[i] = 0;
  if (!BF16 && parts) split_rows(static_cast<const float*>(xv), T * d, parts, block * kThreads + threadIdx.x, nthreads);
  constexpr int kStep = BF16 ? 32 : 16, kVec = BF16 ? 8 : 4;
  const int64_t steps = ceil_div(d, kStep);
  const int64_t j0 = steps * (s * kWaves + wave) / (S * kWaves), j1 = steps * (s * kWaves + wave + 1) / (S * kWaves);
  const int64_t er = std::min(e0 + col, E - 1), tr = std::min(t0 + col, T - 1);
  double acc[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int64_t j = j0; j < j1; ++j) {
    const int64_t c = j * kStep + kVec * quad;
    f32x4 p = {0, 0, 0, 0};
    uint4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    if (c < d) {  // d is a multiple of kVec
      a = *reinterpret_cast<const uint4*>(static_cast<const char*>(wv) + (er * d + c) * (16 / kVec));
      b = *reinterpret_cast<const uint4*>(static_cast<const char*>(xv) + (tr * d + c) * (16 / kVec));
    }
    if constexpr (BF16) {
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), p, 0,
                                                  0, 0);
    } else {
      const f32x4 av = __builtin_bit_cast(f32x4, a), bv = __builtin_bit_cast(f32x4, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x4f32(av[i], bv[i], p, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += static_cast<double>(p[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][lane][i] = acc[i];
  __syncthreads();
  // thread: element i of lane l, i.e. expert row 4 (l / 16) + i and token l % 16
  const int l = threadIdx.x >> 2, i = threadIdx.x & 3;
  double v = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) v += red[w][l][i];
  const int e = e0 + 4 * (l >> 4) + i, t = t0 + (l & 15);
  if (e < E && t < T) part[(static_cast<int64_t>(s) * T + t) * E + e] = v;
}

// ---------------------------------------------------------------------------
// Top-k, gates, slots and the experts' token lists: one work-group.
// ---------------------------------------------------------------------------

// Monotone map of a double to uint64; NaN sorts below every number (its
// choice is unspecified, but stays a distinct expert), and 0 is below NaN.
__device__ inline uint64_t order_key(double v) {
  if (v != v) return 1;
  v += 0.0;  // -0.0 -> +0.0
  const uint64_t u = __double_as_longlong(v);
  return (u >> 63) ? ~u : (u | (uint64_t{1} << 63));
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

template <int NE>  // scores a lane holds: E <= 64 NE
__global__ __launch_bounds__(1024) void few_route_kernel(const double* __restrict__ part, int S,
                                                         const float* __restrict__ bias, int T, int E, int k, int P,
                                                         int M, int64_t C, int64_t row_bytes, RouteOut o, FewLists ls) {
  __shared__ int cnt[kFewMaxE], ecp[kFewMaxCopies], rank[kFewMaxCopies], scratch[kRankChunkInts];
  __shared__ unsigned long long rbest[16][64];
  __shared__ int wsum[17], send_s[64], dropped_tokens;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = E / P;
  const bool limit = M > 0 && M < P;
  for (int e = tid; e < E; e += 1024) cnt[e] = 0;
  if (tid == 0) dropped_tokens = 0;

  for (int t = wave; t < T; t += 16) {
    double v[NE];
    uint64_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      v[i] = 0;
      key[i] = 0;
      if (e < E) {
        for (int s = 0; s < S; ++s) v[i] += part[(static_cast<int64_t>(s) * T + t) * E + e];
        if (bias) v[i] += static_cast<double>(bias[e]);
        key[i] = order_key(v[i]);
      }
    }
    if (limit) {  // P <= 64: lane p holds rank p's best score
      rbest[wave][lane] = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lane + 64 * i < E) atomicMax(&rbest[wave][(lane + 64 * i) / per], static_cast<unsigned long long>(key[i]));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      const uint64_t mine = rbest[wave][lane];
      int ahead = 0;  // ranks ahead of mine: better score, or equal score and lower index
      for (int p = 0; p < P; ++p) {
        const uint64_t q = rbest[wave][p];
        ahead += (q > mine || (q == mine && p < lane)) ? 1 : 0;
      }
      const uint64_t allowed = __ballot(lane < P && ahead < M);
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lane + 64 * i < E && !((allowed >> ((lane + 64 * i) / per)) & 1)) key[i] = 0;
    }
    double sel = 0, top = 0;
    int sel_e = 0;
    for (int r = 0; r < k; ++r) {
      uint64_t bk = key[0];
      int be = lane;
      double bv = v[0];
#pragma unroll
      for (int i = 1; i < NE; ++i)
        if (key[i] > bk) {
          bk = key[i];
          be = lane + 64 * i;
          bv = v[i];
        }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const uint64_t ok = __shfl_xor(static_cast<unsigned long long>(bk), off);
        const int oe = __shfl_xor(be, off);
        const double ov = __shfl_xor(bv, off);
        if (ok > bk || (ok == bk && oe < be)) {
          bk = ok;
          be = oe;
          bv = ov;
        }
      }
      if (r == 0) top = bv;
      if (lane == r) {
        sel = bv;
        sel_e = be;
      }
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (be == lane + 64 * i) key[i] = 0;
    }
    const double z = lane < k ? exp(sel - top) : 0.0;
    double sum = z;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane < k) {
      o.idx[t * k + lane] = sel_e;
      o.w[t * k + lane] = static_cast<float>(z / sum);
      ecp[t * k + lane] = sel_e;
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

// ---------------------------------------------------------------------------
// Products of NS strips of 16 weight rows with NT tiles of 16 rows of x over a
// range of the contraction: acc[r][t] += W_r x_t^T, one 16 x 16 tile in the
// matrix instructions' layout (lane: token lane % 16, features 4 (lane / 16) + i).
// The range is in units of a strip's memory: 128-byte lines of dense rows,
// 128-column tiles of 4-bit ones.
// ---------------------------------------------------------------------------

constexpr bool is_dense(WKind k) { return k == kDenseBf16 || k == kDenseF32; }

// Waves a SIMD that the registers are cut for; LDS allows no more where x takes
// three parts or, beside 4-bit weights, two token tiles.
constexpr int waves_per_simd(WKind k, int parts, bool wide) { return parts == 3 ? 2 : wide && !is_dense(k) ? 3 : 4; }

template <WKind KIND>
using XType = std::conditional_t<KIND == kDenseF32, float, bf16_t>;

// Units of a contraction of K columns.
template <WKind KIND>
__device__ inline int64_t units_of(int64_t K) {
  return KIND == kDenseBf16 ? ceil_div(K, 64) : KIND == kDenseF32 ? ceil_div(K, 32) : ceil_div(K, 128);
}

// One matrix stack [E, N, K] as the kernels take it.
struct WMat {
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

// One strip: where it begins (the same for all lanes, so that loads take a
// scalar base), and each lane's offsets from there. Dense: of its pieces of the
// strip's rows 0 - 7 and 8 - 15.
template <WKind KIND>
struct Strip {
  const char* base;      // first line, or first tile
  const bf16_t* scale;   // first group's rows
  const uint8_t* zero;   // u4: first group's zero points, and the bytes to the next group's
  int zstep;
  uint32_t lo, hi;
};

// n rows of x (at most 64): a common base, and in lane c row c's offset.
struct Rows {
  const char* base;
  uint32_t off;
  int n;
  int64_t part;  // bytes from one bf16 part of fp32 rows to the next
};

// Dense strips are read in whole 128-byte lines, eight rows an instruction:
// lane l takes piece (l / 16) + 4 (l / 8 % 2) of row l % 8. Loads that take
// half lines of all 16 rows, as the operand layout has them, must leave the
// line in the cache for the other half and reach 5.9 TB/s; whole lines can
// stream past it (non-temporal) at 6.6 - 6.9 TB/s. Two such loads hold the
// operands of two steps, up to a rotation by eight lanes (operands()).
__device__ inline int piece_of(int lane) { return (lane >> 4) + 4 * ((lane >> 3) & 1); }

// Rows r0 .. r0 + 15 of matrix e (both the same for all lanes).
template <WKind KIND, int GPT>
__device__ inline Strip<KIND> strip_of(const WMat& m, int64_t e, int64_t r0, int64_t N, int64_t K) {
  const int lane = threadIdx.x & 63;
  Strip<KIND> s = {};
  if constexpr (is_dense(KIND)) {
    const uint32_t row = static_cast<uint32_t>(K * sizeof(XType<KIND>));
    s.base = static_cast<const char*>(m.w) + (e * N + r0) * row;
    // rows past the matrix repeat its last one; their results are not stored
    const int last = static_cast<int>(std::min<int64_t>(15, N - 1 - r0));
    s.lo = std::min(lane & 7, last) * row + piece_of(lane) * 16;
    s.hi = std::min(8 + (lane & 7), last) * row + piece_of(lane) * 16;
  } else {
    const int64_t nt = ceil_div(N, 16), kt = ceil_div(K, 128);
    const int64_t t = (e * nt + r0 / 16) * kt;
    s.base = static_cast<const char*>(m.w) + t * 1024;
    s.lo = lane * 16;
    s.scale = m.scale + t * GPT * 16;
    s.zero = m.zero ? m.zero + t * GPT * 16 : kEights;
    s.zstep = m.zero ? 16 : 0;
  }
  return s;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ inline u32x4 load_once(const char* p, uint32_t off) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + off));
}

__device__ inline u32x4 load_kept(const char* p, uint32_t off) { return *reinterpret_cast<const u32x4*>(p + off); }

// The A operands of a line's two steps from the loads of rows 0 - 7 and 8 - 15:
// step 0 wants piece l / 16 of row l % 16, so lanes 8 - 15 of every 16 take
// the other load's lanes 0 - 7; step 1 the other way round.
__device__ inline void operands(u32x4 lo, u32x4 hi, u32x4& a0, u32x4& a1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr int kRotate8 = 0x128;
    a0[i] = __builtin_amdgcn_update_dpp(lo[i], hi[i], kRotate8, 0xf, 0xc, false);
    a1[i] = __builtin_amdgcn_update_dpp(hi[i], lo[i], kRotate8, 0xf, 0x3, false);
  }
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

// One unit's weights, as loaded. In the last unit of a row that ends inside it
// (dense) the lanes past the end repeat the row's last piece: x is 0 there.
template <WKind KIND, int NS>
struct UnitW {
  u32x4 w[NS][is_dense(KIND) ? 2 : 1];
};

template <WKind KIND, int NS>
__device__ inline void load_weights(const Strip<KIND> (&a)[NS], int64_t K, int64_t j, UnitW<KIND, NS>& u) {
#pragma unroll
  for (int r = 0; r < NS; ++r)
    if constexpr (is_dense(KIND)) {
      const int piece = piece_of(threadIdx.x & 63) * 16;
      const int64_t left = K * static_cast<int64_t>(sizeof(XType<KIND>)) - j * 128;
      const uint32_t over = left < 128 ? std::max(0, piece + 16 - static_cast<int>(left)) : 0;
      u.w[r][0] = load_once(a[r].base + j * 128, a[r].lo - over);
      u.w[r][1] = load_once(a[r].base + j * 128, a[r].hi - over);
    } else {
      u.w[r][0] = load_once(a[r].base + j * 1024, a[r].lo);
    }
}

// x and the scales of a run of units, staged in the wave's own LDS: one wave's
// loads of x from the caches would otherwise pace it (x takes four times the
// registers that the 4-bit codes it meets do, so it cannot be asked for as far
// ahead, and a load takes about 1 us when all of them wait for memory). The
// next run's loads wait in registers while this one is multiplied.
// LDS of a wave: x [PARTS][n rows][run bytes + 16] (the 16 bytes shift each row's
// banks), then scale [NS][units][GPT][16] bf16 and zero [NS][units][GPT][16] bytes.
template <WKind KIND, int GPT, int PARTS, int NS, int NT>
struct Stage {
  static constexpr bool kDense = is_dense(KIND);
  static constexpr int kUnitBytes = kDense ? 128 : 256;  // of a row of x (a part)
  static constexpr int kLoads = kDense ? 2 * NT + (NT == 1 ? 2 : 0) : 4 * NT;  // 1 KiB each, a part
  static constexpr int kMaxUnits = kDense ? 32 : GPT == 4 ? 8 : 16;
  static constexpr int kXBytes = PARTS * (kLoads * 1024 + 16 * NT * 16);
  static constexpr int kGroupsBytes = kDense ? 0 : NS * kMaxUnits * GPT * 48;
  static constexpr int kBytes = kXBytes + kGroupsBytes;

  char* lds;
  int shift, units, stride;     // log2 of a row's 16-byte pieces, units of a run, bytes of a row
  u32x4 x[PARTS][kLoads];
  u32x4 scale[kDense ? 1 : NS], zero[kDense ? 1 : NS];
  uint32_t at[NT];              // this lane's rows (and piece) in the staged x

  __device__ inline void init(char* wave_lds, const Rows& r) {
    const int lane = threadIdx.x & 63;
    lds = wave_lds;
    // as many units, a power of two, as the rows leave room for
    const int log_n = r.n > 1 ? 32 - __clz(r.n - 1) : 0;
    constexpr int kLogRoom = 31 - __builtin_clz(kLoads * 1024 / kUnitBytes), kLogMost = 31 - __builtin_clz(kMaxUnits);
    const int log_units = uniform(std::min(kLogMost, kLogRoom - log_n));
    units = 1 << log_units;
    shift = log_units + (kDense ? 3 : 4);
    stride = (16 << shift) + 16;
#pragma unroll
    for (int t = 0; t < NT; ++t)  // columns past n repeat the last row; their results are not stored
      at[t] = std::min(t * 16 + (lane & 15), r.n - 1) * stride + (lane >> 4) * 16;
  }

  // Asks for units j .. j + units - 1 (up to j1).
  __device__ inline void ask(const Strip<KIND> (&a)[NS], const Rows& r, int64_t K, int64_t j, int64_t j1) {
    const int lane = lane_here();
    const int n_units = static_cast<int>(std::min<int64_t>(units, j1 - j));
    const int64_t left = K * static_cast<int64_t>(sizeof(XType<KIND>)) - j * kUnitBytes;
    const int bytes = static_cast<int>(std::min<int64_t>(left, n_units * kUnitBytes));
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * 64 + lane, row = i >> shift, c = (i & ((1 << shift) - 1)) * 16;
      const uint32_t off = __shfl(r.off, row & 63) + c;
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        x[p][u] = u32x4{0, 0, 0, 0};  // also past the end of the contraction
        if (row < r.n && c < bytes) x[p][u] = load_kept(r.base + p * r.part + j * kUnitBytes, off);
      }
    }
    if constexpr (!kDense) {
      // groups that begin past the end are padding: 0, whatever the arrays hold
      const int64_t groups = std::min<int64_t>(n_units * GPT, ceil_div(K, 128 / GPT) - j * GPT);
#pragma unroll
      for (int r2 = 0; r2 < NS; ++r2) {
        scale[r2] = zero[r2] = u32x4{0, 0, 0, 0};
        if (lane < 2 * groups)
          scale[r2] = load_kept(reinterpret_cast<const char*>(a[r2].scale + j * GPT * 16), lane * 16);
        if (KIND == kU4 && lane < groups)
          zero[r2] = load_kept(reinterpret_cast<const char*>(a[r2].zero) + j * GPT * a[r2].zstep, lane * a[r2].zstep);
      }
    }
  }

  // Puts what was asked for into LDS; the wave's reads of the run before are
  // done (a wave's LDS accesses keep their order).
  __device__ inline void put(int n) {
    const int lane = lane_here();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = u * 64 + lane, row = i >> shift, c = (i & ((1 << shift) - 1)) * 16;
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        if (row < n) *reinterpret_cast<u32x4*>(lds + (p * n + row) * stride + c) = x[p][u];
    }
    if constexpr (!kDense) {
      constexpr int kScale = kMaxUnits * GPT * 32, kZero = kMaxUnits * GPT * 16;
      char* s = lds + kXBytes;
#pragma unroll
      for (int r2 = 0; r2 < NS; ++r2) {
        if (lane < units * GPT * 2) *reinterpret_cast<u32x4*>(s + r2 * kScale + lane * 16) = scale[r2];
        if (KIND == kU4 && lane < units * GPT)
          *reinterpret_cast<u32x4*>(s + NS * kScale + r2 * kZero + lane * 16) = zero[r2];
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  }

  // 64 bytes' worth (step q) of unit i of the run, token tile t, part p.
  __device__ inline u32x4 get(int i, int t, int p, int q, int n) const {
    return *reinterpret_cast<const u32x4*>(lds + p * n * stride + at[t] + i * kUnitBytes + q * 64);
  }
  __device__ inline uint2 get_scale(int i, int r, int g) const {
    return reinterpret_cast<const uint2*>(lds + kXBytes + ((r * kMaxUnits + i) * GPT + g) * 32)[(threadIdx.x & 63) >> 4];
  }
  __device__ inline uint32_t get_zero(int i, int r, int g) const {
    return reinterpret_cast<const uint32_t*>(lds + kXBytes + NS * kMaxUnits * GPT * 32 +
                                             ((r * kMaxUnits + i) * GPT + g) * 16)[(threadIdx.x & 63) >> 4];
  }
};

// acc += unit i of the staged run times its weights.
template <WKind KIND, int GPT, int PARTS, int NS, int NT>
__device__ inline void multiply(const UnitW<KIND, NS>& u, const Stage<KIND, GPT, PARTS, NS, NT>& in, int i, int n,
                                f32x4 (&acc)[NS][NT]) {
  if constexpr (is_dense(KIND)) {
    u32x4 x[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q) x[t][q] = in.get(i, t, 0, q, n);
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
            const bf16x8 xv = __builtin_bit_cast(bf16x8, in.get(i, t, p, st, n));
#pragma unroll
            for (int r = 0; r < NS; ++r)
              sum[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[r], xv, sum[r][t], 0, 0, 0);
            if constexpr (kU) sx[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xv, sx[t], 0, 0, 0);
          }
      }
#pragma unroll
      for (int r = 0; r < NS; ++r) {
        const uint2 sv = in.get_scale(i, r, g);
        const float s[4] = {__uint_as_float(sv.x << 16), __uint_as_float(sv.x & 0xffff0000u),
                            __uint_as_float(sv.y << 16), __uint_as_float(sv.y & 0xffff0000u)};
        float off[4];
        if constexpr (kU) {
          const uint32_t z = in.get_zero(i, r, g);
#pragma unroll
          for (int c = 0; c < 4; ++c) off[c] = 16.f + static_cast<float>((z >> (8 * c)) & 0xffu);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float v = kU ? fmaf(-off[c], sx[t][c], sum[r][t][c]) : sum[r][t][c];
            acc[r][t][c] = fmaf(s[c], v, acc[r][t][c]);
          }
      }
    }
  }
}

// Units j0 .. j1 - 1 of the strips. 8 KiB of weights a wave are in flight all
// the time: each place of the ring is asked for again as soon as its unit is
// multiplied (past the range the last unit, from the cache).
template <WKind KIND, int GPT, int PARTS, int NS, int NT>
__device__ inline void mac(const Strip<KIND> (&a)[NS], const Rows& x, int64_t K, int64_t j0, int64_t j1, char* lds,
                           f32x4 (&acc)[NS][NT]) {
  if (j0 >= j1) return;
  constexpr int U = (is_dense(KIND) ? 4 : 8) / NS;
  UnitW<KIND, NS> w[U];
  Stage<KIND, GPT, PARTS, NS, NT> in;
  in.init(lds, x);
  in.ask(a, x, K, j0, j1);
#pragma unroll
  for (int u = 0; u < U; ++u) load_weights(a, K, std::min(j0 + u, j1 - 1), w[u]);
  int i = in.units;  // unit of the staged run
  for (int64_t j = j0; j < j1; j += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u < j1) {
        if (i == in.units) {
          in.put(x.n);
          in.ask(a, x, K, std::min(j + u + in.units, j1), j1);
          i = 0;
        }
        __builtin_amdgcn_sched_barrier(0);
        multiply<KIND, GPT, PARTS>(w[u], in, i, x.n, acc);
        ++i;
        __builtin_amdgcn_sched_barrier(0);
        load_weights(a, K, std::min(j + u + U, j1 - 1), w[u]);
      }
    }
  }
}

// The waves' sums of both strips, joined in wave order: thread tid gets element
// i = tid % 4 of lane tid / 4 (feature 4 (l / 16) + i, token l % 16).
template <int NT>
__device__ inline void join(f32x4 (&acc)[2][NT], float (&out)[2][NT], f32x4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();  // every wave is done with its staged x
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[((wave * 2 + r) * NT + t) * 64 + lane] = acc[r][t];
  __syncthreads();
  const float* f = reinterpret_cast<const float*>(red);
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float v = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += f[((w * 2 + r) * NT + t) * 256 + threadIdx.x];
      out[r][t] = v;
    }
  __syncthreads();  // the LDS may be staged into again
}

// out[r][t] of two strips: rows r0 of matrix m0 and r1 of m1 (expert e), for
// the x rows given per lane, K the contraction length; its waves split K.
template <WKind KIND, int GPT, int PARTS, int NT>
__device__ inline void strip_pair(const WMat& m0, const WMat& m1, int64_t e, int64_t r0, int64_t r1, int64_t N,
                                  int64_t K, const Rows& x, float (&out)[2][NT], char* lds) {
  const int wave = uniform(threadIdx.x >> 6);
  f32x4 acc[2][NT] = {};
  const int64_t units = units_of<KIND>(K);
  const Strip<KIND> a[2] = {strip_of<KIND, GPT>(m0, e, r0, N, K), strip_of<KIND, GPT>(m1, e, r1, N, K)};
  mac<KIND, GPT, PARTS>(a, x, K, units * wave / kWaves, units * (wave + 1) / kWaves,
                        lds + wave * Stage<KIND, GPT, PARTS, 2, NT>::kBytes, acc);
  join<NT>(acc, out, reinterpret_cast<f32x4*>(lds));
}

// Rows row(c), c = 0 .. n - 1, of `stride` bytes each from base.
template <typename F>
__device__ inline Rows rows_of(const void* base, int64_t stride, int64_t part, int n, F&& row) {
  const int lane = threadIdx.x & 63;
  return Rows{static_cast<const char*>(base),
              static_cast<uint32_t>(row(std::min(lane, n - 1))) * static_cast<uint32_t>(stride), n, part};
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
  void* out;
};

// h = silu(g) u of 16 features for an expert's tokens.
template <WKind KIND, int GPT, int PARTS, int NT>
__device__ inline void gate_up_tile(const FewArgs& a, int64_t e, int p0, int n, int64_t f0, char* lds) {
  constexpr int kElem = sizeof(XType<KIND>);
  const Rows x = rows_of(a.x, a.d * kElem, a.T * a.d * kElem, n, [&](int c) { return a.ls.token[p0 + c]; });
  float v[2][NT];
  strip_pair<KIND, GPT, PARTS, NT>(a.gate, a.up, e, f0, f0, a.f, a.d, x, v, lds);
  const int l = threadIdx.x >> 2;
  const int64_t feat = f0 + 4 * (l >> 4) + (threadIdx.x & 3);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + (l & 15);
    if (c >= n || feat >= a.f) continue;
    const float g = v[0][t], u = v[1][t];
    const float h = g / (1.f + expf(-g)) * u;
    const int64_t at = (p0 + c) * a.ldh + feat;
    if constexpr (KIND == kDenseF32) {
      static_cast<float*>(a.h)[at] = h;
    } else if constexpr (PARTS == 1) {
      static_cast<bf16_t*>(a.h)[at] = f32_to_bf16(h);  // as the layer rounds h between its two products
    } else {
      const int64_t part = static_cast<int64_t>(a.T) * a.k * a.ldh;
      bf16_t q[3];
      split3(h, q);
#pragma unroll
      for (int i = 0; i < 3; ++i) static_cast<bf16_t*>(a.h)[i * part + at] = q[i];
    }
  }
}

// CALL for an expert's copies p .. p + n - 1, 16 at a time or (WIDE) 32. More
// copies read the weights again, from the caches.
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

// LDS bytes of a work-group that works on pairs of strips.
template <WKind KIND, int GPT, int PARTS, bool WIDE>
constexpr int kPairLds = kWaves * Stage<KIND, GPT, PARTS, 2, WIDE ? 2 : 1>::kBytes;

template <WKind KIND, int GPT, int PARTS, bool WIDE>
__global__ __launch_bounds__(kThreads, waves_per_simd(KIND, PARTS, WIDE)) void few_gate_up_kernel(FewArgs a) {
  __shared__ f32x4 lds[kPairLds<KIND, GPT, PARTS, WIDE> / 16];
  const int64_t ft = ceil_div(a.f, 16);
  const int64_t i = blockIdx.x / ft;
  const int n_act = *a.ls.n_act;  // the four loads together: past n_act the lists hold anything
  const int e = uniform(a.ls.act_e[i]), p0 = uniform(a.ls.act_off[i]), p1 = uniform(a.ls.act_off[i + 1]);
  if (i >= n_act) return;
  MOE_BY_TOKENS(p0, p1 - p0,
                (gate_up_tile<KIND, GPT, PARTS, NT>(a, e, p, n, (blockIdx.x % ft) * 16, reinterpret_cast<char*>(lds))));
}

// out for 16 of its columns: x plus the gate-weighted sums of all experts'
// down products. A work-group reads the strip's rows of every expert with
// copies; the units of all of them, expert after expert, are dealt to the
// waves in equal runs. A wave adds each expert's part of its run, times the
// gates, to its own sums of the T tokens in LDS, and these are joined in wave
// order: no y goes to memory, nothing waits for another work-group.
template <WKind KIND, int GPT, int PARTS, int NT>
__device__ inline void down_run(const FewArgs& a, int64_t e, int p0, int n, int64_t c0, int64_t j0, int64_t j1,
                                char* lds, float* sums) {
  const int lane = threadIdx.x & 63;
  const int64_t row = a.ldh * sizeof(XType<KIND>);
  const Rows x = rows_of(static_cast<const char*>(a.h) + p0 * row, row, a.T * a.k * row, n, [](int c) { return c; });
  f32x4 acc[1][NT] = {};
  const Strip<KIND> s[1] = {strip_of<KIND, GPT>(a.down, e, c0, a.d, a.f)};
  mac<KIND, GPT, PARTS>(s, x, a.f, j0, j1, lds, acc);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + (lane & 15);
    if (c >= n) continue;
    const float w = a.ls.gate[p0 + c];
    f32x4* o = reinterpret_cast<f32x4*>(sums + a.ls.token[p0 + c] * 16) + (lane >> 4);
    *o += w * acc[0][t];
  }
}

template <WKind KIND, int GPT, int PARTS, bool WIDE, int WAVES>
__global__ __launch_bounds__(WAVES * 64, is_dense(KIND) || !(WIDE || PARTS == 3) ? 4 : 2) void few_down_kernel(FewArgs a) {
  constexpr int kStage = Stage<KIND, GPT, PARTS, 1, WIDE ? 2 : 1>::kBytes;
  __shared__ f32x4 staged[WAVES * kStage / 16];
  extern __shared__ f32x4 all_sums_[];  // [WAVES][T][16] floats
  float* all_sums = reinterpret_cast<float*>(all_sums_);
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  float* sums = all_sums + wave * a.T * 16;
  char* lds = reinterpret_cast<char*>(staged) + wave * kStage;
  for (int i = lane; i < a.T * 16; i += 64) sums[i] = 0.f;
  const int64_t c0 = blockIdx.x * 16ll;
  const int64_t units = units_of<KIND>(a.f), total = units * uniform(*a.ls.n_act);
  const int64_t end = total * (wave + 1) / WAVES;
  for (int64_t u = total * wave / WAVES; u < end;) {
    const int64_t i = u / units, j0 = u % units, j1 = std::min(units, j0 + end - u);
    const int e = uniform(a.ls.act_e[i]), p0 = uniform(a.ls.act_off[i]);
    MOE_BY_TOKENS(p0, uniform(a.ls.act_off[i + 1]) - p0, (down_run<KIND, GPT, PARTS, NT>(a, e, p, n, c0, j0, j1, lds, sums)));
    u += j1 - j0;
  }
  __syncthreads();
  constexpr bool kBf16 = KIND == kDenseBf16 || (!is_dense(KIND) && PARTS == 1);
  for (int i = threadIdx.x; i < a.T * 16; i += WAVES * 64) {
    const int64_t col = c0 + (i & 15), at = (i >> 4) * a.d + col;
    if (col >= a.d) continue;
    float v = all_sums[i];
    for (int w = 1; w < WAVES; ++w) v += all_sums[w * a.T * 16 + i];
    if constexpr (kBf16)
      static_cast<bf16_t*>(a.out)[at] = f32_to_bf16(bf16_to_f32(static_cast<const bf16_t*>(a.x_res)[at]) + v);
    else
      static_cast<float*>(a.out)[at] = static_cast<const float*>(a.x_res)[at] + v;
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

// Rows with the same expert, grouped by the first wave: groups in the order of
// their first row, rows in order. Rows with an expert outside [0, E) are left out.
struct RowGroups {
  int n, e[64], off[65], row[64];
};

__device__ inline void group_rows(const int32_t* expert, int R, int E, RowGroups& g) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int e = -1;
    if (lane < R) e = expert ? expert[lane] : 0;
    const bool valid = lane < R && e >= 0 && e < E;
    bool leads = valid;
    unsigned long long mates = 0;
    for (int r = 0; r < R; ++r) {
      const int o = __shfl(valid ? e : -1, r);
      if (valid && o == e) {
        mates |= 1ull << r;
        if (r < lane) leads = false;
      }
    }
    const unsigned long long leaders = __ballot(leads), below = (1ull << lane) - 1ull;
    const int size = leads ? __popcll(mates) : 0;
    int off = size;  // exclusive sum of the sizes of the groups before
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(off, o);
      if (lane >= o) off += up;
    }
    if (lane == 63) {
      g.n = __popcll(leaders);
      g.off[g.n] = off;
    }
    off -= size;
    if (leads) {
      const int at = __popcll(leaders & below);
      g.e[at] = e;
      g.off[at] = off;
    }
    const int first = __shfl(off, valid ? __ffsll(mates) - 1 : 0);  // of the group's leader
    if (valid) g.row[first + __popcll(mates & below)] = lane;
  }
  __syncthreads();
}

template <WKind KIND, int GPT, int PARTS, int NT>
__device__ inline void matvec_tile(const MatvecArgs& a, const RowGroups& g, int i, int p0, int n, int64_t n0,
                                   char* lds) {
  const Rows x = rows_of(a.x, a.K * 2, a.R * a.K * 2, n, [&](int c) { return g.row[p0 + c]; });
  float v[2][NT];
  // the last 16 rows of a matrix may have no 16 after them: they are read twice
  const int64_t n1 = n0 + 16 < a.N ? n0 + 16 : n0;
  strip_pair<KIND, GPT, PARTS, NT>(a.w, a.w, uniform(g.e[i]), n0, n1, a.N, a.K, x, v, lds);
  const int l = threadIdx.x >> 2;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + (l & 15);
    if (c >= n) continue;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t col = n0 + 16 * r + 4 * (l >> 4) + (threadIdx.x & 3);
      if (col >= a.N) continue;
      const int64_t at = g.row[p0 + c] * a.N + col;
      if constexpr (PARTS == 1)
        static_cast<bf16_t*>(a.out)[at] = f32_to_bf16(v[r][t]);
      else
        static_cast<float*>(a.out)[at] = v[r][t];
    }
  }
}

template <WKind KIND, int GPT, int PARTS, bool WIDE>
__global__ __launch_bounds__(kThreads, waves_per_simd(KIND, PARTS, WIDE)) void matvec_kernel(MatvecArgs a) {
  __shared__ f32x4 lds[kPairLds<KIND, GPT, PARTS, WIDE> / 16];
  __shared__ RowGroups g;
  group_rows(a.expert, a.R, a.E, g);
  const int64_t nt = ceil_div(a.N, 32);
  const int i = static_cast<int>(blockIdx.x / nt);
  if (i >= g.n) return;
  const int p0 = uniform(g.off[i]);
  MOE_BY_TOKENS(p0, uniform(g.off[i + 1]) - p0,
                (matvec_tile<KIND, GPT, PARTS, NT>(a, g, i, p, n, (blockIdx.x % nt) * 32, reinterpret_cast<char*>(lds))));
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

}  // namespace

// Slices of d for the router scores: enough work-groups to spread W_router
// over the chip, slices of 512 columns at least, and few enough partial scores
// to add up.
int few_router_splits(int64_t T, int64_t d, int E) {
  const int64_t tiles = std::max<int64_t>(1, ceil_div(E, 16) * ceil_div(T, 16));
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, d / 512, 256 / tiles})));
}

hipError_t launch_few_layer(const FewLayer& L, hipStream_t s) {
  const bool bf16 = L.bf16;
  const int S = few_router_splits(L.T, L.d, L.E);
  const dim3 rgrid(static_cast<unsigned>(ceil_div(L.E, 16)), static_cast<unsigned>(ceil_div(L.T, 16)), S);
  if (bf16)
    few_router_kernel<true><<<rgrid, dim3(kThreads), 0, s>>>(L.x, L.wr, L.T, L.E, L.d, S, L.part, nullptr, nullptr, 0);
  else
    few_router_kernel<false><<<rgrid, dim3(kThreads), 0, s>>>(L.x, L.wr, L.T, L.E, L.d, S, L.part, L.xparts, nullptr, 0);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const RouteOut ro{L.idx, L.w, L.slot, L.routed, L.kept, L.send, L.totals};
  const int64_t row = L.d * (bf16 ? 2 : 4);
  if (L.E <= 64)
    few_route_kernel<1><<<dim3(1), dim3(1024), 0, s>>>(L.part, S, L.bias, L.T, L.E, L.k, L.P, L.M, L.C, row, ro, L.ls);
  else if (L.E <= 256)
    few_route_kernel<4><<<dim3(1), dim3(1024), 0, s>>>(L.part, S, L.bias, L.T, L.E, L.k, L.P, L.M, L.C, row, ro, L.ls);
  else
    few_route_kernel<16><<<dim3(1), dim3(1024), 0, s>>>(L.part, S, L.bias, L.T, L.E, L.k, L.P, L.M, L.C, row, ro, L.ls);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  FewArgs a;
  a.T = L.T;
  a.E = L.E;
  a.k = L.k;
  a.d = L.d;
  a.f = L.f;
  a.x = L.xparts ? static_cast<const void*>(L.xparts) : L.x;
  a.x_res = L.x;
  a.gate = {L.wt.w[0], static_cast<const bf16_t*>(L.wt.scale[0]), static_cast<const uint8_t*>(L.wt.zero[0])};
  a.up = {L.wt.w[1], static_cast<const bf16_t*>(L.wt.scale[1]), static_cast<const uint8_t*>(L.wt.zero[1])};
  a.down = {L.wt.w[2], static_cast<const bf16_t*>(L.wt.scale[2]), static_cast<const uint8_t*>(L.wt.zero[2])};
  a.ls = L.ls;
  a.h = L.h;
  a.ldh = few_ld_h(L.f);
  a.out = L.out;
  const int64_t act = std::min<int64_t>(L.E, static_cast<int64_t>(L.T) * L.k);  // experts with copies, at most
  const int64_t strips = ceil_div(L.d, 16);
  // two token tiles at a time where experts have more than half of one on average
  const bool wide = static_cast<int64_t>(L.T) * L.k > 8 * static_cast<int64_t>(L.E);
  return by_weights(L.wt, bf16, wide, [&](auto kind, auto gpt, auto parts, auto two) {
    constexpr WKind kKind = decltype(kind)::value;
    constexpr int kGpt = decltype(gpt)::value, kParts = decltype(parts)::value;
    constexpr bool kWide = decltype(two)::value;
    few_gate_up_kernel<kKind, kGpt, kParts, kWide>
        <<<dim3(static_cast<unsigned>(act * ceil_div(L.f, 16))), dim3(kThreads), 0, s>>>(a);
    constexpr int kMany = kParts == 1 && !kWide ? 16 : 8;
    // enough waves to cover the memory's latency with few columns too
    if (strips > 256)
      few_down_kernel<kKind, kGpt, kParts, kWide, 8>
          <<<dim3(static_cast<unsigned>(strips)), dim3(512), 8 * L.T * 64, s>>>(a);
    else
      few_down_kernel<kKind, kGpt, kParts, kWide, kMany>
          <<<dim3(static_cast<unsigned>(strips)), dim3(kMany * 64), kMany * L.T * 64, s>>>(a);
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
  a.w = {w.w[0], static_cast<const bf16_t*>(w.scale[0]), static_cast<const uint8_t*>(w.zero[0])};
  a.out = out;
  const int64_t groups = expert ? std::min(E, R) : 1;
  return by_weights(w, bf16, R > 8 * groups, [&](auto kind, auto gpt, auto parts_, auto two) {
    constexpr WKind kKind = decltype(kind)::value;
    if constexpr (kKind == kU4 || kKind == kE2m1) {
      matvec_kernel<kKind, decltype(gpt)::value, decltype(parts_)::value, decltype(two)::value>
          <<<dim3(static_cast<unsigned>(groups * ceil_div(N, 32))), dim3(kThreads), 0, s>>>(a);
      return hipGetLastError();
    } else {
      return hipErrorInvalidValue;
    }
  });
}

}  // namespace moe
