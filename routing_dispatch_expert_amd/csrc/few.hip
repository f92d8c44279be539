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

__device__ inline bf16x8 load8(const bf16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

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
    ls.pos[i] = pos;
    if (keep) ls.token[pos] = i / k;
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
// Products of two 16-row weight tiles with NT tiles of 16 rows of x over a
// range of the contraction: acc[r][t] += W_r x_t^T, one 16 x 16 tile in the
// matrix instructions' layout (lane: token lane % 16, features 4 (lane / 16) + i).
// ---------------------------------------------------------------------------

// Weight rows [N, K] of one matrix; x rows given per lane.
template <int NT>
__device__ inline void mac(const bf16_t* a0, const bf16_t* a1, const bf16_t* const (&b)[NT], int64_t K, int64_t j0,
                           int64_t j1, f32x4 (&acc)[2][NT]) {
  const int quad = (threadIdx.x & 63) >> 4;
#pragma unroll 4
  for (int64_t j = j0; j < j1; ++j) {
    const int64_t c = j * 32 + 8 * quad;
    bf16x8 w0 = {}, w1 = {};
    if (c < K) {
      w0 = load8(a0 + c);
      w1 = load8(a1 + c);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      bf16x8 xv = {};
      if (c < K) xv = load8(b[t] + c);
      acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, xv, acc[0][t], 0, 0, 0);
      acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, xv, acc[1][t], 0, 0, 0);
    }
  }
}

template <int NT>
__device__ inline void mac(const float* a0, const float* a1, const float* const (&b)[NT], int64_t K, int64_t j0,
                           int64_t j1, f32x4 (&acc)[2][NT]) {
  const int quad = (threadIdx.x & 63) >> 4;
#pragma unroll 4
  for (int64_t j = j0; j < j1; ++j) {
    const int64_t c = j * 16 + 4 * quad;  // the four columns go to four instructions: any order of k will do
    f32x4 w0 = {}, w1 = {};
    if (c < K) {
      w0 = *reinterpret_cast<const f32x4*>(a0 + c);
      w1 = *reinterpret_cast<const f32x4*>(a1 + c);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 xv = {};
      if (c < K) xv = *reinterpret_cast<const f32x4*>(b[t] + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(w0[i], xv[i], acc[0][t], 0, 0, 0);
        acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(w1[i], xv[i], acc[1][t], 0, 0, 0);
      }
    }
  }
}

// 4-bit weights: tiles [K/128][1024 bytes] of each 16-row strip, and its
// scales and zero points [groups][16]. The codes enter the matrix instruction
// as 16 + q (u4) or as their value (e2m1), exact in bf16; each group's sum is
// scaled in fp32:  sum_k s (q - z) x = s (sum (16 + q) x - (16 + z) sum x), the
// last sum by one more instruction with a tile of ones. The offset is 16 and
// not larger because the difference loses as many bits as it exceeds q.
// PARTS = 3: fp32 x as the exact sum of three bf16 arrays, `part` elements apart.
template <bool U4>
struct Strip {
  const uint4* tiles;    // this lane's 16 bytes of the strip's first tile
  const bf16_t* scale;   // this lane's 4 rows of the strip's first group
  const uint8_t* zero;   // NULL: 8
};

template <bool U4, int GPT>  // groups of a 128-column tile: 4, 2, 1
__device__ inline void rows_scale(const Strip<U4>& st, int64_t grp, float (&s)[4], float (&off)[4]) {
  const uint2 sv = *reinterpret_cast<const uint2*>(st.scale + grp * 16);
  s[0] = __uint_as_float(sv.x << 16);
  s[1] = __uint_as_float(sv.x & 0xffff0000u);
  s[2] = __uint_as_float(sv.y << 16);
  s[3] = __uint_as_float(sv.y & 0xffff0000u);
  if constexpr (U4) {
    uint32_t z = 0x08080808u;
    if (st.zero) z = *reinterpret_cast<const uint32_t*>(st.zero + grp * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) off[i] = 16.f + static_cast<float>((z >> (8 * i)) & 0xffu);
  }
}

template <bool U4, int GPT, int PARTS, int NT>
__device__ inline void mac_q4(const Strip<U4>& a0, const Strip<U4>& a1, const bf16_t* const (&b)[NT], int64_t part,
                              int64_t K, int64_t j0, int64_t j1, f32x4 (&acc)[2][NT]) {
  const int quad = (threadIdx.x & 63) >> 4;
  constexpr int kSteps = 4 / GPT;  // 32-column steps of a group
  bf16x8 ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = static_cast<__bf16>(1.0f);
  for (int64_t j = j0; j < j1; ++j) {
    const uint4 w0 = a0.tiles[j * 64], w1 = a1.tiles[j * 64];
    const uint32_t w0s[4] = {w0.x, w0.y, w0.z, w0.w}, w1s[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int g = 0; g < GPT; ++g) {
      if (j * 128 + g * 32 * kSteps >= K) break;  // padding groups: their scales are not looked at
      f32x4 s0[NT] = {}, s1[NT] = {}, sx[NT] = {};
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const int st = g * kSteps + q;
        const int64_t c = j * 128 + st * 32 + 8 * quad;
        const bf16x8 v0 = q4_decode<U4>(w0s[st]), v1 = q4_decode<U4>(w1s[st]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            bf16x8 xv = {};
            if (c < K) xv = load8(b[t] + p * part + c);
            s0[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, xv, s0[t], 0, 0, 0);
            s1[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, xv, s1[t], 0, 0, 0);
            if constexpr (U4) sx[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xv, sx[t], 0, 0, 0);
          }
      }
      float sc0[4], sc1[4], of0[4], of1[4];
      rows_scale<U4, GPT>(a0, j * GPT + g, sc0, of0);
      rows_scale<U4, GPT>(a1, j * GPT + g, sc1, of1);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (U4) {
            acc[0][t][i] = fmaf(sc0[i], fmaf(-of0[i], sx[t][i], s0[t][i]), acc[0][t][i]);
            acc[1][t][i] = fmaf(sc1[i], fmaf(-of1[i], sx[t][i], s1[t][i]), acc[1][t][i]);
          } else {
            acc[0][t][i] = fmaf(sc0[i], s0[t][i], acc[0][t][i]);
            acc[1][t][i] = fmaf(sc1[i], s1[t][i], acc[1][t][i]);
          }
        }
    }
  }
}

// One matrix stack [E, N, K] as the kernels take it.
struct WMat {
  const void* w;        // dense rows, or code tiles
  const bf16_t* scale;  // 4-bit only
  const uint8_t* zero;  // u4 only; NULL: 8
};

// The waves' sums of both tiles, joined in wave order: thread tid gets element
// i = tid % 4 of lane tid / 4 (feature 4 (l / 16) + i, token l % 16).
template <int NT>
__device__ inline void join(f32x4 (&acc)[2][NT], float (&out)[2][NT], f32x4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();  // the scratch's last readers are done
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
}

// out[r][t] of two 16-row tiles: rows r0 of matrix m0 and r1 of m1 (expert e),
// for the x rows given per lane, K the contraction length.
template <WKind KIND, int GPT, int PARTS, int NT, typename XT>
__device__ inline void tile_pair(const WMat& m0, const WMat& m1, int64_t e, int64_t r0, int64_t r1, int64_t N,
                                 int64_t K, const XT* const (&xr)[NT], int64_t part, float (&out)[2][NT], f32x4* red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  f32x4 acc[2][NT] = {};
  if constexpr (KIND == kDenseBf16 || KIND == kDenseF32) {
    constexpr int kStep = KIND == kDenseBf16 ? 32 : 16;
    const int64_t steps = ceil_div(K, kStep);
    const int64_t j0 = steps * wave / kWaves, j1 = steps * (wave + 1) / kWaves;
    // rows past the matrix repeat its last one; their results are not stored
    const XT* a0 = static_cast<const XT*>(m0.w) + (e * N + std::min(r0 + (lane & 15), N - 1)) * K;
    const XT* a1 = static_cast<const XT*>(m1.w) + (e * N + std::min(r1 + (lane & 15), N - 1)) * K;
    mac<NT>(a0, a1, xr, K, j0, j1, acc);
  } else {
    constexpr bool kIsU4 = KIND == kU4;
    const int64_t nt = ceil_div(N, 16), kt = ceil_div(K, 128);
    const int64_t j0 = kt * wave / kWaves, j1 = kt * (wave + 1) / kWaves;
    const int64_t t0 = e * nt + r0 / 16, t1 = e * nt + std::min(r1 / 16, nt - 1);
    auto strip = [&](const WMat& m, int64_t t) {
      Strip<kIsU4> s;
      s.tiles = static_cast<const uint4*>(m.w) + t * kt * 64 + lane;
      const int64_t at = t * kt * GPT * 16 + 4 * (lane >> 4);
      s.scale = m.scale + at;
      s.zero = m.zero ? m.zero + at : nullptr;
      return s;
    };
    mac_q4<kIsU4, GPT, PARTS, NT>(strip(m0, t0), strip(m1, t1), xr, part, K, j0, j1, acc);
  }
  join<NT>(acc, out, red);
}

struct FewArgs {
  int T, E, k;
  int64_t d, f;
  const void* x;         // x as the experts read it: [T, d], or its bf16 parts [PARTS][T][d]
  const void* x_res;     // the residual, [T, d] in the layer's type
  WMat gate, up, down;
  FewLists ls;
  const float* w;        // gates [T, k]
  void* h;               // [PARTS][T k][ldh], by position in the lists
  float* y;              // [T k][ldy]
  int64_t ldh, ldy;
  void* out;
};

template <WKind KIND, int PARTS>
using XType = std::conditional_t<KIND == kDenseF32, float, bf16_t>;

// h = silu(g) u of 16 features for an expert's tokens.
template <WKind KIND, int GPT, int PARTS, int NT>
__device__ inline void gate_up_tile(const FewArgs& a, int64_t e, int p0, int n, int64_t f0, f32x4* red) {
  using XT = XType<KIND, PARTS>;
  const int lane = threadIdx.x & 63;
  const XT* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)  // columns past the expert's copies repeat its last one; they are not stored
    xr[t] = static_cast<const XT*>(a.x) + static_cast<int64_t>(a.ls.token[p0 + std::min(t * 16 + (lane & 15), n - 1)]) * a.d;
  float v[2][NT];
  tile_pair<KIND, GPT, PARTS, NT, XT>(a.gate, a.up, e, f0, f0, a.f, a.d, xr, a.T * a.d, v, red);
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

// y = h W_down^T for 32 columns of an expert's tokens, kept in fp32.
template <WKind KIND, int GPT, int PARTS, int NT>
__device__ inline void down_tile(const FewArgs& a, int64_t e, int p0, int n, int64_t n0, f32x4* red) {
  using XT = XType<KIND, PARTS>;
  const int lane = threadIdx.x & 63;
  const XT* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    xr[t] = static_cast<const XT*>(a.h) + (p0 + std::min(t * 16 + (lane & 15), n - 1)) * a.ldh;
  float v[2][NT];
  tile_pair<KIND, GPT, PARTS, NT, XT>(a.down, a.down, e, n0, n0 + 16, a.d, a.f, xr,
                                      static_cast<int64_t>(a.T) * a.k * a.ldh, v, red);
  const int l = threadIdx.x >> 2;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = t * 16 + (l & 15);
    if (c >= n) continue;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t col = n0 + 16 * r + 4 * (l >> 4) + (threadIdx.x & 3);
      if (col < a.d) a.y[(p0 + c) * a.ldy + col] = v[r][t];
    }
  }
}

// One instance for each number of 16-token tiles that an expert's copies take.
#define MOE_BY_TOKENS(n, CALL) \
  do {                         \
    if ((n) <= 16) {           \
      constexpr int NT = 1;    \
      CALL;                    \
    } else if ((n) <= 32) {    \
      constexpr int NT = 2;    \
      CALL;                    \
    } else {                   \
      constexpr int NT = 4;    \
      CALL;                    \
    }                          \
  } while (0)

constexpr int kRedWords = kWaves * 2 * 4 * 64;  // f32x4 words of the joining scratch, NT = 4

template <WKind KIND, int GPT, int PARTS>
__global__ __launch_bounds__(kThreads, 4) void few_gate_up_kernel(FewArgs a) {
  __shared__ f32x4 red[kRedWords];
  const int64_t ft = ceil_div(a.f, 16);
  const int64_t i = blockIdx.x / ft;
  if (i >= *a.ls.n_act) return;
  const int e = a.ls.act_e[i], p0 = a.ls.act_off[i], n = a.ls.act_off[i + 1] - p0;
  MOE_BY_TOKENS(n, (gate_up_tile<KIND, GPT, PARTS, NT>(a, e, p0, n, (blockIdx.x % ft) * 16, red)));
}

template <WKind KIND, int GPT, int PARTS>
__global__ __launch_bounds__(kThreads, 4) void few_down_kernel(FewArgs a) {
  __shared__ f32x4 red[kRedWords];
  const int64_t nt = ceil_div(a.d, 32);
  const int64_t i = blockIdx.x / nt;
  if (i >= *a.ls.n_act) return;
  const int e = a.ls.act_e[i], p0 = a.ls.act_off[i], n = a.ls.act_off[i + 1] - p0;
  MOE_BY_TOKENS(n, (down_tile<KIND, GPT, PARTS, NT>(a, e, p0, n, (blockIdx.x % nt) * 32, red)));
}

// out = x + sum over the kept copies, j ascending, of w y: fp32, rounded once.
// A token without a kept copy is copied bit for bit.
template <bool BF16>
__global__ __launch_bounds__(256) void few_combine_kernel(FewArgs a) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= a.T * a.d) return;
  const int64_t t = i / a.d, c = i % a.d;
  float v = BF16 ? bf16_to_f32(static_cast<const bf16_t*>(a.x_res)[i]) : static_cast<const float*>(a.x_res)[i];
  for (int j = 0; j < a.k; ++j) {
    const int pos = a.ls.pos[t * a.k + j];
    if (pos >= 0) v = fmaf(a.w[t * a.k + j], a.y[pos * a.ldy + c], v);
  }
  if (BF16)
    static_cast<bf16_t*>(a.out)[i] = f32_to_bf16(v);
  else
    static_cast<float*>(a.out)[i] = v;
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
__device__ inline void matvec_tile(const MatvecArgs& a, const RowGroups& g, int i, int64_t n0, f32x4* red) {
  const int lane = threadIdx.x & 63;
  const int p0 = g.off[i], n = g.off[i + 1] - p0;
  const bf16_t* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    xr[t] = a.x + static_cast<int64_t>(g.row[p0 + std::min(t * 16 + (lane & 15), n - 1)]) * a.K;
  float v[2][NT];
  tile_pair<KIND, GPT, PARTS, NT, bf16_t>(a.w, a.w, g.e[i], n0, n0 + 16, a.N, a.K, xr, a.R * a.K, v, red);
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

template <WKind KIND, int GPT, int PARTS>
__global__ __launch_bounds__(kThreads, 4) void matvec_kernel(MatvecArgs a) {
  __shared__ f32x4 red[kRedWords];
  __shared__ RowGroups g;
  group_rows(a.expert, a.R, a.E, g);
  const int64_t nt = ceil_div(a.N, 32);
  const int i = static_cast<int>(blockIdx.x / nt);
  if (i >= g.n) return;
  MOE_BY_TOKENS(g.off[i + 1] - g.off[i], (matvec_tile<KIND, GPT, PARTS, NT>(a, g, i, (blockIdx.x % nt) * 32, red)));
}

__global__ __launch_bounds__(256) void split_kernel(const float* x, int64_t n, bf16_t* parts) {
  split_rows(x, n, parts, blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll);
}

// f(kind, groups per tile, parts) with compile-time arguments.
template <typename F>
hipError_t by_weights(const FewWeights& w, bool bf16, F&& f) {
  using std::integral_constant;
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
  a.w = L.w;
  a.h = L.h;
  a.y = L.y;
  a.ldh = few_ld_h(L.f);
  a.ldy = few_ld_y(L.d);
  a.out = L.out;
  const int64_t act = std::min<int64_t>(L.E, static_cast<int64_t>(L.T) * L.k);  // experts with copies, at most
  return by_weights(L.wt, bf16, [&](auto kind, auto gpt, auto parts) {
    constexpr WKind kKind = decltype(kind)::value;
    constexpr int kGpt = decltype(gpt)::value, kParts = decltype(parts)::value;
    few_gate_up_kernel<kKind, kGpt, kParts>
        <<<dim3(static_cast<unsigned>(act * ceil_div(L.f, 16))), dim3(kThreads), 0, s>>>(a);
    few_down_kernel<kKind, kGpt, kParts>
        <<<dim3(static_cast<unsigned>(act * ceil_div(L.d, 32))), dim3(kThreads), 0, s>>>(a);
    const dim3 cg(static_cast<unsigned>(ceil_div(L.T * L.d, 256)));
    if (bf16)
      few_combine_kernel<true><<<cg, dim3(256), 0, s>>>(a);
    else
      few_combine_kernel<false><<<cg, dim3(256), 0, s>>>(a);
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
  return by_weights(w, bf16, [&](auto kind, auto gpt, auto parts_) {
    constexpr WKind kKind = decltype(kind)::value;
    if constexpr (kKind == kU4 || kKind == kE2m1) {
      matvec_kernel<kKind, decltype(gpt)::value, decltype(parts_)::value>
          <<<dim3(static_cast<unsigned>(groups * ceil_div(N, 32))), dim3(kThreads), 0, s>>>(a);
      return hipGetLastError();
    } else {
      return hipErrorInvalidValue;
    }
  });
}

}  // namespace moe
