// The gate of the MoE layer in its general form, and its gradient (gfx950).
//
// Sources: "Expert Parallelism" (klaylearn.com glossary) - scores, top-k choice
// and combine weights; "Expert Parallelism & All-to-All" (neelmishra.github.io),
// "The bandwidth bill" - a token's experts limited to a few nodes.
//
//   s = sigmoid(l) or softmax(l) over the E experts;  v = s + bias, or the order of
//   l itself without a bias (s grows with l); a group's value: the sum of its
//   `best` largest v (of s without a bias and best = 2; max l with best = 1)
//   idx = the k largest v of the top_groups best groups' experts
//   w_j = scale s_j / sum over the chosen of s, or scale s_j
//
// Scores, sums and comparisons are in fp64: the scores of 256 experts lie so
// close that in fp32 a rounding would swap one token's neighbours in some tens
// of thousands, and the choice is compared elsewhere for equality. A wave has a
// token; lane l holds the experts l, l + 64, ...
#include "block.h"

#include <climits>

namespace moe {
namespace {

// Monotone map of a double to uint64; NaN lies below every number, and 0 below NaN.
__device__ inline uint64_t order_of(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));  // -0 as 0
  const uint64_t key = (u >> 63) ? ~u : (u | (uint64_t{1} << 63));
  return v != v ? 1 : key;
}

__device__ inline double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// A word of the lane that many places below (or, from the last two, of the last
// lane of the rows below); 0 where there is none. Register moves, without LDS: a
// wave's reductions here are chains of them, and one through LDS takes ten times
// as long.
template <int CTRL, int ROWS>
__device__ inline uint32_t below(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ inline double below(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  return __longlong_as_double(static_cast<int64_t>(static_cast<uint64_t>(below<CTRL, ROWS>(static_cast<uint32_t>(u >> 32))) << 32 |
                                                   below<CTRL, ROWS>(static_cast<uint32_t>(u))));
}
template <int CTRL, int ROWS>
__device__ inline float below(float v) {
  return __uint_as_float(below<CTRL, ROWS>(__float_as_uint(v)));
}

__device__ inline uint32_t lane_word(uint32_t v, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ inline uint64_t lane_word(uint64_t v, int lane) {
  return static_cast<uint64_t>(lane_word(static_cast<uint32_t>(v >> 32), lane)) << 32 | lane_word(static_cast<uint32_t>(v), lane);
}
__device__ inline double lane_word(double v, int lane) {
  return __longlong_as_double(static_cast<int64_t>(lane_word(static_cast<uint64_t>(__double_as_longlong(v)), lane)));
}
__device__ inline float lane_word(float v, int lane) { return __uint_as_float(lane_word(__float_as_uint(v), lane)); }

// Reductions over the wave, the same in every lane: shifts by 1, 2, 4, 8 within
// rows of 16 lanes, then the rows' last lanes onto the rows above.
template <typename V, typename F>
__device__ inline V wave_reduce(V v, F f) {
  v = f(v, below<0x111, 0xf>(v));
  v = f(v, below<0x112, 0xf>(v));
  v = f(v, below<0x114, 0xf>(v));
  v = f(v, below<0x118, 0xf>(v));
  v = f(v, below<0x142, 0xa>(v));
  v = f(v, below<0x143, 0xc>(v));
  return lane_word(v, 63);
}
// Maxima as integers in the numbers' order, of which 0 is below all.
__device__ inline uint32_t wave_max(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ inline uint64_t wave_max(uint64_t v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32), top = wave_max(hi);
  return static_cast<uint64_t>(top) << 32 | wave_max(hi == top ? static_cast<uint32_t>(v) : 0u);
}
template <typename V>
__device__ inline V wave_sum(V v) {
  return wave_reduce(v, [](V a, V b) { return a + b; });
}
// The same over lanes 0 .. k - 1, one after the other.
__device__ inline double first_sum(double v, int k) {
  double sum = 0;
  for (int j = 0; j < k; ++j) sum += lane_word(v, j);
  return sum;
}
__device__ inline double first_max(double v, int k) {
  double m = -INFINITY;
  for (int j = 0; j < k; ++j) m = fmax(m, lane_word(v, j));
  return m;
}

// The two largest (a >= b) of a lane's and another's.
template <int CTRL>
__device__ inline void join_two(double& a, double& b) {
  const double oa = below<CTRL, 0xf>(a), ob = below<CTRL, 0xf>(b);
  b = fmax(fmin(a, oa), fmax(b, ob));
  a = fmax(a, oa);
}

// The order's inverse, for numbers.
__device__ inline double number_of(uint64_t key) {
  return __longlong_as_double(static_cast<int64_t>(key >> 63 ? key & ~(uint64_t{1} << 63) : ~key));
}

// What the host divides for the kernel (a division by a number known only at run
// time takes some 30 instructions a wave; 8192 tokens, 8 groups of 32: 16.2 -> 15.0
// us without them): the experts of a group, the logarithm of
// the lanes that form a group's value (64 over the groups, rounded down to a power
// of two) and 1 / per.
struct GroupSplit {
  int per, log_lanes;
  float inv_per;
  // The group of expert e: (e + 1/2) / per lies 1 / (2 per) or more from a whole
  // number, and is off by less than 2^-21 E / per.
  __device__ int of(int e) const { return static_cast<int>((e + 0.5f) * inv_per); }
};

// NE: scores a lane holds (E <= 64 NE). LDS: [waves][E] doubles with groups.
template <int NE>
__global__ __launch_bounds__(256) void gate_kernel(const float* __restrict__ logits, const float* __restrict__ bias,
                                                   GateRule g, GroupSplit gs, int64_t T, int E, int k,
                                                   int32_t* __restrict__ idx, float* __restrict__ w) {
  extern __shared__ double smem[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + wave;
  if (t >= T) return;  // no barrier below
  double l[NE], s[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? static_cast<double>(logits[t * E + e]) : -INFINITY;
  }
  bool nan = false;  // a NaN or an infinity makes every score NaN, which a softmax over the chosen alone does not see
  if (!g.sigmoid && g.renormalize) {
#pragma unroll
    for (int i = 0; i < NE; ++i) nan = nan || !(l[i] < INFINITY);
    nan = __ballot(nan) != 0;
  }
  // the scores, where the choice needs them
  const bool scores = bias || (g.groups > 1 && g.best > 1) || (!g.sigmoid && !g.renormalize);
  double top = 0, total = 1;
  if (!g.sigmoid && scores) {
    top = l[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) top = fmax(top, l[i]);
    top = number_of(wave_max(order_of(top)));
    if (!(top > -INFINITY)) top = 0;  // every expert masked: all scores are 0
    total = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      s[i] = lane + 64 * i < E ? exp(l[i] - top) : 0;
      total += s[i];
    }
    total = wave_sum(total);
    if (total == 0) total = 1;
#pragma unroll
    for (int i = 0; i < NE; ++i) s[i] /= total;
  } else if (scores) {
#pragma unroll
    for (int i = 0; i < NE; ++i) s[i] = sigmoid64(l[i]);
  }
  uint64_t key[NE];
  int ex[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = ex[i] = lane + 64 * i;
    key[i] = e < E ? order_of(bias ? s[i] + static_cast<double>(bias[e]) : l[i]) : 0;
  }
  if (g.groups > 1) {
    const int per = gs.per, lpg = 1 << gs.log_lanes, sub = lane & (lpg - 1), mine = lane >> gs.log_lanes;
    double* v = smem + wave * E;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      if (e < E) v[e] = bias ? s[i] + static_cast<double>(bias[e]) : g.best > 1 ? s[i] : l[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    double a = -INFINITY, b = -INFINITY;  // the two largest of the lane's part of its group
    if (mine < g.groups)
      for (int i = sub; i < per; i += lpg) {
        const double x = v[mine * per + i];
        if (x > a) {
          b = a;
          a = x;
        } else if (x > b) {
          b = x;
        }
      }
    // joined over 2, 4, 8, 16 lanes: each with a lane of the other half, whose lanes agree (pairs, quads, mirrors)
    if (lpg > 1) join_two<0xb1>(a, b);
    if (lpg > 2) join_two<0x4e>(a, b);
    if (lpg > 4) join_two<0x141>(a, b);
    if (lpg > 8) join_two<0x140>(a, b);
    if (lpg > 16) {
      const double oa = __shfl_xor(a, 16, 64), ob = __shfl_xor(b, 16, 64);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    const double sum = g.best > 1 ? a + b : a;
    uint64_t value = order_of(sum);
    if (sum == -INFINITY && mine < g.groups) {  // of -inf, or of too few numbers beside NaN: below every number
      int numbers = 0;
      for (int i = 0; i < per; ++i) numbers += v[mine * per + i] == v[mine * per + i] ? 1 : 0;
      if (numbers < g.best) value = order_of(NAN);
    }
    int ahead = 0;  // groups that are better, or as good and before this one
    for (int o = 0; o < g.groups; ++o) {
      const uint64_t ov = lane_word(value, o << gs.log_lanes);
      ahead += (ov > value || (ov == value && o < mine)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(mine < g.groups && ahead < g.top_groups);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (gs.of(e) << gs.log_lanes)) & 1)) key[i] = 0;
    }
  }
  // Each lane's keys in order, of equal ones the lower expert first: a choice is then the best of the lanes' heads.
  // (Beyond eight a lane, a search of the lane's keys for each choice takes fewer steps.)
  constexpr bool SORTED = NE <= 8;
  if constexpr (SORTED) {
#pragma unroll
    for (int a = NE - 1; a > 0; --a)
#pragma unroll
      for (int i = 0; i < a; ++i) {
        const bool swap = key[i] < key[i + 1];
        const uint64_t hi = swap ? key[i + 1] : key[i], lo = swap ? key[i] : key[i + 1];
        const int he = swap ? ex[i + 1] : ex[i], le = swap ? ex[i] : ex[i + 1];
        key[i] = hi;
        key[i + 1] = lo;
        ex[i] = he;
        ex[i + 1] = le;
      }
  }
  int my_e = 0;  // lane j < k: the j-th choice
  for (int j = 0; j < k; ++j) {
    uint64_t best = key[0];
    int be = ex[0];
    if constexpr (!SORTED) {
#pragma unroll
      for (int i = 1; i < NE; ++i) {
        const bool better = key[i] > best;
        best = better ? key[i] : best;
        be = better ? ex[i] : be;
      }
    }
    // two lanes' bests seldom share the upper half; of equal ones the lowest expert
    const uint32_t hi = static_cast<uint32_t>(best >> 32), lo = static_cast<uint32_t>(best);
    const uint32_t top_hi = wave_max(hi);
    uint64_t like = __ballot(hi == top_hi);
    if (like & (like - 1)) {
      const bool in = (like >> lane) & 1;
      const uint32_t top_lo = wave_max(in ? lo : 0u);
      const bool tie = in && lo == top_lo;
      const uint32_t first = ~wave_max(tie ? ~static_cast<uint32_t>(be) : 0u);
      like = __ballot(tie && static_cast<uint32_t>(be) == first);
    }
    const int win = __builtin_ctzll(like);
    const int e = static_cast<int>(lane_word(static_cast<uint32_t>(be), win));
    if (lane == j) my_e = e;
    if (lane == win) {
      if constexpr (SORTED) {
#pragma unroll
        for (int i = 0; i + 1 < NE; ++i) {
          key[i] = key[i + 1];
          ex[i] = ex[i + 1];
        }
        key[NE - 1] = 0;
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (ex[i] == e) key[i] = 0;
      }
    }
  }
  const double my_l = lane < k ? static_cast<double>(logits[t * E + my_e]) : 0;
  // weights of the chosen
  const bool in = lane < k;
  double z;
  if (g.sigmoid) {
    z = in ? sigmoid64(my_l) : 0;
  } else if (g.renormalize) {  // a softmax over the chosen
    const double m = first_max(my_l, k);
    z = in && m > -INFINITY ? exp(my_l - m) : 0;
    if (nan) z = NAN;
  } else {
    z = in ? exp(my_l - top) / total : 0;
  }
  if (g.renormalize) {
    const double sum = first_sum(z, k);
    z = sum == 0 ? 0 : z / sum;  // a NaN stays one
  }
  if (in) {
    idx[t * k + lane] = my_e;
    w[t * k + lane] = static_cast<float>(static_cast<double>(g.scale) * z);
  }
}

// The gradient: with q_j = scale dw_j and D = sum q_i r_i over the chosen,
//   renormalised: r_j = s_j / sum s, and dl_j += r_j (q_j - D) (1 - s_j for sigmoid, 1 for softmax)
//   not:          sigmoid dl_j += q_j s_j (1 - s_j); softmax as if d_scores[j] were larger by q_j
//   d_scores:     sigmoid dl_e += ds_e s_e (1 - s_e), softmax dl_e += s_e (ds_e - sum_i ds_i s_i)
// The chosen ones' terms are in fp64 (a few a token), the dense ones in fp32.
template <int NE>
__global__ __launch_bounds__(256) void gate_backward_kernel(const float* __restrict__ logits,
                                                            const int32_t* __restrict__ idx,
                                                            const float* __restrict__ dw,
                                                            const float* __restrict__ dscores, GateRule g, int64_t T,
                                                            int E, int k, float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x * 4ll + wave;
  if (t >= T) return;
  float l[NE], ds[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? logits[t * E + e] : -INFINITY;
    ds[i] = dscores && e < E ? dscores[t * E + e] : 0.f;
  }
  bool nan = false;  // as in the forward: every score of a softmax is NaN
  if (!g.sigmoid) {
#pragma unroll
    for (int i = 0; i < NE; ++i) nan = nan || !(l[i] < INFINITY);
    nan = __ballot(nan) != 0;
  }
  int e_j = -1;
  double l_j = 0, q_j = 0;
  if (lane < k) {
    e_j = idx[t * k + lane];
    if (e_j >= 0 && e_j < E) {
      l_j = logits[t * E + e_j];
      q_j = static_cast<double>(g.scale) * static_cast<double>(dw[t * k + lane]);
    } else {
      e_j = -1;  // an index outside passes no gradient
    }
  }
  const bool in = e_j >= 0;
  double term;  // of dl, or of d_scores where softmax scores are not renormalised
  if (g.renormalize) {
    double z;
    if (g.sigmoid) {
      z = in ? sigmoid64(l_j) : 0;
    } else {
      const double m = first_max(in ? l_j : -INFINITY, k);
      z = in && m > -INFINITY ? exp(l_j - m) : 0;
      if (in && nan) z = NAN;
    }
    const double sum = first_sum(z, k);
    const double r = sum == 0 ? 0 : z / sum;  // a NaN stays one
    const double D = first_sum(q_j * r, k);
    term = r * (q_j - D) * (g.sigmoid ? sigmoid64(-l_j) : 1.0);
  } else {
    term = g.sigmoid ? q_j * sigmoid64(l_j) * sigmoid64(-l_j) : q_j;
  }
  const float add = in ? static_cast<float>(term) : 0.f;
  const bool soft = !g.sigmoid && !g.renormalize;  // the term belongs to d_scores
  float dl[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) dl[i] = 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = __builtin_amdgcn_readlane(e_j, j);
    const float v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(add), j));
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (e == lane + 64 * i) {
        if (soft)
          ds[i] += v;
        else
          dl[i] += v;
      }
  }
  if (dscores || soft) {
    if (g.sigmoid) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float a = expf(-fabsf(l[i])), b = 1.f / (1.f + a);  // s and 1 - s are b and a b
        dl[i] += ds[i] * (a * b * b);
      }
    } else {
      float m = l[0];
#pragma unroll
      for (int i = 1; i < NE; ++i) m = fmaxf(m, l[i]);
      const uint32_t mu = __float_as_uint(m + 0.f);
      const uint32_t mk = wave_max(mu >> 31 ? ~mu : mu | 0x80000000u);
      m = __uint_as_float(mk >> 31 ? mk & 0x7fffffffu : ~mk);
      float p[NE], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        p[i] = lane + 64 * i < E && m > -INFINITY ? expf(l[i] - m) : 0.f;
        sum += p[i];
        dot += p[i] * ds[i];
      }
      sum = wave_sum(sum);
      dot = wave_sum(dot);
      const float inv = nan ? NAN : sum > 0.f ? 1.f / sum : 0.f;  // 0: every expert masked
      dot *= inv;
#pragma unroll
      for (int i = 0; i < NE; ++i) dl[i] += p[i] * inv * (ds[i] - dot);
    }
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    if (e < E) dlogits[t * E + e] = dl[i];
  }
}

}  // namespace

#define MOE_GATE_BY_E(CALL)   \
  do {                        \
    if (E <= 64) {            \
      CALL(1);                \
    } else if (E <= 128) {    \
      CALL(2);                \
    } else if (E <= 256) {    \
      CALL(4);                \
    } else if (E <= 512) {    \
      CALL(8);                \
    } else if (E <= 1024) {   \
      CALL(16);               \
    } else {                  \
      CALL(64);               \
    }                         \
  } while (0)

hipError_t launch_gate(const float* logits, const float* bias, const GateRule& g, int64_t T, int E, int k, int32_t* idx,
                       float* w, hipStream_t s) {
  const int waves = E <= 1024 ? 4 : 1;  // at most 32 KiB of LDS
  const dim3 grid(static_cast<unsigned>(ceil_div(T, waves)));
  const int per = E / g.groups;
  const GroupSplit gs{per, 31 - __builtin_clz(64 / g.groups), 1.f / per};
  const size_t lds = g.groups > 1 ? waves * static_cast<size_t>(E) * sizeof(double) : 0;
#define MOE_CALL(NE) gate_kernel<NE><<<grid, dim3(64 * waves), lds, s>>>(logits, bias, g, gs, T, E, k, idx, w)
  MOE_GATE_BY_E(MOE_CALL);
#undef MOE_CALL
  return hipGetLastError();
}

hipError_t launch_gate_backward(const float* logits, const int32_t* idx, const float* dw, const float* dscores,
                                const GateRule& g, int64_t T, int E, int k, float* dlogits, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(T, 4)));
#define MOE_CALL(NE) gate_backward_kernel<NE><<<grid, dim3(256), 0, s>>>(logits, idx, dw, dscores, g, T, E, k, dlogits)
  MOE_GATE_BY_E(MOE_CALL);
#undef MOE_CALL
  return hipGetLastError();
}

}  // namespace moe
