// The experts of the MoE layer with 8-bit rows and weights, from a given routing
// (gfx950).
//
// Sources: "Expert Parallelism" (infra.bea.ai guide), section 1 - three weight
// matrices per expert; "Expert Parallelism & All-to-All" (neelmishra.github.io),
// "All-to-all: the distributed transpose" - gate-weighted sum into the residual.
//
//   h = mx8(silu(x Wg^T) * (x Wu^T));  y = h Wd^T, in fp32
//   out[t] = residual[t] + sum_j [slot[t, j] >= 0] w[t, j] y[t, j], rounded once
//
// The products run on the scaled 8-bit matrix instructions: 128 (or 64) columns
// an instruction, a scale for every 32. The weights are the A operand (an
// accumulator's rows are output features), the tokens the columns of B: a lane
// then has neighbouring features of one token, so that the 32 features that share
// a scale of h lie in a few lanes and four codes make a word. Within one
// instruction the matrix unit aligns the products to the largest one and drops
// what lies some 2^13 below it; the accumulators are fp32: sums over 4096 Gaussian
// products are off by 1.3e-5 of their size, far below the 2^-4 that the 8-bit
// operands are rounded by.
//
// No bucket is built: lists of the kept copies by expert, in token order, say
// which rows of x an expert reads and which rows of y it writes.
#include "mx8_experts.h"
#include "q4.h"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Lists, by one work-group. Copies are taken 64 a wave and up to 16 waves at a
// time; a copy's rank among its expert's is found by ballots over the expert's
// bits within its wave, by the waves' counts in LDS before that, and by the
// expert's running count: token order, nothing depends on arrival.
// ---------------------------------------------------------------------------
constexpr int kPlanCounts = 16384;  // counts of a round's waves: waves * E
// With more copies the layer's own launches, 24 us for any number of them, replace
// the one work-group (8192 copies: 23 - 27 us; 16384 53, 98304 272).
constexpr int64_t kPlanCopies = 8192;

// Exclusive prefix sum over the block's 1024 values; the total goes to *total.
__device__ inline int block_prefix(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(s, off, 64);
    if (lane >= off) s += o;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i < wave) before += sums[i];
    all += sums[i];
  }
  *total = all;
  return before + s - v;
}

// Rows, row tiles of bt rows and places among the experts that have rows, as prefix
// sums over the experts' counts by one work-group; count [E] becomes the experts'
// first rows.
__device__ inline void list_experts(int32_t* count, int E, int64_t C, int bt, int32_t* routed, int32_t* kept,
                                    const ExpertLists& ls, int* sums) {
  const int tid = threadIdx.x;
  int rows0 = 0, tiles0 = 0, act0 = 0;
  for (int e0 = 0; e0 < E; e0 += 1024) {
    const int e = e0 + tid;
    const int all = e < E ? count[e] : 0;
    const int mine = static_cast<int>(min(static_cast<int64_t>(all), C));
    int rows, tiles, act;
    const int at = rows0 + block_prefix(mine, sums, &rows);
    const int tile = tiles0 + block_prefix((mine + bt - 1) / bt, sums, &tiles);
    const int place = act0 + block_prefix(mine > 0 ? 1 : 0, sums, &act);
    if (e < E) {
      if (routed) routed[e] = all;
      if (kept) kept[e] = mine;
      count[e] = at;
      ls.off[e] = at;
      ls.tile[e] = tile;
      if (mine > 0) ls.act[place] = e;
    }
    rows0 += rows;
    tiles0 += tiles;
    act0 += act;
  }
  if (tid == 0) {
    ls.off[E] = rows0;
    ls.tile[E] = tiles0;
    *ls.n_act = act0;
  }
}

__global__ __launch_bounds__(1024) void experts_plan_kernel(const int32_t* __restrict__ idx, int64_t T, int k, int E,
                                                            int64_t C, int bt, int32_t* __restrict__ slot,
                                                            int32_t* __restrict__ routed, int32_t* __restrict__ kept,
                                                            ExpertLists ls) {
  __shared__ int cc[kPlanCounts];
  __shared__ int cnt[4096];
  __shared__ int sums[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int W = min(16, kPlanCounts / E);  // at least 4
  const int64_t n = T * k;
  const int nbits = E > 1 ? 32 - __clz(E - 1) : 0;
  const unsigned long long below = (1ull << lane) - 1ull;
  for (int e = tid; e < E; e += 1024) cnt[e] = 0;
  for (int64_t c0 = 0; c0 < n; c0 += 64 * W) {
    for (int i = tid; i < W * E; i += 1024) cc[i] = 0;
    __syncthreads();
    const int64_t i = c0 + tid;
    int e = -1, r = 0;
    if (wave < W) {
      if (i < n) e = idx[i];
      if (e >= E) e = -1;
      unsigned long long mask = __ballot(e >= 0);
      for (int bit = 0; bit < nbits; ++bit) {
        const bool set = (e >> bit) & 1;
        const unsigned long long m = __ballot(e >= 0 && set);
        mask &= set ? m : ~m;
      }
      if (e >= 0) {
        r = __popcll(mask & below);
        if (r == 0) cc[wave * E + e] = __popcll(mask);
      }
    }
    __syncthreads();
    for (int x = tid; x < E; x += 1024) {
      int run = cnt[x];
      for (int w = 0; w < W; ++w) {
        const int c = cc[w * E + x];
        cc[w * E + x] = run;
        run += c;
      }
      cnt[x] = run;
    }
    __syncthreads();
    if (wave < W && i < n) {
      const int64_t rank = e >= 0 ? r + cc[wave * E + e] : C;
      slot[i] = rank < C ? static_cast<int32_t>(rank) : -1;
    }
    __syncthreads();
  }
  list_experts(cnt, E, C, bt, routed, kept, ls, sums);
  __syncthreads();
  // every thread places the copies whose slots it wrote
  for (int64_t c0 = 0; c0 < n; c0 += 64 * W) {
    const int64_t i = c0 + tid;
    if (wave < W && i < n) {
      const int s = slot[i];
      if (s >= 0) ls.copy[cnt[idx[i]] + s] = static_cast<int32_t>(i);
    }
  }
}

// The same for many copies, after the layer's histogram, scan and slots over tiles of
// tokens: the experts' lists from the kept counts, then the copies' places.
__global__ __launch_bounds__(1024) void list_experts_kernel(int32_t* kept, int E, int64_t C, int bt, ExpertLists ls) {
  __shared__ int cnt[4096];
  __shared__ int sums[16];
  for (int e = threadIdx.x; e < E; e += 1024) cnt[e] = kept[e];
  __syncthreads();
  list_experts(cnt, E, C, bt, nullptr, nullptr, ls, sums);
}

__global__ __launch_bounds__(256) void place_copies_kernel(const int32_t* __restrict__ idx,
                                                           const int32_t* __restrict__ slot, int64_t n, ExpertLists ls) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= n) return;
  const int s = slot[i];
  if (s >= 0) ls.copy[ls.off[idx[i]] + s] = static_cast<int32_t>(i);
}

// ---------------------------------------------------------------------------
// Few rows an expert: the weights' strips stream from memory into the operand
// registers. A work-group has a strip of 16 NA weight rows (GU: NA / 2 gate rows'
// tiles and the up rows' of the same features) and the 16 NT rows of x; its waves
// share the columns in turn, 128 at a time, and add their sums in LDS.
// An instruction's A operand is, in lane l, the bytes 16 (l / 16) .. + 15 and 64 +
// 16 (l / 16) .. + 15 of row l % 16's 128, its scale operand the byte of columns 32
// (l / 16) .. + 31. Rows are loaded in whole 128-byte lines, eight rows an
// instruction, and rotated into place (operands()).
// ---------------------------------------------------------------------------
// A range of memory for loads at an offset that is the same for all lanes plus a
// lane's own. A lane whose own offset is past the end gets 0 and touches nothing;
// the common offset is not checked, so what it adds must stay in the range.
struct Range {
  const void* base;
  uint32_t bytes;
  __device__ inline __amdgpu_buffer_rsrc_t rsrc() const {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(bytes),
                                             0x00020000);
  }
  template <bool ONCE>  // read once: not to be kept in the caches
  __device__ inline u32x4 load16(uint32_t lane_off, uint32_t off) const {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(rsrc(), static_cast<int>(lane_off), static_cast<int>(off), ONCE ? 2 : 0);
    return u32x4{static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[1]), static_cast<uint32_t>(v[2]), static_cast<uint32_t>(v[3])};
  }
  __device__ inline uint32_t load4(uint32_t lane_off, uint32_t off) const {
    return __builtin_amdgcn_raw_buffer_load_b32(rsrc(), static_cast<int>(lane_off), static_cast<int>(off), 0);
  }
};
constexpr uint32_t kNowhere = 0x80000000u;  // a lane's offset past every range

template <int NA, int NT>
struct FewStep {
  u32x4 lo[NA], hi[NA], x0[NT], x1[NT];
  uint32_t sa[NA], sx[NT];
};

template <bool GU, int NA, int NT, int WAVES>
__device__ inline void few_rows(const Mx8Gemm& a, int e, int row0, int n, int strip, float* red) {
  constexpr int FT = GU ? NA / 2 : NA;  // tiles of 16 output features
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = lane >> 4, half = (lane >> 3) & 1, col = lane & 15;
  const int K = static_cast<int>(a.K), N = static_cast<int>(a.N), steps = (K + 127) / 128, n0 = strip * 16 * FT;
  const uint32_t span = static_cast<uint32_t>(N) * K, sspan = static_cast<uint32_t>(steps) * N * 4;
  // Rows past the matrix are its last ones again (N is a multiple of 16): what becomes of their features is not stored.
  const Range w0 = {a.a0.codes + static_cast<int64_t>(e) * span, span}, w1 = {a.a1.codes + static_cast<int64_t>(e) * span, span};
  const Range s0 = {a.a0.scale + static_cast<int64_t>(e) * steps * N, sspan}, s1 = {a.a1.scale + static_cast<int64_t>(e) * steps * N, sspan};
  // x's rows: the tokens' (of all) with GU, else the lists' from row0 on
  const int64_t xbase = GU ? 0 : row0;
  const Range x = {a.x.codes + xbase * K, static_cast<uint32_t>((GU ? a.R : n) * K)};
  const Range xs = {a.x.scale, static_cast<uint32_t>(steps * a.R * 4)};
  const uint32_t wv = static_cast<uint32_t>(lane & 7) * K + 16 * (quad + 4 * half), sv = 4 * col;
  uint32_t xv[NT], xsv[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = row0 + min(16 * t + col, n - 1);  // columns past the last row are it again
    const uint32_t xr = GU ? a.ls.copy[r] / a.k : r;
    xv[t] = static_cast<uint32_t>(xr - xbase) * K + 16 * quad;
    xsv[t] = 4 * xr;
  }
  f32x4 acc[NA][NT];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  using Step = FewStep<NA, NT>;
  auto load = [&](Step& b, int s) {
    const uint32_t k0 = s * 128;
    const bool tail = k0 + 128 > static_cast<uint32_t>(K);
    const uint32_t ca = tail && k0 + 16 * (quad + 4 * half) >= static_cast<uint32_t>(K) ? kNowhere : wv;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int row = min(n0 + 16 * (i % FT), N - 16);
      const uint32_t at = static_cast<uint32_t>(row) * K + k0;
      const Range& w = GU && i >= FT ? w1 : w0;
      b.lo[i] = w.load16<true>(ca, at);
      b.hi[i] = w.load16<true>(ca, at + 8 * K);
      b.sa[i] = (GU && i >= FT ? s1 : s0).load4(sv, 4 * (s * N + row));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const bool no0 = tail && k0 + 16 * quad >= static_cast<uint32_t>(K), no1 = tail && k0 + 16 * quad + 64 >= static_cast<uint32_t>(K);
      b.x0[t] = x.load16<false>(no0 ? kNowhere : xv[t], k0);
      b.x1[t] = x.load16<false>(no1 ? kNowhere : xv[t], k0 + 64);
      b.sx[t] = xs.load4(xsv[t], static_cast<uint32_t>(s * a.R * 4));
    }
  };
  auto multiply = [&](const Step& b, int s) {
    const bool past = s * 128 + 32 * quad >= K;  // bytes of columns past the last may be anything
    i32x8 xx[NT];
    int sx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        xx[t][q] = static_cast<int>(b.x0[t][q]);
        xx[t][4 + q] = static_cast<int>(b.x1[t][q]);
      }
      sx[t] = past ? 127 : static_cast<int>(b.sx[t] >> (8 * quad));
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      u32x4 p, q;
      operands(b.lo[i], b.hi[i], p, q);
      i32x8 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = static_cast<int>(p[j]);
        w[4 + j] = static_cast<int>(q[j]);
      }
      const int sa = past ? 127 : static_cast<int>(b.sa[i] >> (8 * quad));
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[i][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, xx[t], acc[i][t], 0, 0, 0, sa, 0, sx[t]);
    }
  };
  // a step is asked for before the last one is multiplied
  if (wave < steps) {
    Step b0, b1;
    load(b0, wave);
    int s = wave;
    for (; s + WAVES < steps; s += 2 * WAVES) {
      load(b1, s + WAVES);
      __builtin_amdgcn_sched_barrier(0);
      multiply(b0, s);
      load(b0, min(s + 2 * WAVES, steps - 1));
      __builtin_amdgcn_sched_barrier(0);
      multiply(b1, s + WAVES);
    }
    if (s < steps) multiply(b0, s);
  }
  // the waves' sums, in their order: wave t has token tile t
  f32x4* mine = reinterpret_cast<f32x4*>(red);
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) mine[((wave * NT + t) * NA + i) * 64 + lane] = acc[i][t];
  __syncthreads();
  static_assert(WAVES >= NT, "a wave a token tile");
  if (wave < NT) {
    f32x4 v[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      v[i] = mine[(wave * NA + i) * 64 + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v[i] += mine[((w * NT + wave) * NA + i) * 64 + lane];
    }
    const int c = 16 * wave + col;  // the row, of n
    if constexpr (GU) {
      static_assert(FT == 2, "a strip is the 32 features of a scale");
      uint32_t big = 0;
      f32x4 h[FT];
#pragma unroll
      for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h[i][q] = n0 + 16 * i + 4 * quad + q < a.N ? silu(v[i][q]) * v[FT + i][q] : 0.f;
          big = max(big, __float_as_uint(h[i][q]) & 0x7fffffffu);
        }
      big = max(big, static_cast<uint32_t>(__shfl_xor(big, 16, 64)));
      big = max(big, static_cast<uint32_t>(__shfl_xor(big, 32, 64)));
      const uint32_t byte = mx8_scale_byte(big);
      const float inv = mx8_inverse(byte);
      if (c < n) {
        const int64_t r = row0 + c;
        if (quad == 0) a.hscale[mx8_scale_at(n0 / 128, a.H, r) * 4 + n0 / 32 % 4] = static_cast<uint8_t>(byte);
#pragma unroll
        for (int i = 0; i < FT; ++i)
          if (n0 + 16 * i < a.N)
            *reinterpret_cast<uint32_t*>(a.hcodes + r * a.N + n0 + 16 * i + 4 * quad) =
                mx8_codes(h[i][0] * inv, h[i][1] * inv, h[i][2] * inv, h[i][3] * inv);
      }
    } else if (c < n) {
      const int64_t r = a.ls.copy[row0 + c];
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int64_t f = n0 + 16 * i + 4 * quad;
        if (f >= a.N) continue;
        *reinterpret_cast<f32x4*>(a.y + r * a.N + f) = v[i];
      }
    }
  }
  __syncthreads();  // the sums are read before the next rows' are written
}

// Up to 32 rows at a time; an expert with more has its weights read again. Bound by
// memory: one token of a DeepSeek-V3-shaped layer (d = 7168, d_ff = 2048, 8 experts)
// 40.5 us for gate and up (242 MB, 6.0 TB/s) and 23.5 for down, 64 tokens 1.03 ms
// (6.7 GB, 6.6 TB/s) and 0.55. With eight waves a work-group gate and up took 42 us
// and 1.06 ms (d_ff = 1408, 24 copies: 28 us instead of 21).
template <bool GU, int NA, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void few_rows_kernel(Mx8Gemm a, int strips) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass has no scaled matrix instruction
  __shared__ float red[WAVES * 2 * NA * 64 * 4];
  const int i = static_cast<int>(blockIdx.x / strips);
  if (i >= *a.ls.n_act) return;
  const int e = __builtin_amdgcn_readfirstlane(a.ls.act[i]);
  const int strip = blockIdx.x % strips;
  const int end = __builtin_amdgcn_readfirstlane(a.ls.off[e + 1]);
  for (int r = __builtin_amdgcn_readfirstlane(a.ls.off[e]); r < end; r += 32) {
    const int n = min(end - r, 32);
    if (n <= 16)
      few_rows<GU, NA, 1, WAVES>(a, e, r, n, strip, red);
    else
      few_rows<GU, NA, 2, WAVES>(a, e, r, n, strip, red);
  }
#endif
}

// out[t] = residual[t] + sum_j w y[t, j] over the kept copies, j ascending, in
// fp32; a token without a kept copy passes bit for bit.
// y comes in fp32: in bf16 its rounding adds to out's own as much as all else does
// (64 tokens, DeepSeek-V3-shaped: 1.84e-3 against 64 bits instead of 1.75e-3, of which
// out's rounding is 1.66e-3). Twice the bytes of y cost nothing there, and 1.1% on 4096
// Mixtral-shaped tokens (1542 -> 1559 us), 6% on 8192 DeepSeek-V3-shaped ones (4430 ->
// 4690 us).
template <bool BF16>
__global__ __launch_bounds__(256) void experts_combine_kernel(const uint4* residual, const uint4* __restrict__ y,
                                                              const float* __restrict__ w,
                                                              const int32_t* __restrict__ slot, int k, int64_t V,
                                                              int64_t blocks, uint4* out) {  // out may be residual
  constexpr int P = BF16 ? 8 : 4;
  const int64_t t = blockIdx.x / blocks, v = blockIdx.x % blocks * 256 + threadIdx.x;
  if (v >= V) return;
  const uint4 in = load_stream(residual + t * V + v);
  float acc[P];
#pragma unroll
  for (int i = 0; i < P; ++i) acc[i] = 0.f;
  bool any = false;
  for (int j = 0; j < k; ++j) {
    if (slot[t * k + j] < 0) continue;
    any = true;
    const uint4* row = y + ((t * k + j) * V + v) * (P / 4);
    uint4 word[P / 4];
#pragma unroll
    for (int h = 0; h < P / 4; ++h) word[h] = load_stream(row + h);
    const float g = w[t * k + j];
#pragma unroll
    for (int h = 0; h < P / 4; ++h) {
      const uint32_t u[4] = {word[h].x, word[h].y, word[h].z, word[h].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[4 * h + q] = fmaf(g, __uint_as_float(u[q]), acc[4 * h + q]);
    }
  }
  uint32_t u[4] = {in.x, in.y, in.z, in.w};
  if (any) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if constexpr (BF16)
        u[q] = f32_to_bf16(__uint_as_float(u[q] << 16) + acc[2 * q]) |
               static_cast<uint32_t>(f32_to_bf16(__uint_as_float(u[q] & 0xffff0000u) + acc[2 * q + 1])) << 16;
      else
        u[q] = __float_as_uint(__uint_as_float(u[q]) + acc[q]);
  }
  store_stream(out + t * V + v, uint4{u[0], u[1], u[2], u[3]});
}

Mx8 view(const Mx8Ptr& p) { return {p.codes, p.scale}; }

}  // namespace

hipError_t launch_experts_mx8(const ExpertsMx8& L, hipStream_t s) {
  const int64_t copies = L.T * L.k, act = std::min<int64_t>(L.E, copies);
  const int tile_rows = mx8_tile_rows(copies, act);
  hipError_t e = hipSuccess;
  if (copies <= kPlanCopies) {
    experts_plan_kernel<<<dim3(1), dim3(1024), 0, s>>>(L.idx, L.T, L.k, L.E, L.C, tile_rows, L.slot, L.routed, L.kept, L.ls);
  } else {
    if ((e = launch_tile_hist(L.idx, L.T, L.k, L.E, L.tile_cnt, s, L.slot)) != hipSuccess ||
        (e = launch_scan(L.tile_cnt, ceil_div(L.T, kTileTokens), L.E, L.C, 1, 0, L.k, L.T, L.tile_off, L.routed, L.kept,
                         nullptr, nullptr, 0, nullptr, nullptr, s)) != hipSuccess ||
        (e = launch_slots_from_ranks(L.idx, L.slot, L.tile_off, L.T, L.k, L.E, L.C, nullptr, nullptr, s)) != hipSuccess)
      return e;
    list_experts_kernel<<<dim3(1), dim3(1024), 0, s>>>(L.kept, L.E, L.C, tile_rows, L.ls);
    place_copies_kernel<<<dim3(static_cast<unsigned>(ceil_div(copies, 256))), dim3(256), 0, s>>>(L.idx, L.slot, copies, L.ls);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  Mx8Gemm a;
  a.a0 = view(L.gate);
  a.a1 = view(L.up);
  a.N = L.f;
  a.K = L.d;
  a.x = view(L.x);
  a.R = L.T;
  a.ls = L.ls;
  a.k = L.k;
  a.hcodes = L.h.codes;
  a.hscale = reinterpret_cast<uint8_t*>(L.h.scale);
  a.H = copies;
  a.y = nullptr;
  a.parts = nullptr;
  const bool many = mx8_many(copies, act);
  const int64_t tiles = copies / tile_rows + act;
  auto few = [&](auto gu, const Mx8Gemm& g) {
    constexpr bool GU = decltype(gu)::value;
    const int strips = static_cast<int>(ceil_div(g.N, 32));
    few_rows_kernel<GU, GU ? 4 : 2, 4><<<dim3(static_cast<unsigned>(act * strips)), dim3(256), 0, s>>>(g, strips);
    return hipGetLastError();
  };
  e = many ? launch_mx8_tiles(a, true, L.E, tiles, tile_rows, s) : few(std::true_type{}, a);
  if (e != hipSuccess) return e;
  Mx8Gemm b = a;
  b.a0 = b.a1 = view(L.down);
  b.N = L.d;
  b.K = L.f;
  b.x = view(L.h);
  b.R = copies;
  b.y = L.y;
  b.parts = L.parts;
  e = many ? launch_mx8_tiles(b, false, L.E, tiles, tile_rows, s) : few(std::false_type{}, b);
  if (e != hipSuccess) return e;
  const int64_t V = L.d / (L.bf16 ? 8 : 4), blocks = ceil_div(V, 256);
  const dim3 grid(static_cast<unsigned>(L.T * blocks));
  const auto* rv = static_cast<const uint4*>(L.residual);
  const auto* yv = reinterpret_cast<const uint4*>(L.y);
  if (L.bf16)
    experts_combine_kernel<true><<<grid, dim3(256), 0, s>>>(rv, yv, L.w, L.slot, L.k, V, blocks, static_cast<uint4*>(L.out));
  else
    experts_combine_kernel<false><<<grid, dim3(256), 0, s>>>(rv, yv, L.w, L.slot, L.k, V, blocks, static_cast<uint4*>(L.out));
  return hipGetLastError();
}

}  // namespace moe
