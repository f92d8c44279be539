// The experts' products with 8-bit rows and weights where an expert has many rows
// (gfx950): blocks of 256 weight rows by 256 (or 128) rows of x, brought into LDS by
// the buffer unit, two (three) stages of 128 columns: a row's stage is a 128-byte line.
//
// As in mx8_experts.hip the weights are the A operand: lane l of a 32 x 32 x 64
// instruction holds, of row l % 32, the bytes 16 (l / 32) .. + 15 and 32 + 16 (l /
// 32) .. + 15 of 64 columns, and the scale byte of columns 32 (l / 32) .. + 31; its
// accumulator element q is feature 8 (q / 4) + 4 (l / 32) + q % 4 of row l % 32 of x.
// With gate and up a wave has the gate rows' and the up rows' tiles of the same
// features, so silu(g) u, the scale of 32 features and the codes stay in its lanes.
//
// LDS rows are eight 16-byte pieces; piece c of row r sits at c ^ ((r / 2) % 8), so
// that 16 lanes reading 16 neighbouring rows meet 16 bank groups. One DMA
// instruction of a wave fills 8 rows: lane L writes row L / 8, position L % 8,
// and fetches the piece that belongs there.
#include "mx8_experts.h"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace moe {
namespace {

#define MOE_LDS(p) ((__attribute__((address_space(3))) void*)(p))

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), static_cast<int>(bytes),
                                           0x00020000);
}

// s_waitcnt: this wave's loads but the last VM of them, and its LDS reads.
template <int VM>
__device__ inline void wait_loads() {
  static_assert(VM < 64, "vmcnt has six bits");
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | (0 << 8) | ((VM >> 4) << 14));
}

// A stage half's schedule: NM products with NR reads of LDS and NV loads spread
// among them. Left to itself the compiler reads an operand right before its
// product and waits.
template <int I, int NM, int NR, int NV>
__device__ inline void interleave_one() {
  constexpr int R = NR * (I + 1) / NM - NR * I / NM, V = NV * (I + 1) / NM - NV * I / NM;
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  if constexpr (R > 0) __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
  if constexpr (V > 0) __builtin_amdgcn_sched_group_barrier(0x020, V, 0);
}
template <int NM, int NR, int NV, int... I>
__device__ inline void interleave_all(std::integer_sequence<int, I...>) {
  (interleave_one<I, NM, NR, NV>(), ...);
}
template <int NM, int NR, int NV>
__device__ inline void interleave() {
  interleave_all<NM, NR, NV>(std::make_integer_sequence<int, NM>{});
}

constexpr int kFeatureGroup = 8;  // feature tiles that go through an expert's row tiles together (shared in L2)

// XCD x takes the x-th contiguous eighth of the live tiles. Its units take 32 of them
// at a time (a block has a unit's LDS to itself), and the rest of them leaves units
// idle for a whole tile: with many columns each of the rest is split over K between
// `parts` blocks, which leave fp32 sums for join_parts_kernel. In turn on one card,
// d = 4096, d_ff = 14336, 2 of 8 experts: 4096 tokens (72 tiles an XCD, the last 8 in
// four parts) 1700 -> 1610 us in all, 512 tokens 471 -> 425; with tiles of 128 rows
// 256 tokens (16 tiles an XCD in two parts) 410 -> 363, 128 tokens 397 -> 347.
struct Split {
  int64_t per, whole;  // tiles of an XCD; those before `whole` are not split
  int parts;
};
constexpr int kUnits = 32;       // of an XCD
constexpr int kPartFloats = 256 * 256;  // or half of them

// A part has 16 stages of 128 columns or more, and is 32 shorter than the tile at
// least (60 us; what it writes and what the join reads take 20 to 25).
__host__ __device__ inline Split split_of(int64_t live, int64_t steps) {
  Split s{(live + 7) / 8, (live + 7) / 8, 1};
  const int64_t rest = s.per % kUnits;
  if (rest == 0) return s;
  const int64_t parts = kUnits / rest < steps / 16 ? kUnits / rest : steps / 16;
  if (parts < 2 || steps - (steps + parts - 1) / parts < 32) return s;
  s.whole = s.per - rest;
  s.parts = static_cast<int>(parts);
  return s;
}

struct Tile {
  int e, row0, rows;  // rows of the expert's list
  int64_t n0;
};

__device__ inline int64_t live_tiles(const ExpertLists& ls, int E, int feature_tile, int64_t N) {
  return static_cast<int64_t>(ls.tile[E]) * ((N + feature_tile - 1) / feature_tile);
}

__device__ inline bool tile_at(const ExpertLists& ls, int E, int feature_tile, int64_t N, int64_t id, Tile* t) {
  const int ft = static_cast<int>((N + feature_tile - 1) / feature_tile);
  if (id >= static_cast<int64_t>(ls.tile[E]) * ft) return false;
  const int rt = static_cast<int>(id / ft);
  int lo = 0, hi = E;  // tile[lo] <= rt < tile[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ls.tile[mid] <= rt)
      lo = mid;
    else
      hi = mid;
  }
  const int first = ls.tile[lo], n = ls.tile[lo + 1] - first;
  const int64_t in = id - static_cast<int64_t>(first) * ft;
  const int64_t group = in / (static_cast<int64_t>(n) * kFeatureGroup);
  const int wide = static_cast<int>(min(static_cast<int64_t>(kFeatureGroup), ft - group * kFeatureGroup));
  const int rest = static_cast<int>(in - group * n * kFeatureGroup);
  t->e = lo;
  t->n0 = (group * kFeatureGroup + rest % wide) * feature_tile;
  // the expert's rows are shared evenly by its tiles, in whole blocks of 32
  const int all = ls.off[lo + 1] - ls.off[lo], each = 32 * ((all + 32 * n - 1) / (32 * n));
  t->row0 = rest / wide * each;
  t->rows = min(all - t->row0, each);
  return true;
}

// WM x WN waves of TM x TN tiles of 32 x 32, NS slots for stages: 2 x 2 of 4 x 4 and
// two slots, or of 4 x 2 and three. The former's stage is 32 products
// a wave (2048 clocks), 128 KiB of LDS read and 66 written, and takes 1.9 us where
// the products alone take 1.0 at the clock that they leave (4.25 PFLOP/s in
// registers; the library's product of 16384^3 reaches 3.27). One wave a SIMD: its
// waits for loads, LDS and the stages' barriers are filled by nothing (the matrix
// cores are busy 52 - 54% of the time). Mixtral-shaped, 4096 tokens: gate and up 1.06
// - 1.17 ms (1.92 TFLOP: 1.65 - 1.82 PFLOP/s), down 0.55 - 0.57 and 0.017 for the join
// of its split tiles (some 0.65 without the split).
// Measured and dropped: 2 x 4 waves of 4 x 2 tiles (256 registers do not hold them:
// twice the time), 128 features a block (down 0.81 ms), a word of each weight line
// asked for two stages before (down 0.61 ms, but 64 rows an expert 12% more).
template <bool GU, int WM, int WN, int TM, int TN, int NS>
__global__ __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(WM* WN / 4, WM* WN / 4))) void mx8_tile_kernel(
    Mx8Gemm a, int E) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass has no scaled matrix instruction and would drop the kernel without a word
  constexpr int NW = WM * WN, MA = WM * TM * 32, MX = WN * TN * 32;
  constexpr int FW = (GU ? TM / 2 : TM) * 32;          // features of a wave
  constexpr int FB = WM * FW;                          // and of the block
  constexpr int PA = MA / 8 / NW, PX = MX / 8 / NW;    // 8-row DMA pieces of a wave
  constexpr int SETS = (MA + MX) / 64, PS = (SETS + NW - 1) / NW;  // sets of 64 scales, and a wave's
  static_assert(NS == 2 || NS == 3, "two or three slots");
  constexpr int THIRD = NS == 3;
  // a slot's arrays each by themselves, so that the compiler tells the stages apart
  __shared__ uint4 As0[MA * 8], As1[MA * 8], As2[THIRD ? MA * 8 : 1], Xs0[MX * 8], Xs1[MX * 8], Xs2[THIRD ? MX * 8 : 1];
  __shared__ uint32_t Sc0[MA + MX], Sc1[MA + MX], Sc2[THIRD ? MA + MX : 1];

  constexpr bool SPLIT = !GU;
  const int64_t xcd = blockIdx.x % 8, all_steps = ceil_div(a.K, 128), live_all = live_tiles(a.ls, E, FB, a.N);
  int64_t at = blockIdx.x / 8, first_step = 0, end_step = all_steps;
  int part_slot = -1;
  Split sp{(live_all + 7) / 8, (live_all + 7) / 8, 1};
  if constexpr (SPLIT) {
    if (a.parts) sp = split_of(live_all, all_steps);
    if (at >= sp.whole && sp.parts > 1) {
      const int64_t o = at - sp.whole, p = o % sp.parts;
      if (o >= (sp.per - sp.whole) * sp.parts) return;
      at = sp.whole + o / sp.parts;
      part_slot = __builtin_amdgcn_readfirstlane(static_cast<int>(xcd * kUnits + o));
      first_step = __builtin_amdgcn_readfirstlane(static_cast<int>(all_steps * p / sp.parts));
      end_step = __builtin_amdgcn_readfirstlane(static_cast<int>(all_steps * (p + 1) / sp.parts));
    }
  }
  Tile tl;
  if (at >= sp.per || !tile_at(a.ls, E, FB, a.N, xcd * sp.per + at, &tl)) return;
  const int e = __builtin_amdgcn_readfirstlane(tl.e);
  const int rows = __builtin_amdgcn_readfirstlane(tl.rows);
  const int first = __builtin_amdgcn_readfirstlane(a.ls.off[e] + tl.row0);  // row of the lists
  const int64_t n0 = __builtin_amdgcn_readfirstlane(static_cast<int>(tl.n0));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, lr = lane & 31, lq = lane >> 5;
  const int64_t K = a.K, N = a.N, steps = end_step - first_step;  // stages are counted from the block's first

  // Row r of the block's A operand is this feature of this matrix. Past the matrix its last 16 rows stand in (N is a
  // multiple of 16, so eight rows that are loaded together are all in it or all past it): a load's common offset is
  // not checked against the buffer's size, and what becomes of those features is not stored.
  auto feature = [&](int r) {
    const int64_t f = n0 + r / (TM * 32) * FW + (GU ? r / 32 % TM % (TM / 2) : r / 32 % TM) * 32 + (r & 31);
    return f < N ? f : N - 16 + (r & 15);
  };
  auto is_up = [&](int r) { return GU && r / 32 % TM >= TM / 2; };
  const int64_t span = N * K;
  const auto ra0 = rsrc(a.a0.codes + e * span, span), ra1 = rsrc(a.a1.codes + e * span, span);
  // GU reads the tokens' rows (all of x), else the lists' rows from the tile's first
  const int64_t xbase = GU ? 0 : first, xrows = GU ? a.R : rows;
  const auto rx = rsrc(a.x.codes + xbase * K, xrows * K);
  auto x_row = [&](int r) {
    const int at = first + min(r, rows - 1);  // past the last row: it again
    return GU ? static_cast<int64_t>(a.ls.copy[at] / a.k) : static_cast<int64_t>(at);
  };
  // the piece at this lane's position of the 8 rows of an even or odd DMA instruction, in bytes of the row's 128
  const int piece[2] = {16 * ((lane & 7) ^ (lane >> 4)), 16 * ((lane & 7) ^ (4 + (lane >> 4)))};
  const uint32_t va = static_cast<uint32_t>((lane >> 3) * K);
  uint32_t vx[PX];
#pragma unroll
  for (int i = 0; i < PX; ++i)
    vx[i] = static_cast<uint32_t>((x_row((wave * PX + i) * 8 + (lane >> 3)) - xbase) * K + piece[i & 1]);
  static_assert(PA % 2 == 0 && PX % 2 == 0, "a wave's DMA instructions begin with an even one");
  // the scales: rows 64 (PS wave + i) + lane of A's (of one matrix: TM % 4 == 0), then of x's
  static_assert(!GU || TM % 4 == 0, "64 rows of A are of one matrix");
  const int64_t sbytes = all_steps * N * 4;
  const auto rs0 = rsrc(a.a0.scale + e * all_steps * N, sbytes), rs1 = rsrc(a.a1.scale + e * all_steps * N, sbytes);
  const auto rsx = rsrc(a.x.scale, all_steps * a.R * 4);
  uint32_t vs[PS];
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    const int r = min(wave * PS + i, SETS - 1) * 64;  // the last set may be loaded twice, with the same
    vs[i] = static_cast<uint32_t>(4 * (r < MA ? feature(r + lane) : x_row(r + lane - MA)));
  }
  auto dma = [&](uint4* as, uint4* xs, uint32_t* sc, int64_t s) {
    s += first_step;
    const int k0 = static_cast<int>(s * 128);
    // pieces past the last column: zero (an offset past the buffer)
    const bool in[2] = {k0 + piece[0] < K, k0 + piece[1] < K};
    const uint32_t v[2] = {in[0] ? va + piece[0] : 0x80000000u, in[1] ? va + piece[1] : 0x80000000u};
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int r = (wave * PA + i) * 8;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_up(r) ? ra1 : ra0, MOE_LDS(as + r * 8), 16, v[i & 1],
                                               static_cast<int>(feature(r) * K) + k0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PX; ++i) {
      const int r = (wave * PX + i) * 8;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, MOE_LDS(xs + r * 8), 16, in[i & 1] ? vx[i] : 0x80000000u, k0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      const int r = min(wave * PS + i, SETS - 1) * 64;
      const int soff = static_cast<int>(s * (r < MA ? N : a.R) * 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r >= MA ? rsx : is_up(r) ? rs1 : rs0, MOE_LDS(sc + r), 4, vs[i], soff, 0, 0);
    }
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // a wave multiplies the 32-row blocks of x that have rows
  const int left = rows - wn * TN * 32;
  const int live = __builtin_amdgcn_readfirstlane(left <= 0 ? 0 : min(TN, (left + 31) / 32));
  const int sw = (lr >> 1) & 7;
  auto loop = [&](auto live_c) {
    constexpr int TX = decltype(live_c)::value;
    i32x8 fa[2][TM], fx[2][TN];
    uint32_t sa[TM], sx[TN];
    auto read = [&](const uint4* base, int row, int h) {
      const uint4* p = base + row * 8;
      const uint4 lo = p[(4 * h + lq) ^ sw], hi = p[(4 * h + 2 + lq) ^ sw];
      return i32x8{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
                   static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
    };
    auto fload = [&](const uint4* as, const uint4* xs, int h, int slot) {
      if constexpr (TX > 0) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[slot][i] = read(as, (wm * TM + i) * 32 + lr, h);
#pragma unroll
        for (int j = 0; j < TX; ++j) fx[slot][j] = read(xs, (wn * TN + j) * 32 + lr, h);
      }
    };
    // the stage's scales as they lie, and made ready: byte 0 of an operand is that of the first 64 columns' block lq,
    // byte 2 of the second's
    uint32_t ra[TM], rx_[TN];
    auto sload = [&](const uint32_t* sc) {
      if constexpr (TX > 0) {
#pragma unroll
        for (int i = 0; i < TM; ++i) ra[i] = sc[(wm * TM + i) * 32 + lr];
#pragma unroll
        for (int j = 0; j < TX; ++j) rx_[j] = sc[MA + (wn * TN + j) * 32 + lr];
      }
    };
    auto sready = [&](int64_t s) {
      if constexpr (TX > 0) {
        const int64_t groups = ceil_div(K - (first_step + s) * 128, 32);  // with columns; bytes past them may be anything
        const uint32_t mask = groups >= 4 ? ~0u : (1u << (8 * groups)) - 1;
        auto fix = [&](uint32_t v) { return ((v & mask) | (0x7f7f7f7fu & ~mask)) >> (8 * lq); };
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = fix(ra[i]);
#pragma unroll
        for (int j = 0; j < TX; ++j) sx[j] = fix(rx_[j]);
      }
    };
    auto multiply = [&](auto half) {
      constexpr int H = decltype(half)::value;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TX; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[H][i], fx[H][j], acc[i][j], 0, 0, 2 * H,
                                                                     static_cast<int>(sa[i]), 2 * H, static_cast<int>(sx[j]));
    };
    using Half0 = std::integral_constant<int, 0>;
    using Half1 = std::integral_constant<int, 1>;
    // Stage s is in (as, xs, sc), its first half's operands in slot 0 of the registers; the stages after it are on
    // their way into the other slots. Half way through, stage s + 1 has landed (of the loads under way the last `later`
    // may be out), and stage s + NS is asked for in this one's place.
    // What follows a stage is known here: a branch around the matrix work instead made the compiler keep the
    // accumulators twice.
    constexpr int LOADS = PA + PX + PS;
    auto stage = [&](auto next, auto refill, auto later, uint4* as, uint4* xs, uint32_t* sc, uint4* an, uint4* xn,
                     uint32_t* sn, int64_t s) {
      constexpr int READS = 2 * (TM + TX), PRODUCTS = TM * TX;
      fload(as, xs, 1, 1);
      multiply(Half0{});
      if constexpr (TX > 0) interleave<PRODUCTS, READS, 0>();
      if constexpr (decltype(next)::value) {
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<decltype(later)::value>();  // own share of stage s + 1 landed, reads of stage s done ...
        __builtin_amdgcn_s_barrier();          // ... and everyone's
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(refill)::value) dma(as, xs, sc, s + NS);
        fload(an, xn, 0, 0);
        sload(sn);
      }
      multiply(Half1{});
      if constexpr (TX > 0 && decltype(next)::value)
        interleave<PRODUCTS, READS + TM + TX, decltype(refill)::value ? LOADS : 0>();
      if constexpr (decltype(next)::value) sready(s + 1);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    using None = std::integral_constant<int, 0>;
    using Later = std::integral_constant<int, (NS - 2) * LOADS>;
    int64_t s = 0;
    for (; s < steps % NS; ++s) {  // what does not fill all slots: one stage after the other
      dma(As0, Xs0, Sc0, s);
      wait_loads<0>();
      __builtin_amdgcn_s_barrier();
      fload(As0, Xs0, 0, 0);
      sload(Sc0);
      sready(s);
      stage(No{}, No{}, None{}, As0, Xs0, Sc0, As1, Xs1, Sc1, s);
      wait_loads<0>();
      __builtin_amdgcn_s_barrier();
    }
    if (s < steps) {
      dma(As0, Xs0, Sc0, s);
      dma(As1, Xs1, Sc1, s + 1);
      if constexpr (NS == 3) dma(As2, Xs2, Sc2, s + 2);
      wait_loads<(NS - 1) * LOADS>();
      __builtin_amdgcn_s_barrier();
      fload(As0, Xs0, 0, 0);
      sload(Sc0);
      sready(s);
      if constexpr (NS == 2) {
        for (; s + 2 < steps; s += 2) {
          stage(Yes{}, Yes{}, Later{}, As0, Xs0, Sc0, As1, Xs1, Sc1, s);
          stage(Yes{}, Yes{}, Later{}, As1, Xs1, Sc1, As0, Xs0, Sc0, s + 1);
        }
        stage(Yes{}, No{}, None{}, As0, Xs0, Sc0, As1, Xs1, Sc1, s);
        stage(No{}, No{}, None{}, As1, Xs1, Sc1, As0, Xs0, Sc0, s + 1);
      } else {
        for (; s + 3 < steps; s += 3) {
          stage(Yes{}, Yes{}, Later{}, As0, Xs0, Sc0, As1, Xs1, Sc1, s);
          stage(Yes{}, Yes{}, Later{}, As1, Xs1, Sc1, As2, Xs2, Sc2, s + 1);
          stage(Yes{}, Yes{}, Later{}, As2, Xs2, Sc2, As0, Xs0, Sc0, s + 2);
        }
        stage(Yes{}, No{}, Later{}, As0, Xs0, Sc0, As1, Xs1, Sc1, s);
        stage(Yes{}, No{}, None{}, As1, Xs1, Sc1, As2, Xs2, Sc2, s + 1);
        stage(No{}, No{}, None{}, As2, Xs2, Sc2, As0, Xs0, Sc0, s + 2);
      }
    }
  };
  if (live == TN)
    loop(std::integral_constant<int, TN>{});
  else if (TN > 2 && live > TN / 2)
    loop(std::integral_constant<int, TN>{});
  else if (live > 0)
    loop(std::integral_constant<int, (TN + 1) / 2>{});
  else
    loop(std::integral_constant<int, 0>{});

  if constexpr (SPLIT)
    if (part_slot >= 0) {
      f32x4* p = reinterpret_cast<f32x4*>(a.parts + static_cast<int64_t>(part_slot) * kPartFloats) + wave * TM * TN * 256 + lane;
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if ((wn * TN + j) * 32 < rows)
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
              p[((i * TN + j) * 4 + g) * 64] = f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
      return;
    }
  const int64_t nw = n0 + wm * FW;  // the wave's first feature
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int c = (wn * TN + j) * 32 + lr;  // the row, of `rows`
    if constexpr (GU) {
      const int64_t r = first + c;
#pragma unroll
      for (int i = 0; i < TM / 2; ++i) {
        const int64_t f0 = nw + 32 * i;
        float h[16];
        uint32_t big = 0;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          h[q] = f0 + 8 * (q / 4) + 4 * lq + q % 4 < N ? silu(acc[i][j][q]) * acc[i + TM / 2][j][q] : 0.f;
          big = max(big, __float_as_uint(h[q]) & 0x7fffffffu);
        }
        big = max(big, static_cast<uint32_t>(__shfl_xor(big, 32, 64)));
        const uint32_t byte = mx8_scale_byte(big);
        const float inv = mx8_inverse(byte);
        uint32_t w[4];  // words 0, 2, 4, 6 (lanes 0 - 31) or 1, 3, 5, 7 of the 32 codes
#pragma unroll
        for (int g = 0; g < 4; ++g)
          w[g] = mx8_codes(h[4 * g] * inv, h[4 * g + 1] * inv, h[4 * g + 2] * inv, h[4 * g + 3] * inv);
        // the halves exchange two words each and have 16 codes in a row
        const uint32_t o0 = __shfl_xor(lq ? w[0] : w[2], 32, 64), o1 = __shfl_xor(lq ? w[1] : w[3], 32, 64);
        const uint4 out = lq ? uint4{o0, w[2], o1, w[3]} : uint4{w[0], o0, w[1], o1};
        if (c < rows && f0 + 16 * lq < N) {
          *reinterpret_cast<uint4*>(a.hcodes + r * N + f0 + 16 * lq) = out;
          if (lq == 0) a.hscale[mx8_scale_at(f0 / 128, a.H, r) * 4 + f0 / 32 % 4] = static_cast<uint8_t>(byte);
        }
      }
    } else {
      const int64_t r = c < rows ? a.ls.copy[first + c] : 0;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int64_t f0 = nw + 32 * i;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int64_t f = f0 + 8 * g + 4 * lq;
          if (c < rows && f < N)
            *reinterpret_cast<f32x4*>(a.y + r * N + f) =
                f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        }
      }
    }
  }
#endif
}

// The split tiles' rows of y: their parts' sums, in order. A block takes a sixteenth
// of 256 rows' tile, on the XCD whose L2 has the parts. TN: 32-row blocks of a wave.
template <int TN>
__global__ __launch_bounds__(256) void join_parts_kernel(Mx8Gemm a, int E) {
  static_assert(TN == 2 || TN == 4, "tiles of 128 or 256 rows");
  constexpr int CHUNKS = 4 * TN;
  const int64_t xcd = blockIdx.x % 8, r = blockIdx.x / 8 / CHUNKS, chunk = blockIdx.x / 8 % CHUNKS;
  const Split sp = split_of(live_tiles(a.ls, E, 256, a.N), ceil_div(a.K, 128));
  Tile tl;
  if (sp.parts < 2 || r >= sp.per - sp.whole || !tile_at(a.ls, E, 256, a.N, xcd * sp.per + sp.whole + r, &tl)) return;
  const f32x4* parts = reinterpret_cast<const f32x4*>(a.parts + (xcd * kUnits + r * sp.parts) * kPartFloats);
  const int first = a.ls.off[tl.e] + tl.row0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // as the product's waves (two by two of 4 x TN tiles) left them
    const int v = static_cast<int>(chunk * 1024) + q * 256 + threadIdx.x;
    const int lane = v & 63, g = v >> 6 & 3, j = v / 256 % TN, i = v / (256 * TN) % 4, wave = v / (1024 * TN);
    const int c = ((wave & 1) * TN + j) * 32 + (lane & 31);
    const int64_t f = tl.n0 + (wave >> 1) * 128 + 32 * i + 8 * g + 4 * (lane >> 5);
    if (c >= tl.rows || f >= a.N) continue;
    f32x4 sum = parts[v];
    for (int p = 1; p < sp.parts; ++p) sum += parts[static_cast<int64_t>(p) * (kPartFloats / 4) + v];
    const int64_t at = static_cast<int64_t>(a.ls.copy[first + c]) * a.N + f;
    *reinterpret_cast<f32x4*>(a.y + at) = sum;
  }
}

template <bool GU, int WM, int WN, int TM, int TN, int NS>
hipError_t launch(const Mx8Gemm& a, int E, int64_t tiles, hipStream_t s) {
  const int64_t ft = ceil_div(a.N, WM * (GU ? TM / 2 : TM) * 32);
  const dim3 grid(static_cast<unsigned>((ceil_div(tiles * ft, 8) + (a.parts ? kUnits : 0)) * 8));
  mx8_tile_kernel<GU, WM, WN, TM, TN, NS><<<grid, dim3(WM * WN * 64), 0, s>>>(a, E);
  return hipGetLastError();
}

}  // namespace

// With few rows an expert the weights' way from memory bounds the products, and what
// counts is how much of it is asked for at once: 128 rows leave room for three
// slots, two stages under way (the same weights: 64 rows an expert of d = 7168,
// d_ff = 2048 2.8 ms instead of 3.0, 32 rows 2.6 instead of 3.0; 96 rows of d = 4096,
// d_ff = 14336 437 us instead of 491, 128 rows, which half the experts exceed, 537
// instead of 497; all before down's tiles were split).
int mx8_tile_rows(int64_t copies, int64_t experts) { return copies > 96 * experts ? 256 : 128; }

int64_t mx8_parts_bytes(int64_t copies, int64_t experts, int64_t K) {
  const int64_t steps = ceil_div(K, 128);
  bool any = false;  // with some number of tiles
  for (int rest = 1; rest <= kUnits; ++rest) any = any || split_of(8 * rest, steps).parts > 1;
  return any && mx8_many(copies, experts) ? int64_t{8} * kUnits * kPartFloats * 4 : 0;
}

hipError_t launch_mx8_tiles(const Mx8Gemm& a, bool gate_up, int E, int64_t tiles, int tile_rows, hipStream_t s) {
  const bool tall = tile_rows == 256;
  if (gate_up) return tall ? launch<true, 2, 2, 4, 4, 2>(a, E, tiles, s) : launch<true, 2, 2, 4, 2, 3>(a, E, tiles, s);
  const hipError_t e = tall ? launch<false, 2, 2, 4, 4, 2>(a, E, tiles, s) : launch<false, 2, 2, 4, 2, 3>(a, E, tiles, s);
  if (e != hipSuccess || !a.parts) return e;
  if (tall)
    join_parts_kernel<4><<<dim3(8 * 16 * (kUnits / 2)), dim3(256), 0, s>>>(a, E);
  else
    join_parts_kernel<2><<<dim3(8 * 8 * (kUnits / 2)), dim3(256), 0, s>>>(a, E);
  return hipGetLastError();
}

}  // namespace moe
