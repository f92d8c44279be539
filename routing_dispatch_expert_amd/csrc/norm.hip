// The root-mean-square norm in front of the MoE layer, with the residual's
// addition and an output in 8 bits, and its gradient (gfx950).
//
//   h = x + residual, rounded to the type: the stream that the layer adds to
//   rstd = 1 / sqrt(mean h^2 + eps);  y = h rstd weight
//   y8: y's values in 8 bits (mx8.h), from the fp32 y and not from its bf16
//   rounding (one rounding instead of two)
// gradient, with a = dy weight, n = h rstd, dres what arrives at h otherwise:
//   dh = rstd (a - n mean(a n)) + dres;  dweight = sum over rows of dy n
//
// A row is read once: its 16-byte words stay in registers between the sum and
// the use of it. Sums are in fp32 within a thread (64 numbers at most) and, of the
// squares, in fp64 between threads, in a fixed order. Bound by memory: 8192 x 7168
// bf16 with a residual and all outputs 87 us (530 MB, 6.1 TB/s).
#include "mx8.h"

#include <algorithm>

namespace moe {
namespace {

template <bool BF16>
__device__ inline void unpack(uint4 w, float (&v)[BF16 ? 8 : 4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if constexpr (BF16) {
      v[2 * q] = __uint_as_float(u[q] << 16);
      v[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
    } else {
      v[q] = __uint_as_float(u[q]);
    }
}

template <bool BF16>
__device__ inline uint4 pack(const float (&v)[BF16 ? 8 : 4]) {
  uint32_t u[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if constexpr (BF16)
      u[q] = f32_to_bf16(v[2 * q]) | static_cast<uint32_t>(f32_to_bf16(v[2 * q + 1])) << 16;
    else
      u[q] = __float_as_uint(v[q]);
  return uint4{u[0], u[1], u[2], u[3]};
}

// Sum over the THR threads that share a row (a wave, or the whole block): the
// same in all of them. red: LDS, one number a wave.
template <int THR, typename V>
__device__ inline V row_sum(V v, V* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if constexpr (THR > 64) {
    lds_barrier();  // the last sum's reads are over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    lds_barrier();
    v = 0;
#pragma unroll
    for (int i = 0; i < THR / 64; ++i) v += red[i];
  }
  return v;
}

// THR threads a row (64: four rows a block of 256), U words a thread, word tid +
// THR u: a 32-column group's words lie in neighbouring lanes.
template <bool BF16, int THR, int U>
__global__ __launch_bounds__(THR > 256 ? THR : 256) void rmsnorm_kernel(
    const uint4* x, const uint4* residual, const uint4* __restrict__ weight, float eps, int64_t R, int64_t d,
    uint4* h, uint4* __restrict__ y,  // h may be x or residual
    uint8_t* __restrict__ codes,
    uint32_t* __restrict__ scale, float* __restrict__ rstd) {
  constexpr int P = BF16 ? 8 : 4;   // elements of a word
  constexpr int L = 128 / P;        // lanes of a 128-column step
  __shared__ double red[16];
  const int tid = THR == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t r = THR == 64 ? blockIdx.x * 4ll + (threadIdx.x >> 6) : blockIdx.x;
  if (r >= R) return;  // whole waves, and no barrier with THR = 64
  const int64_t V = d / P;
  uint4 in[U], re[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t v = tid + THR * u;
    in[u] = uint4{0, 0, 0, 0};
    if (v < V) in[u] = load_stream(x + r * V + v);
  }
  if (residual) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = tid + THR * u;
      re[u] = uint4{0, 0, 0, 0};
      if (v < V) re[u] = load_stream(residual + r * V + v);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float a[P], b[P];
    unpack<BF16>(in[u], a);
    if (residual) {
      unpack<BF16>(re[u], b);
#pragma unroll
      for (int i = 0; i < P; ++i) a[i] += b[i];
      in[u] = pack<BF16>(a);
      unpack<BF16>(in[u], a);  // as it is stored
      const int64_t v = tid + THR * u;
      if (h && v < V) h[r * V + v] = in[u];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) sum = fmaf(a[i], a[i], sum);
  }
  // the threads' sums in 64 bits, and each of y's numbers rounded once: a value near a border of the 8-bit grid goes
  // to the other side of it the more seldom, and memory bounds the kernel all the same (8192 x 7168 bf16, eight inputs:
  // 18 to 31 of 59 million values beyond half a step of those in 64 bits, with fp32 throughout 22 to 40)
  const double total = row_sum<THR>(static_cast<double>(sum), red);
  const float rs = static_cast<float>(1.0 / sqrt(total / static_cast<double>(d) + static_cast<double>(eps)));
  if (rstd && tid == 0) rstd[r] = rs;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t v = tid + THR * u;
    if (THR * u >= V) break;  // the same for the whole row
    float a[P], w[P];
    unpack<BF16>(in[u], a);
    unpack<BF16>(v < V ? weight[v] : uint4{0, 0, 0, 0}, w);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float n = a[i] * rs, rest = fmaf(a[i], rs, -n);
      a[i] = rest == rest ? fmaf(n, w[i], rest * w[i]) : n * w[i];  // no rest of an infinite n
    }
    if (y && v < V) y[r * V + v] = pack<BF16>(a);
    if (codes) {
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) big = max(big, v < V ? __float_as_uint(a[i]) & 0x7fffffffu : 0u);
#pragma unroll
      for (int off = 1; off < 32 / P; off <<= 1) big = max(big, static_cast<uint32_t>(__shfl_xor(big, off, 64)));
      const uint32_t byte = mx8_scale_byte(big);
      const float inv = mx8_inverse(byte);
      const int lane = threadIdx.x & 63;
      uint32_t word = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) word |= static_cast<uint32_t>(__shfl(byte, (lane & ~(L - 1)) + b * (L / 4), 64)) << (8 * b);
      if (v % L == 0 && v < V) scale[mx8_scale_at(v / L, R, r)] = word;
      if (v < V) {
        const uint32_t lo = mx8_codes(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
        if constexpr (BF16)
          *reinterpret_cast<uint2*>(codes + r * d + v * P) =
              uint2{lo, mx8_codes(a[4] * inv, a[5] * inv, a[6] * inv, a[7] * inv)};
        else
          *reinterpret_cast<uint32_t*>(codes + r * d + v * P) = lo;
      }
    }
  }
}

// Gradient of the rows that the block (THR = 64: each of its four waves) takes in
// turn; its sum of dweight's terms stays in registers until the end and becomes a
// row of parts [gridDim][d]. 8192 x 4096 bf16 with dh_in: 45 us (268 MB, 6 TB/s; with 1024 blocks 50).
// Rows of more than 2048 words take 1024 threads, which have 128 registers each: three
// rows of words and dweight's sums do not fit them (bf16 4 words a thread 336 bytes of
// scratch a lane, 8 words 1112; fp32 8 words 468). With dweight_kernel, 268 MB each:
// bf16 d = 16384 64 us, 32768 155, 65536 405; fp32 16384 46 us, 32768 140.
template <bool BF16, int THR, int U>
__global__ __launch_bounds__(THR > 256 ? THR : 256) void rmsnorm_backward_kernel(
    const uint4* dy, const uint4* h, const uint4* __restrict__ weight, const float* __restrict__ rstd,
    const uint4* dres, int64_t R, int64_t d, uint4* dh,  // dh may be one of the inputs
    float* __restrict__ parts) {
  constexpr int P = BF16 ? 8 : 4;
  __shared__ float red[16];
  const int tid = THR == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t shares = THR == 64 ? gridDim.x * 4ll : gridDim.x;
  const int64_t part = THR == 64 ? blockIdx.x * 4ll + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t V = d / P;
  float dw[U][P];
  uint4 wt[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t v = tid + THR * u;
    wt[u] = v < V ? weight[v] : uint4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < P; ++i) dw[u][i] = 0.f;
  }
  for (int64_t r = part; r < R; r += shares) {
    const float rs = rstd[r];
    uint4 gy[U], gh[U], gr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = tid + THR * u;
      gy[u] = gh[u] = gr[u] = uint4{0, 0, 0, 0};
      if (v < V) {
        gy[u] = load_stream(dy + r * V + v);
        gh[u] = load_stream(h + r * V + v);
        if (dres) gr[u] = load_stream(dres + r * V + v);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float g[P], n[P], w[P];
      unpack<BF16>(gy[u], g);
      unpack<BF16>(gh[u], n);
      unpack<BF16>(wt[u], w);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        n[i] *= rs;
        dw[u][i] = fmaf(g[i], n[i], dw[u][i]);
        dot = fmaf(g[i] * w[i], n[i], dot);
      }
    }
    dot = row_sum<THR>(dot, red) / static_cast<float>(d);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = tid + THR * u;
      if (v >= V) continue;
      float g[P], n[P], w[P], o[P];
      unpack<BF16>(gy[u], g);
      unpack<BF16>(gh[u], n);
      unpack<BF16>(wt[u], w);
      unpack<BF16>(gr[u], o);
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = fmaf(rs, g[i] * w[i] - n[i] * rs * dot, o[i]);
      store_stream(dh + r * V + v, pack<BF16>(o));
    }
  }
  if constexpr (THR == 64) {  // the waves' sums, in their order, as one row
    __shared__ float4 sums[4][U * P / 4][64];
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < P; i += 4)
        sums[wave][(u * P + i) / 4][tid] = float4{dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]};
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 1; w < 4; ++w)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < P; i += 4) {
          const float4 o = sums[w][(u * P + i) / 4][tid];
          dw[u][i] += o.x;
          dw[u][i + 1] += o.y;
          dw[u][i + 2] += o.z;
          dw[u][i + 3] += o.w;
        }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t v = tid + THR * u;
    if (v >= V) continue;
#pragma unroll
    for (int i = 0; i < P; i += 4)
      *reinterpret_cast<float4*>(parts + blockIdx.x * d + v * P + i) = float4{dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]};
  }
}

// dweight = the parts' sums: a block has 32 columns, 32 slices of the parts side by
// side, each with eight loads on their way (one at a time, over 64 columns and 16
// slices, 1024 x 4096 parts took 17 us).
template <bool BF16>
__global__ __launch_bounds__(1024) void dweight_kernel(const float* __restrict__ parts, int64_t shares, int64_t d,
                                                       void* __restrict__ out) {
  __shared__ float red[32][32];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * 32ll + col;
  float sum = 0.f;
  if (c < d)
    for (int64_t p0 = slice; p0 < shares; p0 += 32 * 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p0 + 32 * i < shares ? parts[(p0 + 32 * i) * d + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
  red[slice][col] = sum;
  __syncthreads();
  if (slice || c >= d) return;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += red[i][col];
  if (BF16)
    static_cast<bf16_t*>(out)[c] = f32_to_bf16(sum);
  else
    static_cast<float*>(out)[c] = sum;
}

// Threads a row and words a thread for rows of V words: a wave up to 256 words,
// else 256 threads up to 2048, else 1024.
template <typename F>
bool norm_shape(int64_t V, F&& f) {
  using std::integral_constant;
#define MOE_SHAPE(T, U) f(integral_constant<int, T>{}, integral_constant<int, U>{})
  if (V <= 64)
    MOE_SHAPE(64, 1);
  else if (V <= 128)
    MOE_SHAPE(64, 2);
  else if (V <= 256)
    MOE_SHAPE(64, 4);
  else if (V <= 512)
    MOE_SHAPE(256, 2);
  else if (V <= 1024)
    MOE_SHAPE(256, 4);
  else if (V <= 2048)
    MOE_SHAPE(256, 8);
  else if (V <= 4096)
    MOE_SHAPE(1024, 4);
  else if (V <= 8192)
    MOE_SHAPE(1024, 8);
  else
    return false;
#undef MOE_SHAPE
  return true;
}

}  // namespace

int64_t rmsnorm_max_width(bool bf16) { return 8192 * (bf16 ? 8 : 4); }

hipError_t launch_rmsnorm(const void* x, const void* residual, const void* weight, float eps, int64_t R, int64_t d,
                          bool bf16, void* h, void* y, uint8_t* codes, uint32_t* scale, float* rstd, hipStream_t s) {
  const int64_t V = d / (bf16 ? 8 : 4);
  const auto* xv = static_cast<const uint4*>(x);
  const auto* rv = static_cast<const uint4*>(residual);
  const auto* wv = static_cast<const uint4*>(weight);
  auto* hv = static_cast<uint4*>(h);
  auto* yv = static_cast<uint4*>(y);
  const bool ok = norm_shape(V, [&](auto thr, auto u) {
    constexpr int T = decltype(thr)::value, U = decltype(u)::value;
    const dim3 grid(static_cast<unsigned>(T == 64 ? ceil_div(R, 4) : R));
    if (bf16)
      rmsnorm_kernel<true, T, U><<<grid, dim3(T == 64 ? 256 : T), 0, s>>>(xv, rv, wv, eps, R, d, hv, yv, codes, scale, rstd);
    else
      rmsnorm_kernel<false, T, U><<<grid, dim3(T == 64 ? 256 : T), 0, s>>>(xv, rv, wv, eps, R, d, hv, yv, codes, scale, rstd);
  });
  return ok ? hipGetLastError() : hipErrorInvalidValue;
}

// Blocks, and with them partial sums of dweight: by the sizes alone, so that
// results do not depend on the card's state.
int64_t rmsnorm_shares(int64_t R, int64_t d, bool bf16) {
  const int64_t V = d / (bf16 ? 8 : 4);
  if (V <= 256) return std::min<int64_t>(ceil_div(R, 4), 512);
  return std::min<int64_t>(R, V <= 2048 ? 512 : 256);
}

hipError_t launch_rmsnorm_backward(const void* dy, const void* h, const void* weight, const float* rstd,
                                   const void* dres, int64_t R, int64_t d, bool bf16, void* dh, void* dweight,
                                   float* parts, hipStream_t s) {
  const int64_t V = d / (bf16 ? 8 : 4), shares = rmsnorm_shares(R, d, bf16);
  const auto* gv = static_cast<const uint4*>(dy);
  const auto* hv = static_cast<const uint4*>(h);
  const auto* wv = static_cast<const uint4*>(weight);
  const auto* rv = static_cast<const uint4*>(dres);
  auto* ov = static_cast<uint4*>(dh);
  const bool ok = R == 0 || norm_shape(V, [&](auto thr, auto u) {
    constexpr int T = decltype(thr)::value, U = decltype(u)::value;
    const dim3 grid(static_cast<unsigned>(shares));
    if (bf16)
      rmsnorm_backward_kernel<true, T, U><<<grid, dim3(T == 64 ? 256 : T), 0, s>>>(gv, hv, wv, rstd, rv, R, d, ov, parts);
    else
      rmsnorm_backward_kernel<false, T, U><<<grid, dim3(T == 64 ? 256 : T), 0, s>>>(gv, hv, wv, rstd, rv, R, d, ov, parts);
  });
  if (!ok) return hipErrorInvalidValue;
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>(ceil_div(d, 32)));
  if (bf16)
    dweight_kernel<true><<<grid, dim3(1024), 0, s>>>(parts, shares, d, dweight);
  else
    dweight_kernel<false><<<grid, dim3(1024), 0, s>>>(parts, shares, d, dweight);
  return hipGetLastError();
}

}  // namespace moe
