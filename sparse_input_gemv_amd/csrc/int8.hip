// Linear layers in 8-bit integers for gfx950: a scale per token and per output
// channel, exact 32-bit sums.
//
//   act_quantize_int8     s = fp32(max|x| / 127), q = round(x / s), by rows
//   weight_quantize_int8  the same by columns of WT, written as W [d_out][d_in]
//   int8_linear           y = act(sx sw sum_k xq wq + bias) + residual
//
// The product has k contiguous on both sides (a lane's operand is 16 bytes of
// one row), so W is stored untransposed here, and the dense layers' engine
// runs it in dx's layout with two integers to a 16-bit word: the same bytes per
// step and per matrix instruction, twice the operations.  Integer sums may be
// split anywhere and added in any order: equal calls give equal bits.
//
// Up to 4 tokens (and up to 8 of large weights) take dot products instead: a
// workgroup's 256 threads hold x in registers, 16 values of every 4096 each, and
// stream rows of W past it.  For one token of 16-bit values every workgroup
// quantises x itself (d_in values from L2), which saves the second launch.  More
// tokens, up to 64, of weights that are not too large take 16 channels per
// workgroup (k_int8_rows).
//
// Measured on MI355X, calls back to back, over several GPUs: 1 token 4096 -> 11008
// 9.4-10.3 us where the last-level cache holds a part of the few weights that take
// turns, 10.9 where it holds none (45 MB at 4.1 TB/s; a large copy runs at 4.8-5.1);
// 33 tokens 11008 -> 4096 19.6-20.6 (in a trace, which lengthens each launch: codes
// 4.0, product 12.8, its partial sums 4.2); 8192 tokens 4096 -> 14336 with bias and
// silu 408-449: 2140-2360 TOPS (the library's product of that size alone, with
// 32-bit sums written: 2261-2267 with both operands k-contiguous, 1986-2002 else).
#define SA_LINEAR_ENGINE_ONLY
#include "linear.hip"
#include "validate.hpp"

namespace sa {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// ---- rounding to 8 bits ------------------------------------------------------------
// A row's scale from its largest magnitude (the bits of a 16-bit value without
// its sign, which order magnitudes with Inf and NaN above all others): the
// rounded quotient, or NaN if the row holds Inf or NaN.
template <int DT>
__device__ __forceinline__ float scale_of(uint32_t most) {
  constexpr uint32_t inf = DT == SA_F16 ? 0x7c00u : 0x7f80u;
  if (most >= inf) return __builtin_nanf("");
  return to_f<DT>((uint16_t)most) / 127.f;
}
// x / s of the exact quotient, halves to even.
//
// x times the reciprocal of s is off the quotient by 2^-14 at most (127 times
// the reciprocal's and the product's 2^-22), so it rounds as the quotient does
// unless it lies that near to half a step.  Adding 3 2^22 rounds it to an
// integer, which the sum's low byte holds: a product, three sums and a byte
// move per value.  Where one of a lane's 4 values is within 2^-13 of half a step
// (5 in 10000 lanes), the remainders x - q s decide.  They are exact in fp32: x
// and q s are multiples of the last place of s unless |x| < s / 2^13, where q =
// 0.  Scales below 2^-100 (bf16 alone has them), zero and NaN always take that
// way, values and scale first multiplied by 2^64 so that the reciprocal exists.
struct Rounder {
  float s, inv, up;
  bool plain;
  __device__ __forceinline__ explicit Rounder(float scale) {
    plain = scale >= 0x1p-100f;
    up = plain ? 1.f : 0x1p64f;
    s = scale * up;
    inv = s > 0.f ? __builtin_amdgcn_rcpf(s) : 0.f;  // NaN, 0: every q is 0
  }
  __device__ __forceinline__ uint32_t exact(float x) const {
    const float v = x * up;
    float q = __builtin_rintf(v * inv);
    const float r = __builtin_fmaf(-q, s, v), twice = 2.f * fabsf(r);
    const bool odd = (int)q & 1;
    if (twice > s || (twice == s && odd)) q += __builtin_copysignf(1.f, r);
    return inv == 0.f ? 0u : (uint32_t)(int)q & 255u;
  }
  // The codes of four values, the first in the low byte.
  __device__ __forceinline__ uint32_t operator()(float a, float b, float c, float d) const {
    constexpr float kRound = 12582912.f;  // 3 2^22: a step there is 1
    const float v[4] = {a, b, c, d};
    float m[4], off = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = __builtin_fmaf(v[i], inv, kRound);
      off = fmaxf(off, fabsf(__builtin_fmaf(v[i], inv, kRound - m[i])));
    }
    if (__builtin_expect(plain && off <= 0.5f - 0x1p-13f, 1)) {
      // bytes 0 of two sums, then of the two pairs
      const uint32_t lo = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, m[1]), __builtin_bit_cast(uint32_t, m[0]), 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, m[3]), __builtin_bit_cast(uint32_t, m[2]), 0x04000c0cu);
      return lo | hi;
    }
    return exact(a) | exact(b) << 8 | exact(c) << 16 | exact(d) << 24;
  }
};
template <int DT>
__device__ __forceinline__ uint2 quant8(u32x4 v, const Rounder& r) {
  const F8 f = widen8<DT>(v);
  return uint2{r(f.v[0], f.v[1], f.v[2], f.v[3]), r(f.v[4], f.v[5], f.v[6], f.v[7])};
}
// The larger magnitudes of two pairs of 16-bit values.
__device__ __forceinline__ u16x2 larger(u16x2 a, uint32_t b) {
  return __builtin_elementwise_max(a, __builtin_bit_cast(u16x2, b & 0x7fff7fffu));
}
__device__ __forceinline__ u16x2 larger(u16x2 a, u32x4 b) {
  return larger(larger(larger(larger(a, b[0]), b[1]), b[2]), b[3]);
}
// The largest of the wave's values, uniform.
__device__ __forceinline__ uint32_t wave_most(u16x2 m) {
  int v = m[0] > m[1] ? m[0] : m[1];
  v = wave_running_max(v);
  return (uint32_t)__builtin_amdgcn_readlane(v, kWave - 1);
}

// ---- rows --------------------------------------------------------------------------
// A row per wave (NT = 64: 4 rows per workgroup) or per workgroup of NT threads,
// held in registers between its maximum and its rounding (NV chunks of 8 values
// per thread), or with NV = 0 read twice.  Bound by memory: 2 bytes read and one
// written per value.  8192 x 14336: 70 us, 5.0 TB/s (a large copy: 5.1).  Few
// rows are bound by latency, so they take 1024 threads each.
template <int DT, int NT, int NV>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void k_quant_rows(const uint16_t* __restrict__ x, int64_t ldx,
                                                                    int64_t T, int d, int8_t* __restrict__ xq,
                                                                    int64_t ldq, float* __restrict__ sx) {
  constexpr bool kWide = NT > 64;
  __shared__ uint32_t part[kWide ? NT / kWave : 1];
  const int lane = lane_id(), w = uni((int)threadIdx.x / kWave);
  const int64_t t = kWide ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + w;
  if (!kWide && t >= T) return;
  const int at = kWide ? (int)threadIdx.x : lane, chunks = d / 8;
  const u32x4* row = reinterpret_cast<const u32x4*>(x + t * ldx);
  constexpr int N = NV > 0 ? NV : 1;
  u32x4 v[N];
  u16x2 m = {0, 0};
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = at + j * NT < chunks ? row[at + j * NT] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NV; ++j) m = larger(m, v[j]);
  } else {
#pragma unroll 4
    for (int c = at; c < chunks; c += NT) m = larger(m, row[c]);
  }
  uint32_t most = wave_most(m);
  if constexpr (kWide) {
    if (lane == 0) part[w] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / kWave; ++i) most = part[i] > most ? part[i] : most;
  }
  const float s = scale_of<DT>(most);
  const Rounder r(s);
  if (at == 0) sx[t] = s;
  uint2* out = reinterpret_cast<uint2*>(xq + t * ldq);
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (at + j * NT < chunks) out[at + j * NT] = quant8<DT>(v[j], r);
  } else {
#pragma unroll 4
    for (int c = at; c < chunks; c += NT) out[c] = quant8<DT>(row[c], r);
  }
}

template <int DT>
void quant_rows(const uint16_t* x, int64_t ldx, int64_t T, int64_t d, int8_t* xq, int64_t ldq, float* sx,
                hipStream_t s) {
  auto run = [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, threads = NT > 64 ? NT : 256, rows = NT > 64 ? 1 : 4;
    // a launch counts its threads in 32 bits: 2^22 rows of 1024 threads are one too many
    constexpr int64_t most = (int64_t)0xffffffff / threads * rows;
    for (int64_t t = 0; t < T; t += most) {
      const int64_t n = T - t < most ? T - t : most;
      hipLaunchKernelGGL((k_quant_rows<DT, NT, decltype(nv)::value>), dim3((unsigned)((n + rows - 1) / rows)),
                         dim3(threads), 0, s, x + t * ldx, ldx, n, (int)d, xq + t * ldq, ldq, sx + t);
    }
  };
  using std::integral_constant;
  const integral_constant<int, 64> wave;
  const integral_constant<int, 256> wide;
  const integral_constant<int, 1024> widest;
  // a row per wave where that fills the CUs and a lane holds its part
  if (d <= 2048 && T >= 4 * kCus) run(wave, integral_constant<int, 4>{});
  else if (d <= 2048) run(wide, integral_constant<int, 1>{});
  else if (T < 2 * kCus && d <= 8192) run(widest, integral_constant<int, 1>{});
  else if (T < 2 * kCus && d <= 16384) run(widest, integral_constant<int, 2>{});
  else if (d <= 4096) run(wide, integral_constant<int, 2>{});
  else if (d <= 8192) run(wide, integral_constant<int, 4>{});
  else if (d <= 16384) run(wide, integral_constant<int, 8>{});
  else if (d <= 32768) run(widest, integral_constant<int, 4>{});
  else run(widest, integral_constant<int, 0>{});
}

// ---- columns (weights) ----------------------------------------------------------------
// The largest magnitudes of a strip's columns: 512 columns per workgroup, 8
// per lane, the strip's rows dealt over the waves.
constexpr int kColStrips = 64;  // at most
__global__ __launch_bounds__(256) void k_col_most(const uint16_t* __restrict__ wt, int64_t ldw, int64_t K,
                                                  int N, int64_t strip, uint16_t* __restrict__ part) {
  __shared__ u32x4 most[4][64];
  const int lane = lane_id(), w = uni((int)threadIdx.x / kWave);
  const int n = ((int)blockIdx.x * 64 + lane) * 8;
  const int64_t k0 = blockIdx.y * strip, k1 = k0 + strip < K ? k0 + strip : K;
  u16x2 m[4] = {};
  if (n < N) {
#pragma unroll 8
    for (int64_t k = k0 + w; k < k1; k += 4) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(wt + k * ldw + n);
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = larger(m[i], (uint32_t)v[i]);
    }
  }
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(uint32_t, m[i]);
  most[w][lane] = o;
  __syncthreads();
  if (w == 0 && n < N) {
#pragma unroll
    for (int j = 1; j < 4; ++j) {
      const u32x4 v = most[j][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = larger(m[i], (uint32_t)v[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_bit_cast(uint32_t, m[i]);
    *reinterpret_cast<u32x4*>(part + (int64_t)blockIdx.y * N + n) = o;
  }
}
// 256 k x 64 columns of WT, rounded and turned in LDS: a thread rounds 4 k of 8
// columns and writes a word of 4 k per column; rows of 65 words keep the
// lanes' banks apart.
template <int DT>
__global__ __launch_bounds__(256) void k_quant_cols(const uint16_t* __restrict__ wt, int64_t ldw, int64_t K,
                                                    int N, const uint16_t* __restrict__ part, int strips,
                                                    int8_t* __restrict__ wq, int64_t ldq,
                                                    float* __restrict__ sw) {
  __shared__ uint32_t most[4][64];
  __shared__ float scale[64];
  __shared__ uint32_t S[64 * 65];
  const int tid = (int)threadIdx.x, n0 = (int)blockIdx.x * 64;
  const int64_t k0 = (int64_t)blockIdx.y * 256;
  u32x4 v[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = k0 + (tid / 8 + 32 * h) * 4 + i;
      const int n = n0 + (tid % 8) * 8;
      v[h][i] = k < K && n < N ? *reinterpret_cast<const u32x4*>(wt + k * ldw + n) : u32x4{0, 0, 0, 0};
    }
  uint32_t m = 0;
  const int mine = n0 + tid % 64 < N ? n0 + tid % 64 : N - 1;
#pragma unroll
  for (int i = 0; i < kColStrips / 4; ++i) {  // all under way at once
    const int s = tid / 64 + 4 * i < strips ? tid / 64 + 4 * i : 0;
    const uint32_t o = part[(int64_t)s * N + mine];
    m = o > m ? o : m;
  }
  most[tid / 64][tid % 64] = m;
  __syncthreads();
  if (tid < 64) {
#pragma unroll
    for (int j = 1; j < 4; ++j) m = most[j][tid] > m ? most[j][tid] : m;
    scale[tid] = scale_of<DT>(m);
    if (blockIdx.y == 0 && n0 + tid < N) sw[n0 + tid] = scale[tid];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = (tid % 8) * 8 + i;
    const Rounder r(scale[c]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = to_f<DT>((uint16_t)(v[h][k][i / 2] >> (16 * (i % 2))));
      S[c * 65 + tid / 8 + 32 * h] = r(f[0], f[1], f[2], f[3]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int c = tid / 16 + 16 * h, k = (tid % 16) * 4;
    if (n0 + c < N && k0 + k * 4 < K) {  // K is a multiple of 16
      const uint32_t* p = S + c * 65 + k;
      *reinterpret_cast<u32x4*>(wq + (n0 + c) * ldq + k0 + k * 4) = u32x4{p[0], p[1], p[2], p[3]};
    }
  }
}
int64_t col_strip(int64_t K) {  // rows of a strip: 32 at least
  const int64_t s = (K + kColStrips - 1) / kColStrips;
  return s < 32 ? 32 : s;
}

// ---- dot products: few tokens ---------------------------------------------------------
struct GemvP {
  const void* x;    // QUANT: one 16-bit row; else 8-bit rows
  int64_t ldx;
  const float* sx;
  const int8_t* wq;
  int64_t ldw;
  const float* sw;
  int T, N, K;
  const uint16_t *bias, *res;
  int64_t ldr;
  int act;
  uint16_t* y;
  int64_t ldy;
};
constexpr int kGemvRows = 8, kGemvChannels = 64;  // per workgroup at most
constexpr int64_t kGemvPiece = 4096, kGemvPieces = 4;
// Adds lane sums: the wave's total in its last lane.
__device__ __forceinline__ int wave_total(int v) {
  v = row16_inclusive_scan(v);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return v;
}
// NT rows of x (those past T are zeros), KP pieces of 4096 k.  The channels are
// dealt evenly over the workgroups; U of them are under way per wave while U
// are multiplied, 8 loads of 1 KB at least.
template <int DT, int NT, int KP, bool QUANT>
__global__ __launch_bounds__(256) void k_int8_gemv(GemvP p) {
  static_assert(!QUANT || NT == 1, "one row is quantised in place");
  __shared__ uint32_t most[4];
  __shared__ __align__(16) int part[4][kGemvChannels * NT];
  const int tid = (int)threadIdx.x, lane = lane_id(), w = uni(tid / kWave);
  const int c0 = uni((int)((int64_t)p.N * (int)blockIdx.x / (int)gridDim.x));
  const int c1 = uni((int)((int64_t)p.N * ((int)blockIdx.x + 1) / (int)gridDim.x));
  constexpr int U = KP >= 3 ? 2 : 8 / KP;
  u32x4 next[U][KP];
  auto fetch = [&](int c) SA_INLINE {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int8_t* row = p.wq + (int64_t)(c + u < c1 ? c + u : c1 - 1) * p.ldw;  // past the end: not used
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        const int k = j * (int)kGemvPiece + tid * 16;
        next[u][j] = k < p.K ? *reinterpret_cast<const u32x4*>(row + k) : u32x4{0, 0, 0, 0};
      }
    }
  };
  fetch(c0);  // under way while x is made ready
  u32x4 x[NT][KP];
  float s = 0.f;
  if constexpr (QUANT) {
    const u32x4* row = reinterpret_cast<const u32x4*>(p.x);
    u32x4 v[KP][2];
    u16x2 m = {0, 0};
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const int k = j * (int)kGemvPiece + tid * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) v[j][h] = k < p.K ? row[k / 8 + h] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < KP; ++j) m = larger(larger(m, v[j][0]), v[j][1]);
    const uint32_t mine = wave_most(m);
    if (lane == 0) most[w] = mine;
    __syncthreads();
    const uint32_t a = most[0] > most[1] ? most[0] : most[1], b = most[2] > most[3] ? most[2] : most[3];
    s = scale_of<DT>(a > b ? a : b);
    const Rounder r(s);
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      const uint2 lo = quant8<DT>(v[j][0], r), hi = quant8<DT>(v[j][1], r);
      x[0][j] = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        const int k = j * (int)kGemvPiece + tid * 16;
        x[t][j] = t < p.T && k < p.K
                      ? *reinterpret_cast<const u32x4*>(static_cast<const int8_t*>(p.x) + t * p.ldx + k)
                      : u32x4{0, 0, 0, 0};
      }
  }
  for (int c = c0; c < c1; c += U) {
    u32x4 cur[U][KP];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < KP; ++j) cur[u][j] = next[u][j];
    if (c + U < c1) fetch(c + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int sum[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        int a = 0;
#pragma unroll
        for (int j = 0; j < KP; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) a = __builtin_amdgcn_sdot4((int)cur[u][j][e], (int)x[t][j][e], a, false);
        sum[t] = wave_total(a);
      }
      if (lane == kWave - 1 && c + u < c1) {
#pragma unroll
        for (int t = 0; t < NT; ++t) part[w][(c + u - c0) * NT + t] = sum[t];
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < (c1 - c0) * NT; i += 256) {
    const int t = i % NT, n = c0 + i / NT;
    if (t >= p.T) continue;
    const int sum = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
    float f = scaled_sum<false>(sum, p.sw[n], QUANT ? s : p.sx[t]);
    if (p.bias) f += to_f<DT>(p.bias[n]);
    with_act(p.act, [&](auto A) { f = act_value<decltype(A)::value>(f); });
    if (p.res) f += to_f<DT>(p.res[t * p.ldr + n]);
    p.y[t * p.ldy + n] = from_f<DT>(f);
  }
}

template <int DT, int NT, bool QUANT>
hipError_t gemv(const GemvP& p, hipStream_t s) {
  // two workgroups per CU, of four channels at least
  int64_t blocks = (p.N + 3) / 4 < 2 * kCus ? (p.N + 3) / 4 : 2 * kCus;
  const int64_t least = (p.N + kGemvChannels - 1) / kGemvChannels;
  blocks = blocks > least ? blocks : least;
  auto run = [&](auto kp) {
    hipLaunchKernelGGL((k_int8_gemv<DT, NT, decltype(kp)::value, QUANT>), dim3((unsigned)blocks), dim3(256), 0, s, p);
  };
  switch ((p.K + kGemvPiece - 1) / kGemvPiece) {
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 3: if constexpr (NT <= 4) run(std::integral_constant<int, 3>{}); break;
    default: if constexpr (NT <= 4) run(std::integral_constant<int, 4>{});
  }
  return hipGetLastError();
}

// ---- up to 64 tokens: 16 channels per workgroup ------------------------------------------
// Eight waves share d_in, 256 of every 2048 k each, and keep their own sums of
// 16 channels by 16 RB tokens; operands go straight from memory to registers (a
// lane's 16 bytes of a channel or a token are the matrix instruction's), and the
// next 256 k are under way while 256 are multiplied.  W is read once, x by every
// workgroup from L2.  No partial sums leave the workgroup, so there is no second
// launch.  Bound by the loads in flight: (1 + RB) bytes per weight arrive at 8 to
// 11 TB/s, so it pays while those are 92 MB at most (codes given; 33 tokens 4096
// -> 4096: 9.5 us, the split product 12.2; 16 tokens 11008 -> 4096: 12.8 against
// 14.2; but 33 tokens there 20.2 against 15.7).
constexpr int kRowsWaves = 8, kRowsK = 256;
constexpr int64_t kRowsMost = 64, kRowsBytes = 92 << 20;
template <int DT, int RB>
__global__ __launch_bounds__(kRowsWaves * 64) void k_int8_rows(GemvP p) {
  constexpr int U = kRowsK / 64;
  __shared__ __align__(16) int S[kRowsWaves][RB * 256];
  const int tid = (int)threadIdx.x, lane = lane_id(), w = uni(tid / kWave);
  const int i = lane % 16, g = lane / 16, c0 = (int)blockIdx.x * 16;
  // past the last channel or token: a row that exists, whose sums are not used
  const int8_t* wrow = p.wq + (int64_t)(c0 + i < p.N ? c0 + i : p.N - 1) * p.ldw;
  const int8_t* xrow[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r)
    xrow[r] = static_cast<const int8_t*>(p.x) + (int64_t)(r * 16 + i < p.T ? r * 16 + i : p.T - 1) * p.ldx;
  i4v a[U], b[U][RB];
  auto fetch = [&](int k0) SA_INLINE {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 64 + g * 16;
      const bool in = k < p.K;  // past the end: zero weights, any x
      const int at = in ? k : 0;
      const i4v v = *reinterpret_cast<const i4v*>(wrow + at);
      a[u] = in ? v : i4v{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < RB; ++r) b[u][r] = *reinterpret_cast<const i4v*>(xrow[r] + at);
    }
  };
  i4v sum[RB] = {};
  fetch(w * kRowsK);
  for (int k = w * kRowsK; k < p.K; k += kRowsWaves * kRowsK) {
    i4v ca[U], cb[U][RB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ca[u] = a[u];
#pragma unroll
      for (int r = 0; r < RB; ++r) cb[u][r] = b[u][r];
    }
    if (k + kRowsWaves * kRowsK < p.K) fetch(k + kRowsWaves * kRowsK);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RB; ++r)
        sum[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(ca[u], cb[u][r], sum[r], 0, 0, 0);
  }
  // lane: token 16 r + i, channels 4 g .. 4 g + 3
#pragma unroll
  for (int r = 0; r < RB; ++r) *reinterpret_cast<i4v*>(&S[w][(r * 16 + i) * 16 + 4 * g]) = sum[r];
  __syncthreads();
  for (int o = tid; o < RB * 256; o += kRowsWaves * 64) {
    const int t = o / 16, n = c0 + o % 16;
    if (t >= p.T || n >= p.N) continue;
    uint32_t total = 0;  // (int: 2^31 would overflow)
#pragma unroll
    for (int j = 0; j < kRowsWaves; ++j) total += (uint32_t)S[j][o];
    float f = scaled_sum<true>((int)total, p.sw[n], p.sx[t]);
    if (p.bias) f += to_f<DT>(p.bias[n]);
    with_act(p.act, [&](auto A) { f = act_value<decltype(A)::value>(f); });
    if (p.res) f += to_f<DT>(p.res[t * p.ldr + n]);
    p.y[t * p.ldy + n] = from_f<DT>(f);
  }
}
template <int DT>
hipError_t rows(const GemvP& p, hipStream_t s) {
  auto run = [&](auto rb) {
    hipLaunchKernelGGL((k_int8_rows<DT, decltype(rb)::value>), dim3((unsigned)((p.N + 15) / 16)),
                       dim3(kRowsWaves * 64), 0, s, p);
  };
  switch ((p.T + 15) / 16) {
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 3: run(std::integral_constant<int, 3>{}); break;
    default: run(std::integral_constant<int, 4>{});
  }
  return hipGetLastError();
}

// ---- matrix instructions ----------------------------------------------------------------
template <int DT, int EPI, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(256, 1) void k_int8(Int8P p) {
  __shared__ __align__(16) uint8_t S[lin_lds<kDx, BM, BN, NS>()];
  lin_run<DT, kDx, false, EPI, BM, BN, WM, WN, NS>(p, blockIdx.x, gridDim.x, S);
}
// Adds the shares' integer partials of 4 columns of a row and finishes them.
template <int DT>
__global__ __launch_bounds__(256) void k_int8_reduce(Int8P p, int lbm, int lbn) {
  const uint32_t n4 = p.N / 4, id = blockIdx.x * 256 + threadIdx.x;
  const uint32_t m = id / n4;
  const int n = (int)(id - m * n4) * 4;
  if (m >= (uint32_t)p.M) return;
  const int mt = (p.M + (1 << lbm) - 1) >> lbm, nt = (p.N + (1 << lbn) - 1) >> lbn;
  const uint32_t steps = (uint32_t)((p.K + BK - 1) / BK), TS = mt * nt * steps;
  const uint32_t at = (uint32_t)((n >> lbn) * mt + (int)(m >> lbm)) * steps;
  const int slots = share_of(at + steps - 1, TS, p.split) - share_of(at, TS, p.split) + 1;
  const u32x4* q = reinterpret_cast<const u32x4*>(p.part + (int64_t)m * p.N + n);
  const int64_t slot = (int64_t)p.M * p.N / 4;
  u32x4 sum = {0, 0, 0, 0};
#pragma unroll 8
  for (int s = 0; s < slots; ++s) sum += q[s * slot];
  const float sx = p.sx[m];
  uint16_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f = scaled_sum<true>((int)sum[i], p.sw[n + i], sx);
    if (p.bias) f += to_f<DT>(p.bias[n + i]);
    with_act(p.act, [&](auto A) { f = act_value<decltype(A)::value>(f); });
    if (p.res) f += to_f<DT>(p.res[m * (int64_t)p.ldr + n + i]);
    o[i] = from_f<DT>(f);
  }
  *reinterpret_cast<uint2*>(p.y[0] + m * (int64_t)p.ldy[0] + n) =
      uint2{(uint32_t)o[0] | (uint32_t)o[1] << 16, (uint32_t)o[2] | (uint32_t)o[3] << 16};
}

Plan int8_plan(int64_t T, int64_t d_in, int64_t d_out) {
  return lin_plan(kDx, false, T, d_out, d_in / 2, 1, 1);
}
// Which kernel: dot products (x in at most 64 registers), 16 channels per
// workgroup, or the tiles.  From 5 tokens on the second is as fast as the first
// or faster (8 tokens 4096 -> 4096 8.7 and 8.7 us, 11008 -> 4096 12.1 against the
// tiles' 13.9).
enum Kernel { kDots, kRows, kTilesOf };
Kernel kernel_of(int64_t T, int64_t d_in, int64_t d_out) {
  if (T <= 4 && d_in <= kGemvPiece * kGemvPieces) return kDots;
  if (T <= kRowsMost && (1 + (T + 15) / 16) * d_in * d_out <= kRowsBytes) return kRows;
  return T <= kGemvRows && d_in <= kGemvPiece * kGemvPieces / 2 ? kDots : kTilesOf;
}
// A single token of 16-bit values is quantised by the product's own launch.
bool quantise_first(int64_t T, int64_t d_in, int64_t d_out, bool quantised) {
  return !quantised && !(T == 1 && kernel_of(T, d_in, d_out) == kDots);
}

template <int DT>
hipError_t matmul(Int8P p, void* ws, hipStream_t s) {
  const Plan pl = int8_plan(p.M, (int64_t)p.K * 2, p.N);
  if (pl.tiles > 0x7fffffffLL) return hipErrorNotSupported;
  p.split = pl.split;
  p.part = reinterpret_cast<float*>(ws);
  const int64_t items = pl.split ? pl.split : pl.tiles;
  auto run = [&](auto bm, auto bn, auto wm, auto ns) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, NS = decltype(ns)::value;
    constexpr int64_t most = kCus * (160 * 1024 / lin_lds<kDx, BM, BN, NS>());
    const dim3 grid((unsigned)(p.split || items < most ? items : most));
    if (p.K * 2 == kMaxInt8Dim && !p.split)  // shares are added in k_int8_reduce
      hipLaunchKernelGGL((k_int8<DT, kInt8Long, BM, BN, WM, 4 / WM, NS>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_int8<DT, kInt8, BM, BN, WM, 4 / WM, NS>), grid, dim3(256), 0, s, p);
  };
  using std::integral_constant;
  const integral_constant<int, 1> c1;
  const integral_constant<int, 2> c2;
  const integral_constant<int, 3> c3;
  const integral_constant<int, 4> c4;
  const integral_constant<int, 128> c128;
  const integral_constant<int, 256> c256;
  switch (pl.tile) {
    case 0: run(c256, c256, c2, c2); break;
    case kNarrow: run(c256, integral_constant<int, 192>{}, c2, c2); break;
    case 1: run(c128, c128, c2, c2); break;
    case 2: run(integral_constant<int, 64>{}, c128, c1, c3); break;
    case 3: run(integral_constant<int, 32>{}, c128, c1, c3); break;
    default: run(integral_constant<int, 16>{}, c128, c1, c4);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !pl.split) return e;
  const int64_t n = ((int64_t)p.M * (p.N / 4) + 255) / 256;
  hipLaunchKernelGGL((k_int8_reduce<DT>), dim3((unsigned)n), dim3(256), 0, s, p,
                     __builtin_ctz(kTileM[pl.tile]), __builtin_ctz(kTileN[pl.tile]));
  return hipGetLastError();
}

// Scratch: 16-bit x's codes and scales, then the split product's partial sums.
struct Scratch {
  size_t codes = 0, scales = 0, end = 0;
};
Scratch scratch_of(int64_t T, int64_t d_in, int64_t d_out, bool quantised) {
  Scratch b;
  if (!quantise_first(T, d_in, d_out, quantised)) return b;
  b.scales = round256((size_t)(T * d_in));
  b.end = b.scales + round256((size_t)T * 4);
  return b;
}

template <int DT>
hipError_t linear_dt(const Int8Call& c, hipStream_t s) {
  char* ws = static_cast<char*>(c.ws);
  const Scratch b = scratch_of(c.T, c.d_in, c.d_out, c.sx != nullptr);
  const Kernel kernel = kernel_of(c.T, c.d_in, c.d_out);
  const void* x = c.x;
  int64_t ldx = c.ldx;
  const float* sx = c.sx;
  if (quantise_first(c.T, c.d_in, c.d_out, c.sx != nullptr)) {
    int8_t* codes = reinterpret_cast<int8_t*>(ws + b.codes);
    float* scales = reinterpret_cast<float*>(ws + b.scales);
    quant_rows<DT>(static_cast<const uint16_t*>(c.x), c.ldx, c.T, c.d_in, codes, c.d_in, scales, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    x = codes;
    ldx = c.d_in;
    sx = scales;
  }
  if (kernel != kTilesOf) {
    const GemvP p{x, ldx, sx, c.wq, c.ldw, c.sw, (int)c.T, (int)c.d_out, (int)c.d_in, c.bias, c.res,
                  c.ldr, c.act, c.y, c.ldy};
    if (kernel == kRows) return rows<DT>(p, s);
    if (c.T == 1) return sx ? gemv<DT, 1, false>(p, s) : gemv<DT, 1, true>(p, s);
    if (c.T == 2) return gemv<DT, 2, false>(p, s);
    return c.T <= 4 ? gemv<DT, 4, false>(p, s) : gemv<DT, 8, false>(p, s);
  }
  Int8P p{};
  p.p[0] = reinterpret_cast<const uint16_t*>(x);
  p.ldp = (int)(ldx / 2);
  p.q[0] = reinterpret_cast<const uint16_t*>(c.wq);
  p.ldq[0] = (int)(c.ldw / 2);
  p.M = (int)c.T;
  p.N = (int)c.d_out;
  p.K = (int)(c.d_in / 2);
  p.segs = p.outs = 1;
  p.act = c.act;
  p.bias = c.bias;
  p.res = c.res;
  p.ldr = (int)c.ldr;
  p.y[0] = c.y;
  p.ldy[0] = (int)c.ldy;
  p.sx = sx;
  p.sw = c.sw;
  return matmul<DT>(p, ws + b.end, s);
}

}  // namespace

hipError_t launch_act_quantize_int8(int dtype, const uint16_t* x, int64_t ldx, int64_t T, int64_t d, int8_t* xq,
                                    int64_t ldq, float* sx, hipStream_t s) {
  if (dtype == SA_F16) quant_rows<SA_F16>(x, ldx, T, d, xq, ldq, sx, s);
  else quant_rows<SA_BF16>(x, ldx, T, d, xq, ldq, sx, s);
  return hipGetLastError();
}

size_t weight_quantize_int8_workspace_bytes(int64_t d_in, int64_t d_out) {
  const int64_t strip = col_strip(d_in);
  return (size_t)((d_in + strip - 1) / strip * d_out * 2);
}

hipError_t launch_weight_quantize_int8(int dtype, const uint16_t* wt, int64_t ldw, int64_t d_in, int64_t d_out,
                                       int8_t* wq, int64_t ldq, float* sw, void* ws, hipStream_t s) {
  const int64_t strip = col_strip(d_in), strips = (d_in + strip - 1) / strip;
  const int64_t deep = (d_in + 255) / 256;
  uint16_t* part = static_cast<uint16_t*>(ws);
  hipLaunchKernelGGL(k_col_most, dim3((unsigned)((d_out + 511) / 512), (unsigned)strips), dim3(256), 0, s, wt, ldw,
                     d_in, (int)d_out, strip, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((d_out + 63) / 64), (unsigned)deep);
  if (dtype == SA_F16)
    hipLaunchKernelGGL((k_quant_cols<SA_F16>), grid, dim3(256), 0, s, wt, ldw, d_in, (int)d_out, part, (int)strips,
                       wq, ldq, sw);
  else
    hipLaunchKernelGGL((k_quant_cols<SA_BF16>), grid, dim3(256), 0, s, wt, ldw, d_in, (int)d_out, part,
                       (int)strips, wq, ldq, sw);
  return hipGetLastError();
}

size_t int8_linear_workspace_bytes(int64_t T, int64_t d_in, int64_t d_out, bool quantised) {
  const size_t b = scratch_of(T, d_in, d_out, quantised).end;
  return b + (kernel_of(T, d_in, d_out) != kTilesOf ? 0 : part_bytes(int8_plan(T, d_in, d_out), T, d_out, d_in / 2, 1, 1));
}

hipError_t launch_int8_linear(const Int8Call& c, hipStream_t s) {
  return c.dtype == SA_F16 ? linear_dt<SA_F16>(c, s) : linear_dt<SA_BF16>(c, s);
}

}  // namespace sa
