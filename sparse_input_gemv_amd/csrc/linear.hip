// Dense linear layers for gfx950: the product with its epilogue, the gated
// pair of projections, and their gradients, fp16 or bf16 with fp32 sums.
//
//   dense_linear           y = act(x W^T + bias) + residual
//   gated_linear           h = act(x Wg^T) * (x Wu^T)
//   dense_linear_backward  d = dy * act'(pre); dx = d W, dW^T = x^T d,
//                          dbias = sum over rows of d
//   gated_linear_backward  dg = dh * u * act'(g), du = dh * act(g);
//                          dx = dg Wg + du Wu, dWg^T = x^T dg, dWu^T = x^T du
//
// Every product is one kernel, k_lin: C[m][n] = sum_k P[m][k] Q[k][n] for a
// row operand P and a column operand Q, each stored with k contiguous ("KC")
// or with m or n contiguous ("NC"):
//   forward  P = x  [T][d_in]  KC,  Q = WT [d_in][d_out] NC;
//   dx       P = d  [T][d_out] KC,  Q = WT, read as n = d_in, k = d_out: KC
//            (gated: the K loop runs over dg, Wg and then du, Wu);
//   dWT      P = x, read as m = d_in, k = T: NC,  Q = d [T][d_out]: NC
//            (gated: both outputs in one launch, side by side).
// The gated forward tile holds 128 columns of g and the same 128 of u, so the
// wave that ends with a g has its u, and x is read once for both.
//
// What bounds it, and what it measured on MI355X (bf16, random data; ranges
// are over GPUs):
//   large: the matrix cores' power.  MFMAs alone run at 2025 TFLOP/s with
//     random operands on all CUs (2414 with zeros, 2448 on one CU); the
//     kernel runs 8192 x 14336 x 4096 at 1295-1420 TFLOP/s, dx 4096 x 11008 x
//     4096 at 1340-1360, dW 4096 x 4096 x 11008 at 1240-1270 (2.7 rounds of
//     tiles; 4096 x 4096 x 16384, which fills its rounds, 1310-1390), gate and
//     up 8192 x 4096 x 14336 with g and u kept at 1270-1350.  The library's
//     product reaches 1410-1540 at 8192^3 with both operands K-contiguous,
//     1320 in the forward layout and 1150 in dW's.
//   few rows: the weights' stream.  1 x 4096 x 11008 gate and up 35 us (180
//     MB: 5.1 TB/s; a plain read runs at 7.2, a copy at 5.1), 8 x 11008 x
//     4096 19 us, 1 x 4096 x 4096 10 us (most of it launch and fill).
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "../../include/sparse_act.h"
#include "common.hpp"
#include "launch.hpp"

namespace sa {
namespace {

typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

// ---- element types ---------------------------------------------------------
template <int DT>
__device__ __forceinline__ float to_f(uint16_t b) {
  if constexpr (DT == SA_F16) return h2f(b);
  else return __builtin_bit_cast(float, (uint32_t)b << 16);
}
template <int DT>
__device__ __forceinline__ uint16_t from_f(float f) {  // round to nearest even
  if constexpr (DT == SA_F16) return f2h(f);
  else return __builtin_bit_cast(uint16_t, (__bf16)f);
}
// acc += a b on one 16 x 16 block, K = 32, in place in accumulation registers.
// Inline asm ties the result to the sum's registers: with 256 of them in use
// the compiler's own choice moves sums between registers in the K loop.
// Nothing reads a sum inside the loop; acc_settle() makes it readable.
template <int DT>
__device__ __forceinline__ void mfma16(f4v& acc, s8v a, s8v b) {
  if constexpr (DT == SA_F16)
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// Wait states that the compiler does not place around inline asm: after the
// last product, before other instructions read a sum (18 for a 16-pass
// product; this one takes 4 passes), and between other instructions' writes
// and a product (2).
__device__ __forceinline__ void acc_wait() { asm volatile("s_nop 15\n\ts_nop 7" ::: "memory"); }
__device__ __forceinline__ void acc_settle(f4v& acc) { asm volatile("" : "+a"(acc)); }

// ---- activations and their slopes (fp32) -------------------------------------
// sigma(z) = 1 / (1 + e^-z).  gelu's normal distribution function is, for
// z <= 0, e^(-z^2/2) erfcx(x) / 2 at x = -z / sqrt 2, with erfcx(x) = e^(x^2)
// erfc(x) as t times a polynomial of degree 8 in t = 1 / (1 + 0.4 x), fitted
// to the least largest relative error over x >= 0 (4.5e-7 in fp32); so it
// keeps its relative accuracy in the lower tail, and shares its exponential
// with the density.  erfcf took three times as long in the elementwise
// gradient, which it bound.
constexpr float kTanhA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;
__device__ __forceinline__ float normal_cdf(float z, float& e) {  // e: e^(-z^2/2)
  e = __expf(-0.5f * z * z);
  const float t = __builtin_amdgcn_rcpf(1.f + 0.28284271247461901f * fabsf(z));
  float q = 0.05026216432452202f;
  q = q * t - 0.18290163576602936f;
  q = q * t + 0.16908571124076843f;
  q = q * t - 0.005607785657048225f;
  q = q * t + 0.1414315551519394f;
  q = q * t + 0.16854193806648254f;
  q = q * t + 0.20784270763397217f;
  q = q * t + 0.22566959261894226f;
  q = q * t + 0.22567586600780487f;
  const float h = 0.5f * t * q * e;
  return z < 0.f ? h : 1.f - h;
}
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}
// The activation is a template argument where it is applied: a branch per
// value costs more than the value.
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (ACT == SA_ACT_RELU) return v <= 0.f ? 0.f : v;  // NaN stays NaN
  if constexpr (ACT == SA_ACT_RELU2) return v <= 0.f ? 0.f : v * v;
  if constexpr (ACT == SA_ACT_SILU) return v * sigmoid(v);
  if constexpr (ACT == SA_ACT_GELU) {
    float e;
    return v * normal_cdf(v, e);
  }
  if constexpr (ACT == SA_ACT_GELU_TANH)
    return v * sigmoid(2.f * kTanhA * (v + kTanhB * v * v * v));
  return v;
}
// Value and slope, sharing their transcendental part.
template <int ACT>
__device__ __forceinline__ void act_both(float v, float& f, float& df) {
  f = v;
  df = 1.f;
  if constexpr (ACT == SA_ACT_RELU) {
    f = v <= 0.f ? 0.f : v;
    df = v <= 0.f ? 0.f : 1.f;
  }
  if constexpr (ACT == SA_ACT_RELU2) {
    f = v <= 0.f ? 0.f : v * v;
    df = v <= 0.f ? 0.f : 2.f * v;
  }
  if constexpr (ACT == SA_ACT_SILU) {
    const float s = sigmoid(v);
    f = v * s;
    df = s * (1.f + v * (1.f - s));
  }
  if constexpr (ACT == SA_ACT_GELU) {
    float e;
    const float c = normal_cdf(v, e);
    f = v * c;
    df = c + v * 0.3989422804014327f * e;
  }
  if constexpr (ACT == SA_ACT_GELU_TANH) {
    const float s = sigmoid(2.f * kTanhA * (v + kTanhB * v * v * v));
    f = v * s;
    // s (1 - s) first: where v^2 is cut off, or v overflows a product, it is 0
    df = s + s * (1.f - s) * v * (2.f * kTanhA * (1.f + 3.f * kTanhB * fminf(v * v, 1e6f)));
  }
}
// f(integral_constant<act>) for the call's activation.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case SA_ACT_RELU: f(std::integral_constant<int, SA_ACT_RELU>{}); break;
    case SA_ACT_RELU2: f(std::integral_constant<int, SA_ACT_RELU2>{}); break;
    case SA_ACT_SILU: f(std::integral_constant<int, SA_ACT_SILU>{}); break;
    case SA_ACT_GELU: f(std::integral_constant<int, SA_ACT_GELU>{}); break;
    case SA_ACT_GELU_TANH: f(std::integral_constant<int, SA_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, SA_ACT_NONE>{});
  }
}

// ---- global memory to LDS ------------------------------------------------------
// Buffer loads straight into LDS: lane l's 16 bytes land at the LDS base +
// 16 l; a lane whose offset is not below the resource's size reads zeros.
// The resource's size is the operand's remaining bytes, so rows past an
// operand's end become zero rows.  Inline asm with a memory clobber, no
// result register, and waits stated by hand: the compiler cannot tell the
// stages apart and would drain every load before each LDS read.
typedef int i4v __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p);
}
// A value the whole wave shares, in a scalar register.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uni(const void* p) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return (uint64_t)(uint32_t)uni((int)(a >> 32)) << 32 | (uint32_t)uni((int)a);
}
constexpr uint32_t kOutOfRange = 0x80000000u;  // past every resource
// The LDS base goes in M0, which nothing else in these kernels uses.  The
// write needs one instruction between it and the load: the K loop puts a
// product there, load_lds16_now a no-op.
__device__ __forceinline__ void set_lds(uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0" : : "s"(lds) : "memory");
}
__device__ __forceinline__ void load_lds16(uint32_t voff, i4v rsrc) {
  asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(rsrc) : "memory");
}
// Non-temporal: for weights that are read once.
__device__ __forceinline__ void load_lds16_nt(uint32_t voff, i4v rsrc) {
  asm volatile("buffer_load_dwordx4 %0, %1, 0 offen nt lds" : : "v"(voff), "s"(rsrc) : "memory");
}

// Waits until at most VM loads and LG LDS reads are outstanding (63, 15: no
// wait), then the workgroup barrier.  s_waitcnt encoding: vmcnt bits 3:0 and
// 15:14, expcnt 6:4 (7: no wait), lgkmcnt 11:8.
template <int VM, int LG>
__device__ __forceinline__ void stage_barrier() {
  static_assert(VM >= 0 && VM < 64 && LG >= 0 && LG < 16, "counter ranges");
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | (LG << 8) | ((VM >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// ---- LDS tiles -----------------------------------------------------------------
// A K step covers 64 k.
//   KC tile: [rows][64] halves, 128-byte rows; 16-byte chunk c of row r lies
//     at chunk c ^ swz_kc(r), so the 8 (or 16) rows a read's lanes touch
//     together fall in distinct banks.  A lane's operand (8 consecutive k of
//     one row) is one 16-byte read.
//   NC tile: [64][128] halves per 128 columns, 256-byte rows; chunk c of row
//     k lies at chunk c ^ swz_nc(k).  A lane's operand (8 consecutive k of one
//     column) is two transpose reads (ds_read_b64_tr_b16: in a 16-lane group,
//     lane s addresses 4 halves of row k0 + s/4 at column c0 + 4 (s%4), lane i
//     receives column c0 + i of rows k0..k0+3).
constexpr int BK = 64;
constexpr int kHalfTile = BK * 128 * 2;  // bytes of an NC half tile
__device__ __forceinline__ int swz_kc(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int swz_nc(int k) { return 2 * ((k & 3) + 4 * ((k >> 3) & 1)); }

#define SA_INLINE __attribute__((always_inline))
#define SA_LDS(T, a) ((const __attribute__((address_space(3))) T*)(uintptr_t)(a))

__device__ __forceinline__ s8v read_kc(uint32_t a) { return *SA_LDS(s8v, a); }
__device__ __forceinline__ s8v read_nc(uint32_t a) {
  typedef __attribute__((address_space(3))) s4v* lp;
  const s4v q0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)a);
  const s4v q1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)(a + 4 * 256));
  return s8v{q0[0], q0[1], q0[2], q0[3], q1[0], q1[1], q1[2], q1[3]};
}

constexpr int kTicketStride = 32;  // 128 bytes: counters in one line would wait for each other
constexpr int kTicketTiles = 512;
enum Layout { kFwd = 0, kDx = 1, kDw = 2 };
// Epilogues, each compiled by itself (the general one needs registers that
// the plain one's K loop would have to give up): the sums as they are (gated:
// h alone), plus the residual, or everything; for fp16 gradients, the sums
// times their row's (dx) or column's (dW) power of two.
enum Epilogue { kPlain = 0, kResidual = 1, kGeneral = 2, kScaled = 3 };

struct LinP {
  const uint16_t* p[2];  // row operand (per K segment)
  const uint16_t* q[2];  // column operand (per K segment, gated half or output)
  int ldp, ldq[2];
  int M, N, K;           // K per segment
  int segs;              // K segments (dx of the gated pair: 2)
  int outs;              // outputs side by side (dW of the gated pair: 2)
  int split;             // 0: whole tiles; else the workgroups (a power of two) that
                         // share all tiles' steps
  float* part;           // split: [slot][outs * M][N * (gated ? 2 : 1)]
  uint32_t* tickets;     // split, or NULL: a zero counter per tile and wave, kTicketStride apart
  // epilogue
  int act;
  const uint16_t* bias;
  const uint16_t* res;
  int ldr;
  uint16_t* y[2];        // output (per outs)
  int ldy[2];
  uint16_t* pre[2];      // pre-activation, or g and u
  int ldpre[2];
  // scaled gradients (fp16), or NULL: powers of two that undo d's scales
  const float* rs;       // dx: [M]
  const float* cs;       // dW: [outs][N]
  const uint32_t* scaled;  // dx: not 0: the row operand is alt, not p
  const uint16_t* alt[2];
};

// f(0), ..., f(N - 1) with compile-time arguments.
template <class F, int... I>
__device__ __forceinline__ void static_for_(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_(std::make_integer_sequence<int, N>{}, f);
}

struct F8 {
  float v[8];
};
template <int DT>
__device__ __forceinline__ F8 load8(const uint16_t* p) {
  const u16x8 r = *reinterpret_cast<const u16x8*>(p);
  F8 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.v[i] = to_f<DT>(r[i]);
  return f;
}
template <int DT>
__device__ __forceinline__ void store8(uint16_t* p, const F8& f) {
  u16x8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = from_f<DT>(f.v[i]);
  *reinterpret_cast<u16x8*>(p) = o;
}

// f = act(f), value by value.
__device__ __forceinline__ void act8(int act, F8& f) {
  with_act(act, [&](auto A) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = act_value<decltype(A)::value>(f.v[i]);
  });
}

// Eight values of the element type.
template <int DT>
__device__ __forceinline__ F8 widen8(u32x4 r) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = r[i];
    f.v[2 * i] = to_f<DT>((uint16_t)(u & 0xffffu));
    f.v[2 * i + 1] = to_f<DT>((uint16_t)(u >> 16));
  }
  return f;
}
template <int DT>
__device__ __forceinline__ u32x4 round8(const F8& f) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)from_f<DT>(f.v[2 * i]) | (uint32_t)from_f<DT>(f.v[2 * i + 1]) << 16;
  return o;
}

// Slots are added in kChains chains (slot s to chain s % kChains), the chains
// then in order, wherever the sum is taken.
constexpr int kChains = 4;
__device__ __forceinline__ F8 add_chains(const F8 (&c)[kChains]) {
  F8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = ((c[0].v[e] + c[1].v[e]) + c[2].v[e]) + c[3].v[e];
  return f;
}

// A matrix's rows from m0 on as a buffer resource: rows past the last lie
// out of range (stores are dropped, loads read zeros).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint16_t* m, int64_t ld, int m0,
                                                            int rows, int N) {
  const uint64_t base = uni(m + (int64_t)m0 * ld);
  const int bytes = uni((rows - 1) * (int)ld * 2 + N * 2);
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00020000);
}

// Eight outputs of row m from column n on (n a multiple of 8 below N).
template <int DT, bool SCALED>
__device__ __forceinline__ void finish_linear(const LinP& p, int o, int64_t m, int n, F8 f) {
  if constexpr (SCALED) {
    const float r = p.rs ? p.rs[m] : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] *= p.cs ? p.cs[(int64_t)o * p.N + n + i] : r;
  }
  if (p.bias) {
    const F8 b = load8<DT>(p.bias + n);
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] += b.v[i];
  }
  if (p.pre[0]) store8<DT>(p.pre[0] + m * p.ldpre[0] + n, f);
  act8(p.act, f);
  if (p.res) {
    const F8 r = load8<DT>(p.res + m * p.ldr + n);
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] += r.v[i];
  }
  store8<DT>((o ? p.y[1] : p.y[0]) + m * (o ? p.ldy[1] : p.ldy[0]) + n, f);
}
template <int DT>
__device__ __forceinline__ void finish_gated(const LinP& p, int64_t m, int n, F8 g, const F8& u) {
  if (p.pre[0]) {
    store8<DT>(p.pre[0] + m * p.ldpre[0] + n, g);
    store8<DT>(p.pre[1] + m * p.ldpre[1] + n, u);
  }
  act8(p.act, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) g.v[i] *= u.v[i];
  store8<DT>(p.y[0] + m * p.ldy[0] + n, g);
}

// Two neighbouring blocks' sums of one row: lane group g holds columns
// 4g..4g+3 of each.  Swapping the odd groups of the first with the even
// groups of the second leaves every lane 8 consecutive columns: of the first
// block (g even) or the second (g odd), from column 8 (g / 2) on.
__device__ __forceinline__ F8 pair8(const f4v& a, const f4v& b) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = a[i], y = b[i];
    const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                    __builtin_bit_cast(uint32_t, y), false, false);
    const uint32_t lo = s[0], hi = s[1];
    f.v[i] = __builtin_bit_cast(float, lo);
    f.v[4 + i] = __builtin_bit_cast(float, hi);
  }
  return f;
}
__device__ __forceinline__ void store_part(float* p, const F8& f) {
  *reinterpret_cast<f4v*>(p) = f4v{f.v[0], f.v[1], f.v[2], f.v[3]};
  *reinterpret_cast<f4v*>(p + 4) = f4v{f.v[4], f.v[5], f.v[6], f.v[7]};
}
__device__ __forceinline__ void add_part(F8& f, const float* p) {
  const f4v a = *reinterpret_cast<const f4v*>(p), b = *reinterpret_cast<const f4v*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[i] += a[i];
    f.v[4 + i] += b[i];
  }
}

// The hardware deals workgroups over the 8 XCDs in turn; this gives each XCD a
// contiguous run of [0, total).  A bijection.
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t total) {
  const uint32_t x = b % 8, per = total / 8, rem = total % 8;
  return x * per + (x < rem ? x : rem) + b / 8;
}
// Whole tiles: an XCD's run goes through kGroupM row tiles across all column
// tiles, so tiles that run together on one XCD share operands in its L2.
constexpr int kGroupM = 4;
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t total, uint32_t mt, uint32_t nt, int& m,
                                        int& n) {
  const uint32_t t = xcd_run(b, total);
  const uint32_t gsz = kGroupM * nt;
  const uint32_t grp = t / gsz, first = grp * kGroupM;
  const uint32_t gm = (mt - first < kGroupM) ? mt - first : kGroupM;
  const uint32_t in = t - grp * gsz;
  n = uni((int)(in / gm));
  m = uni((int)(first + in - (uint32_t)n * gm));
}
// Split tiles: the steps of all tiles in a row (tile t's at t * steps ...)
// are dealt evenly: share i of G (a power of two) holds positions [i TS / G,
// (i + 1) TS / G).  share_of(P): the share that holds position P.  TS * G is
// at most 2^31.
__host__ __device__ __forceinline__ int share_of(uint32_t P, uint32_t TS, uint32_t G) {
  return (int)(((P + 1) * G - 1) / TS);
}

// One operand's tile: R rows (KC) or columns (NC) by 64 k, loaded by four
// waves with I instructions of 1 KB each.  start() places it at a K step;
// every next() moves one step on, and after `left` k has run out the loads
// read zeros.
template <bool NC, int R>
struct Operand {
  static constexpr int kRows = NC ? R : (R < 32 ? 32 : R);
  static constexpr int kBytes = kRows * BK * 2;
  static constexpr int I = kBytes / 1024 / 4;
  static_assert(!NC || R % 128 == 0, "NC tiles come in halves of 128 columns");
  static_assert(I >= 1, "one load per wave at least");
  uint32_t voff[I];
  int kc[2];              // KC: the lane's first k (even and odd instructions)
  uint64_t base;          // address of the step
  int64_t step;           // bytes per step
  int span, cols, ld;     // KC: bytes of the rows before the last; NC: columns left, row stride
  __device__ __forceinline__ void init(int w, int ldv) {
    const int lane = lane_id();
    ld = ldv;
    static_for<I>([&](auto J) {
      constexpr int j = decltype(J)::value;
      const int id = w * I + j;
      if constexpr (NC) {
        const int k = (id % 16) * 4 + lane / 16;
        const int c = (lane % 16) ^ swz_nc(k);
        voff[j] = (uint32_t)(k * ld * 2 + c * 16);
      } else {
        const int r = id * 8 + lane / 8;
        const int c = (lane % 8) ^ swz_kc(r);
        voff[j] = (uint32_t)(r * ld * 2 + c * 16);
        if constexpr (j < 2) kc[j] = 8 * c;
      }
    });
    if constexpr (!NC && I == 1) kc[1] = kc[0];
  }
  // The tile that starts at row (column) r0 of `rows`, at k0 of matrix m.
  __device__ __forceinline__ void start(const uint16_t* m, int r0, int rows, int k0, int w) {
    if constexpr (NC) {
      const int c0 = r0 + 128 * ((w * I) / 16);  // the wave's loads lie in one half tile
      cols = uni(rows - c0 > 0 ? rows - c0 : -(1 << 29));  // none left: no bytes at any step
      base = uni(m + (int64_t)k0 * ld + c0);
      step = (int64_t)BK * 2 * ld;
    } else {
      const int left = rows - r0 < R ? rows - r0 : R;
      span = uni((left - 1) * ld * 2);
      base = uni(m + (int64_t)r0 * ld + k0);
      step = BK * 2;
    }
  }
  // The step's resource: the bytes from its base to the operand's end, with
  // `left` k to come (0 or less: none).
  __device__ __forceinline__ i4v rsrc(int left) const {
    int bytes;
    if constexpr (NC) {
      bytes = (((left < BK ? left : BK) - 1) * ld + cols) * 2;  // cols <= ld
      bytes = bytes > 0 ? bytes : 0;
    } else {
      bytes = left > 0 ? span + left * 2 : 0;
    }
    return i4v{uni((int)(uint32_t)base), uni((int)((uint32_t)(base >> 32) & 0xffffu)), uni(bytes),
               0x00020000};
  }
  __device__ __forceinline__ void next() { base += step; }
  // Load j of the step, in two parts: its place in LDS (M0), then the load.
  // KC chunks past the row's end are zeros, not the next row.
  __device__ __forceinline__ static void place(int j, uint32_t lds, int w) {
    set_lds(lds + (w * I + j) * 1024);
  }
  __device__ __forceinline__ void load(int j, i4v rs, int left, bool once) const {
    uint32_t v = voff[j];
    if constexpr (!NC) v = kc[j & 1] < left ? v : kOutOfRange;
    if (once) load_lds16_nt(v, rs);
    else load_lds16(v, rs);
  }
};

// C tiles of BM x BN (gated: BN / 2 columns of g and of u), 256 threads as
// WM x WN waves.  A workgroup takes tiles blockIdx.x, blockIdx.x + gridDim.x,
// ..., or, where tiles are few, an even share of all tiles' steps, whose
// partial sums k_lin_reduce adds.  It runs one K loop over all its items: the
// loads of the next item's first steps are under way while an item's outputs
// are written.
//
// A step is two halves of 32 k, each N products per wave.  Operands are
// double buffered in registers by halves: half 0 carries the LDS reads of
// half 1 in its first RS products, half 1 those of the next step's half 0.
// After REL products of half 0 every wave has read all of the stage (one
// barrier), and its buffer takes the loads of stage t + NS, spread evenly over
// the products up to product X of the next step's half 0: a CU's loads share
// one address path that takes 16 cycles per load, and the waves issue them
// together.  After RDY products of half 1 (the other barrier) stage t + 1 has
// arrived.  Loads past the last item read zeros, so counts never change.
// gfx950 at 256 x 256: 64 KB per stage, two stages, one wave per SIMD with
// 256 sums in accumulation registers.
template <int LAY, int BM, int BN, int NS>
constexpr int lin_lds() {
  return NS * (Operand<LAY == kDw, BM>::kBytes +
               Operand<LAY != kDx, LAY != kDx ? (BN + 127) / 128 * 128 : BN>::kBytes);
}
// Workgroup `block` of `blocks`, with lin_lds bytes at S.
template <int DT, int LAY, bool GATED, int EPI, int BM, int BN, int WM, int WN, int NS>
__device__ __forceinline__ void lin_run(const LinP& p, int block, int blocks, uint8_t* S) {
  constexpr bool PNC = LAY == kDw, QNC = LAY != kDx;
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
  static_assert(WM * WN == 4 && MB >= 1 && NB >= 2 && NB % (GATED ? 4 : 2) == 0, "four waves");
  using OP = Operand<PNC, BM>;
  using OQ = Operand<QNC, QNC ? (BN + 127) / 128 * 128 : BN>;  // NC: whole halves are loaded
  constexpr int L = OP::I + OQ::I;
  const uint32_t lp = lds_addr(S), lq = lp + NS * OP::kBytes;

  constexpr int N = MB * NB, R = MB + NB;
  constexpr int RS = N * 5 / 8 > 0 ? N * 5 / 8 : 1;
  constexpr int REL = RS + N / 16, RDY = N * 5 / 16, X = N * 5 / 16;
  constexpr int SPAN = 2 * N + X - REL;
  static_assert(REL < N && RDY + RS <= N && X <= REL, "schedule");
  // Load j's position is REL + j * SPAN / L products from the start of the
  // step; loads at positions below q:
  constexpr auto before = [](int q) constexpr {
    int c = 0;
    for (int j = 0; j < L; ++j) c += (REL + j * SPAN / L) < q;
    return c;
  };
  // product of half 0 that carries piece i of the move to the next stage:
  // after the loads left over from the step before, up to 6 before REL
  constexpr auto piece = [](int i) constexpr {
    return REL - X > 12 ? X + i * (REL - 6 - X) / 6 : X;
  };
  constexpr int J1 = before(2 * N);       // loads within the step; the others in the next
  constexpr int CR = before(N + RDY);     // loads issued when stage t + 1 must have arrived

  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wm = w / WN, wn = w % WN;
  constexpr int BNO = GATED ? BN / 2 : BN;  // output columns per tile
  const int mt = (p.M + BM - 1) / BM, nt1 = (p.N + BNO - 1) / BNO;
  const int nt = nt1 * p.outs;
  const int tiles = mt * nt;
  const int ks = (p.K + BK - 1) / BK;  // steps per segment
  const int steps = ks * p.segs;
  // A cursor goes over the workgroup's items: a tile's number, or (split) a
  // position among all tiles' steps, up to `end`.
  const bool split = p.split > 0;
  // Row tiles that read the same weights are kept on one XCD; with a single
  // one nothing is shared, and neighbouring shares on different XCDs stream
  // faster (one row of 4096 x 4096: 11.4 -> 11.1 us).
  const int share = !split ? 0 : mt == 1 ? block : (int)xcd_run(block, blocks);
  const int lg = split ? __builtin_ctz(p.split) : 0;
  const int begin = split ? (int)((uint32_t)share * (uint32_t)(tiles * steps) >> lg) : block;
  const int end = split ? (int)((uint32_t)(share + 1) * (uint32_t)(tiles * steps) >> lg) : tiles;
  struct Item {
    int m0, n0, out, s0, s1, next;
  };
  auto item_at = [&](int cur) SA_INLINE {
    Item it;
    int mi, ni;
    if (split) {
      const int t = uni((int)((uint32_t)cur / (uint32_t)steps));
      ni = mt == 1 ? t : uni((int)((uint32_t)t / (uint32_t)mt));
      mi = t - ni * mt;
      it.s0 = cur - t * steps;
      it.s1 = uni(it.s0 + end - cur < steps ? it.s0 + end - cur : steps);
      it.next = cur + it.s1 - it.s0;
    } else {
      tile_of(cur, tiles, mt, nt, mi, ni);
      it.s0 = 0;
      it.s1 = steps;
      it.next = cur + blocks;
    }
    it.out = ni >= nt1;
    it.m0 = mi * BM;
    it.n0 = (ni - (it.out ? nt1 : 0)) * BNO;
    return it;
  };

  // ---- the loading side: the stage under way
  OP op;
  OQ oq;
  // gated: the waves of the second half load u's weight
  const int qh = GATED ? (w * OQ::I) / 16 : 0;
  op.init(w, p.ldp);
  oq.init(w, qh ? p.ldq[1] : p.ldq[0]);
  const uint16_t *p0 = p.p[0], *p1 = p.p[1];
  if constexpr (EPI == kScaled && LAY == kDx) {
    if (p.scaled && uni((int)*p.scaled)) {
      p0 = p.alt[0];
      p1 = p.alt[1];
    }
  }
  Item li = item_at(begin);
  int at = li.s0;  // its step
  int stop = 0;    // the step at which the segment or the item ends
  int left = 0;    // k left in the segment (0 or less: past the last item)
  i4v rp, rq;
  auto place = [&]() SA_INLINE {  // at step `at` of item li
    const int seg = at >= ks;
    const int k0 = (at - seg * ks) * BK;
    left = uni(p.K - k0);
    stop = uni(!seg && ks < li.s1 ? ks : li.s1);
    if (LAY == kDx && p.segs == 2) oq.init(w, seg ? p.ldq[1] : p.ldq[0]);
    const bool second = GATED ? qh : LAY == kDx ? seg : LAY == kDw ? li.out : 0;
    op.start(LAY == kDx && seg ? p1 : p0, li.m0, p.M, k0, w);
    // gated: half 0 is g's columns, half 1 u's, both from n0 on
    oq.start(second ? p.q[1] : p.q[0], GATED ? li.n0 - 128 * qh : li.n0, p.N, k0, w);
  };
  // The move to the next stage, in pieces that the K loop spreads over its
  // products.  The resources' scalar registers must be written 5 instructions
  // before a load reads them (the compiler places no wait states around
  // inline asm); settle() fixes them there.
  auto advance = [&]() SA_INLINE {
    ++at;
    left -= BK;
  };
  auto turn = [&]() SA_INLINE {
    if (__builtin_expect(at == stop, 0)) {
      if (at == li.s1) {
        if (li.next < end) {
          li = item_at(li.next);
          at = li.s0;
        } else {
          left = 0;
          stop = -1;  // never reached
        }
      }
      if (stop >= 0) place();
    }
  };
  auto settle = [&]() SA_INLINE { asm volatile("" : "+s"(rp), "+s"(rq)); };
  auto set_one = [&](int j, int buf) SA_INLINE {
    if (j < OP::I) OP::place(j, lp + buf * OP::kBytes, w);
    else OQ::place(j - OP::I, lq + buf * OQ::kBytes, w);
  };
  // A single row tile reads its weights once, past the caches (one row of
  // 4096 x 4096: 13.4 -> 11.4 us, gate and up 4096 x 11008: 40.4 -> 37.1).
  const bool once = BM <= 64 && LAY != kDw && mt == 1;
  auto load_one = [&](int j) SA_INLINE {
    if (j < OP::I) op.load(j, rp, left, false);
    else oq.load(j - OP::I, rq, left, once);
  };

  // ---- the computing side
  // LDS addresses of a lane's operands: KC one per half step (blocks are 16
  // rows, a constant apart), NC one per block of 16 columns (the swizzle
  // acts on the block's bits; half steps are a constant apart).
  const int g = lane / 16, i = lane % 16;
  auto kc_addr = [&](int row0, int kk) SA_INLINE {
    return (uint32_t)((row0 + i) * 128 + (((4 * kk + g) ^ swz_kc(i)) * 16));
  };
  auto nc_addr = [&](int blk) SA_INLINE {  // block of 16 columns
    const int s = (i >> 2) + 4 * (g & 1);
    return (uint32_t)((blk >> 3) * kHalfTile + (8 * g + (i >> 2)) * 256 +
                      ((2 * ((blk & 7) ^ s) + ((i >> 1) & 1)) * 16) + (i & 1) * 8);
  };
  constexpr int PA = PNC ? MB : 2, QA = QNC ? NB : 2;
  uint32_t pa[PA], qa[QA];
#pragma unroll
  for (int j = 0; j < PA; ++j)
    pa[j] = lp + (PNC ? nc_addr(wm * MB + j) : kc_addr(wm * MB * 16, j));
#pragma unroll
  for (int j = 0; j < QA; ++j) {
    if constexpr (QNC) {
      const int blk = GATED ? (j < NB / 2 ? wn * (NB / 2) + j : 8 + wn * (NB / 2) + j - NB / 2)
                            : wn * NB + j;
      qa[j] = lq + nc_addr(blk);
    } else {
      qa[j] = lq + kc_addr(wn * NB * 16, j);
    }
  }

  f4v acc[MB][NB];
  auto clear = [&]() SA_INLINE {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        acc[a][b] = f4v{0.f, 0.f, 0.f, 0.f};
        acc_settle(acc[a][b]);
      }
    acc_wait();
  };
  s8v fp[2][MB], fq[2][NB];
  // operand r of a half step, in the order of their first use: Q, then P
  auto read_one = [&](int r, int kk, int buf) SA_INLINE {
    const uint32_t po = buf * OP::kBytes, qo = buf * OQ::kBytes;
    if (r < NB)
      fq[kk][r] = QNC ? read_nc(qa[QNC ? r : 0] + qo + kk * 32 * 256)
                      : read_kc(qa[QNC ? 0 : kk] + qo + r * 16 * 128);
    else
      fp[kk][r - NB] = PNC ? read_nc(pa[PNC ? r - NB : 0] + po + kk * 32 * 256)
                           : read_kc(pa[PNC ? 0 : kk] + po + (r - NB) * 16 * 128);
  };
  // Half kk of a step on stage buffer `buf` (before: pbuf, next: nbuf).  The
  // order is pinned product by product.
  auto half = [&](auto KK, int pbuf, int buf, int nbuf) SA_INLINE {
    constexpr int kk = decltype(KK)::value;
    static_for<N>([&](auto M) {
      constexpr int m = decltype(M)::value;
      if constexpr (kk == 0 && m == REL) stage_barrier<63, 0>();
      if constexpr (kk == 0) {
        if constexpr (m == piece(0)) advance();
        if constexpr (m == piece(1)) op.next();
        if constexpr (m == piece(2)) oq.next();
        if constexpr (m == piece(3)) turn();
        if constexpr (m == piece(4)) rp = op.rsrc(left);
        if constexpr (m == piece(5)) rq = oq.rsrc(left);
        if constexpr (m == piece(6)) {
          settle();
          if constexpr (REL - piece(6) < 5) asm volatile("s_nop 4" ::: "memory");
        }
      }
      if constexpr (kk == 1 && m == RDY) stage_barrier<CR + (NS - 2) * L, 15>();
      constexpr int rs = kk == 0 ? m : m - RDY;  // reads r with r * RS / R == rs
      static_for<(rs >= 0 && rs < RS ? ((rs + 1) * R + RS - 1) / RS - (rs * R + RS - 1) / RS : 0)>(
          [&](auto I) {
            read_one((rs * R + RS - 1) / RS + decltype(I)::value, 1 - kk, kk == 0 ? buf : nbuf);
          });
      // the loads at this position, or left over from the step before
      constexpr int q = kk == 1 ? N + m : m < X ? 2 * N + m : m;
      constexpr int j0 = before(q), jn = before(q + 1) - j0;
      const int lbuf = kk == 0 && m < X ? pbuf : buf;
      if constexpr (jn > 0) set_one(j0, lbuf);
      mfma16<DT>(acc[m / NB][m % NB], fq[kk][m % NB], fp[kk][m / NB]);
      if constexpr (jn > 0) load_one(j0);
      static_for<(jn > 1 ? jn - 1 : 0)>([&](auto I) {
        set_one(j0 + 1 + decltype(I)::value, lbuf);
        asm volatile("s_nop 0" ::: "memory");
        load_one(j0 + 1 + decltype(I)::value);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // Writes an item's outputs (or its partial sums) and clears the sums.
  // Lane: row 16 a + i, 8 columns from 16 (b + g % 2) + 8 (g / 2) on of every
  // pair (b, b + 1) of output blocks.
  constexpr int NO = GATED ? NB / 2 : NB;  // output blocks
  // Row by row, as few registers are free beside the next item's operands: a
  // spill's reload would wait for the stores before it.
  auto take_row = [&](int a) SA_INLINE {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < NB; ++b) acc_settle(acc[a][b]);
  };
  // One-launch joining (a wave owns its columns): partials are stored through
  // to memory (sc1: coherent between XCDs); when they have arrived, the wave
  // counts itself in, and the last of a tile's shares adds all of them and
  // finishes the outputs.  No wave waits for another.
  constexpr bool kJoin = LAY == kFwd && WM == 1;
  constexpr int kCoherent = 16;  // buffer accesses' sc1 bit
  const auto part_rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p.part, 0, 0x7fffffff, 0x00020000);
  auto part_at = [&](int slot, int m, int n) SA_INLINE {
    return (uint32_t)((slot * p.M + m) * (GATED ? 2 : 1) * p.N + n) * 4u;
  };
  auto put_part = [&](uint32_t at, const F8& f) SA_INLINE {
    u32x4 lo, hi;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = f.v[e], y = f.v[4 + e];
      lo[e] = __builtin_bit_cast(uint32_t, x);
      hi[e] = __builtin_bit_cast(uint32_t, y);
    }
    __builtin_amdgcn_raw_buffer_store_b128(lo, part_rsrc, at, 0, kCoherent);
    __builtin_amdgcn_raw_buffer_store_b128(hi, part_rsrc, at + 16, 0, kCoherent);
  };
  auto get_part = [&](uint32_t at, F8& f) SA_INLINE {
    const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(part_rsrc, at, 0, kCoherent);
    const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(part_rsrc, at + 16, 0, kCoherent);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = lo[e], y = hi[e];
      f.v[e] += __builtin_bit_cast(float, x);
      f.v[4 + e] += __builtin_bit_cast(float, y);
    }
  };
  auto join = [&](const Item& it, int t) SA_INLINE {
    const int slots = uni(share_of(t * steps + steps - 1, tiles * steps, p.split) -
                          share_of(t * steps, tiles * steps, p.split) + 1);
    uint32_t* const ticket = p.tickets + (t * 4 + w) * kTicketStride;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int before_me = 0;
    if (lane == 0)
      before_me = (int)__hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (uni(before_me) != slots - 1) return;
    if (lane == 0) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    constexpr int OC = NO * 2;  // octets of the wave's columns
    const int rows = p.M - it.m0 < BM ? p.M - it.m0 : BM;
    for (int o = lane; o < rows * OC; o += 64) {
      const int m = it.m0 + o / OC, n = it.n0 + wn * NO * 16 + (o % OC) * 8;
      if (n >= p.N) continue;
      F8 f[kChains] = {}, u[kChains] = {};
      for (int s = 0; s < slots; s += kChains) {
#pragma unroll
        for (int c = 0; c < kChains; ++c) {
          if (s + c >= slots) break;
          const uint32_t q = part_at(s + c, m, n);
          get_part(q, f[c]);
          if constexpr (GATED) get_part(q + 4 * p.N, u[c]);
        }
      }
      const F8 fs = add_chains(f);
      if constexpr (GATED) finish_gated<DT>(p, m, n, fs, add_chains(u));
      else finish_linear<DT, EPI == kScaled>(p, it.out, m, n, fs);
    }
  };
  auto finish_parts = [&](const Item& it) SA_INLINE {
    // slot: how many shares before this one hold part of the tile
    const int t = (it.n0 / BNO + (it.out ? nt1 : 0)) * mt + it.m0 / BM;
    const int slot = it.s0 == 0 ? 0 : uni(share - share_of(t * steps, tiles * steps, p.split));
    static_for<MB>([&](auto A) {
      constexpr int a = decltype(A)::value;
      take_row(a);
      const int m = it.m0 + (wm * MB + a) * 16 + i;
#pragma unroll
      for (int b = 0; b < NO; b += 2) {
        const F8 f = pair8(acc[a][b], acc[a][b + 1]);
        const int n = it.n0 + (wn * NO + b + (g & 1)) * 16 + 8 * (g >> 1);
        if constexpr (kJoin) {
          if (p.tickets) {
            const uint32_t q = m < p.M && n < p.N ? part_at(slot, m, n) : kOutOfRange;
            put_part(q, f);
            if constexpr (GATED)
              put_part(q + 4 * p.N, pair8(acc[a][b + NO], acc[a][b + NO + 1]));
            continue;
          }
        }
        if constexpr (GATED) {
          const F8 u = pair8(acc[a][b + NO], acc[a][b + NO + 1]);
          if (m >= p.M || n >= p.N) continue;
          float* q = p.part + (((int64_t)slot * p.M + m) * 2) * p.N + n;
          store_part(q, f);
          store_part(q + p.N, u);
        } else {
          if (m >= p.M || n >= p.N) continue;
          store_part(p.part + ((int64_t)(slot * p.outs + it.out) * p.M + m) * p.N + n, f);
        }
      }
    });
    if constexpr (kJoin) {
      if (p.tickets) join(it, t);
    }
  };
  auto finish_rows = [&](const Item& it) SA_INLINE {
    constexpr int mode = EPI;
    const int rows = p.M - it.m0 < BM ? p.M - it.m0 : BM;
    const int ldy = it.out ? p.ldy[1] : p.ldy[0];
    const auto yr = rows_rsrc(it.out ? p.y[1] : p.y[0], ldy, it.m0, rows, p.N);
    const int row = wm * MB * 16 + i;
    uint32_t col[NO / 2];  // byte offset of the lane's columns, or out of range
#pragma unroll
    for (int b = 0; b < NO / 2; ++b) {
      const int n = it.n0 + (wn * NO + 2 * b + (g & 1)) * 16 + 8 * (g >> 1);
      col[b] = n < p.N ? (uint32_t)n * 2 : kOutOfRange;
    }
    const uint32_t yo = (uint32_t)(row * ldy * 2);
    const int ystep = 16 * ldy * 2;  // added to the lane's offset: the range check covers that
    if constexpr (GATED) {
      const bool gu = mode == kGeneral && p.pre[0];
      const auto gr = rows_rsrc(gu ? p.pre[0] : p.y[0], gu ? p.ldpre[0] : 0, it.m0, gu ? rows : 1, gu ? p.N : 0);
      const auto ur = rows_rsrc(gu ? p.pre[1] : p.y[0], gu ? p.ldpre[1] : 0, it.m0, gu ? rows : 1, gu ? p.N : 0);
      static_for<MB>([&](auto A) {
        constexpr int a = decltype(A)::value;
        take_row(a);
#pragma unroll
        for (int b = 0; b < NO; b += 2) {
          F8 f = pair8(acc[a][b], acc[a][b + 1]);
          const F8 u = pair8(acc[a][b + NO], acc[a][b + NO + 1]);
          if constexpr (mode == kGeneral) {
            __builtin_amdgcn_raw_buffer_store_b128(round8<DT>(f), gr,
                (uint32_t)((row + 16 * a) * p.ldpre[0] * 2) + col[b / 2], 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(round8<DT>(u), ur,
                (uint32_t)((row + 16 * a) * p.ldpre[1] * 2) + col[b / 2], 0, 0);
          }
          act8(p.act, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f.v[e] *= u.v[e];
          __builtin_amdgcn_raw_buffer_store_b128(round8<DT>(f), yr, yo + (uint32_t)(a * ystep) + col[b / 2], 0, 0);
        }
      });
    } else {
      constexpr bool residual = mode == kResidual || mode == kGeneral;
      const bool hr = residual && p.res, hp = mode == kGeneral && p.pre[0], hb = mode == kGeneral && p.bias;
      const auto rr = rows_rsrc(hr ? p.res : p.y[0], hr ? p.ldr : 0, it.m0, hr ? rows : 1, hr ? p.N : 0);
      const auto pr = rows_rsrc(hp ? p.pre[0] : p.y[0], hp ? p.ldpre[0] : 0, it.m0, hp ? rows : 1, hp ? p.N : 0);
      const auto br = __builtin_amdgcn_make_buffer_rsrc((void*)uni(hb ? p.bias : p.y[0]), 0,
                                                        uni(hb ? p.N * 2 : 0), 0x00020000);
      const uint32_t ro = hr ? (uint32_t)(row * p.ldr * 2) : 0;
      const int rstep = hr ? 16 * p.ldr * 2 : 0;
      const uint32_t po = hp ? (uint32_t)(row * p.ldpre[0] * 2) : 0;
      const int pstep = hp ? 16 * p.ldpre[0] * 2 : 0;
      u32x4 rv[2][NO / 2], bv[NO / 2];  // the residual's rows, one row of blocks ahead
      if constexpr (mode == kGeneral) {
#pragma unroll
        for (int b = 0; b < NO / 2; ++b) bv[b] = __builtin_amdgcn_raw_buffer_load_b128(br, col[b], 0, 0);
      }
      // a row's or a column's scale: a lane's rows or columns of the tile
      float rsv[MB];
      F8 csv[NO / 2];
      if constexpr (mode == kScaled && LAY == kDx) {
        const auto r = __builtin_amdgcn_make_buffer_rsrc((void*)uni(p.rs), 0, uni(p.rs ? p.M * 4 : 0), 0x00020000);
#pragma unroll
        for (int a = 0; a < MB; ++a) {
          const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(r, (uint32_t)(it.m0 + row + 16 * a) * 4, 0, 0);
          rsv[a] = p.rs ? __builtin_bit_cast(float, v) : 1.f;
        }
      }
      if constexpr (mode == kScaled && LAY == kDw) {
        const auto r = __builtin_amdgcn_make_buffer_rsrc((void*)uni(p.cs + (it.out ? p.N : 0)), 0,
                                                         uni(p.cs ? p.N * 4 : 0), 0x00020000);
#pragma unroll
        for (int b = 0; b < NO / 2; ++b) {
          const uint32_t n = it.n0 + (wn * NO + 2 * b + (g & 1)) * 16 + 8 * (g >> 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, n * 4 + 16 * h, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t x = v[e];
              csv[b].v[4 * h + e] = p.cs ? __builtin_bit_cast(float, x) : 1.f;
            }
          }
        }
      }
      if constexpr (residual) {
#pragma unroll
        for (int b = 0; b < NO / 2; ++b)
          rv[0][b] = __builtin_amdgcn_raw_buffer_load_b128(rr, ro + col[b], 0, 0);
      }
      static_for<MB>([&](auto A) {
        constexpr int a = decltype(A)::value;
        take_row(a);
        if constexpr (residual) {
          if constexpr (a + 1 < MB) {
#pragma unroll
            for (int b = 0; b < NO / 2; ++b)
              rv[(a + 1) & 1][b] =
                  __builtin_amdgcn_raw_buffer_load_b128(rr, ro + (uint32_t)((a + 1) * rstep) + col[b], 0, 0);
          }
        }
#pragma unroll
        for (int b = 0; b < NO; b += 2) {
          F8 f = pair8(acc[a][b], acc[a][b + 1]);
          if constexpr (mode == kGeneral) {
            const F8 bias = widen8<DT>(bv[b / 2]);
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] += bias.v[e];
            __builtin_amdgcn_raw_buffer_store_b128(round8<DT>(f), pr, po + (uint32_t)(a * pstep) + col[b / 2], 0, 0);
            act8(p.act, f);
          }
          if constexpr (mode == kScaled) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] *= LAY == kDx ? rsv[a] : csv[b / 2].v[e];
          }
          if constexpr (residual) {
            const F8 r = widen8<DT>(rv[a & 1][b / 2]);
#pragma unroll
            for (int e = 0; e < 8; ++e) f.v[e] += r.v[e];
          }
          __builtin_amdgcn_raw_buffer_store_b128(round8<DT>(f), yr, yo + (uint32_t)(a * ystep) + col[b / 2], 0, 0);
        }
      });
    }
  };
  auto finish = [&](const Item& it) SA_INLINE {
    acc_wait();
    if (split) finish_parts(it);
    else finish_rows(it);
    clear();
  };

  clear();
  if (steps > 0) {
    place();
    static_for<NS>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (j > 0) {
        advance();
        op.next();
        oq.next();
        turn();
      }
      rp = op.rsrc(left);
      rq = oq.rsrc(left);
      settle();
      asm volatile("s_nop 4" ::: "memory");
      static_for<(j < NS - 1 ? L : J1)>([&](auto I) {
        set_one(decltype(I)::value, j);
        asm volatile("s_nop 0" ::: "memory");
        load_one(decltype(I)::value);
      });
    });
    stage_barrier<(NS - 2) * L + J1, 0>();
    static_for<R>([&](auto I) { read_one(decltype(I)::value, 0, 0); });
  }
  int pbuf = NS - 1, buf = 0;
  for (int cur = begin; cur < end;) {
    const Item it = item_at(cur);
    cur = it.next;
    for (int t = it.s0; t < it.s1; ++t) {
      const int nbuf = buf + 1 == NS ? 0 : buf + 1;
      half(std::integral_constant<int, 0>{}, pbuf, buf, nbuf);
      half(std::integral_constant<int, 1>{}, pbuf, buf, nbuf);
      pbuf = buf;
      buf = nbuf;
    }
    finish(it);
  }
  stage_barrier<0, 0>();  // no load may land in LDS after the workgroup's end
}

template <int DT, int LAY, bool GATED, int EPI, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(256, 1) void k_lin(LinP p) {
  __shared__ __align__(16) uint8_t S[lin_lds<LAY, BM, BN, NS>()];
  lin_run<DT, LAY, GATED, EPI, BM, BN, WM, WN, NS>(p, blockIdx.x, gridDim.x, S);
}

// Small gradients: dx (the first `first` workgroups) and dW in one launch, a
// workgroup of each on a CU.  One after the other, each leaves the chip
// waiting for its own latency (the whole backward call of 509 rows 1024 ->
// 4096: 34.8 -> 28.1 us, gated with 300 rows 39.5 -> 33.8, both before fp16's
// scales).
template <int DT, int XM>
__global__ __launch_bounds__(256, 1) void k_lin_pair(LinP x, LinP w, int first) {
  constexpr int NX = XM == 64 ? 3 : 2, WX = XM == 64 ? 1 : 2;
  constexpr int EPI = DT == SA_F16 ? kScaled : kPlain;
  constexpr int lx = lin_lds<kDx, XM, 128, NX>(), lw = lin_lds<kDw, 128, 128, 2>();
  __shared__ __align__(16) uint8_t S[lx > lw ? lx : lw];
  if ((int)blockIdx.x < first)
    lin_run<DT, kDx, false, EPI, XM, 128, WX, 4 / WX, NX>(x, blockIdx.x, first, S);
  else
    lin_run<DT, kDw, false, EPI, 128, 128, 2, 2, 2>(w, (int)blockIdx.x - first,
                                                       (int)gridDim.x - first, S);
}

// Sums the shares' partials of each tile (2^lbm x 2^lbn outputs) and finishes the outputs, 8
// columns of a row per thread, or (groups = kChains, for few outputs) one of
// their chains per thread.
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void k_lin_reduce(LinP p, int groups, int lbm, int lbn) {
  __shared__ float part[256][GATED ? 17 : 9];  // odd rows: lanes in different banks
  const uint32_t n8 = p.N / 8, rows = p.M * p.outs;  // few tiles: 32 bits hold their sizes
  const int per = 256 / groups;
  const int o = (int)threadIdx.x % per, k = (int)threadIdx.x / per;
  const uint32_t id = blockIdx.x * per + o;
  const bool in = id < rows * n8;
  const uint32_t mo = in ? id / n8 : 0;
  const int n = in ? (int)(id - mo * n8) * 8 : 0;
  const int out = mo >= (uint32_t)p.M;
  const int row = (int)(mo - (out ? p.M : 0));
  F8 f[kChains] = {}, u[kChains] = {};
  if (in) {
    const int mt = (p.M + (1 << lbm) - 1) >> lbm, nt1 = (p.N + (1 << lbn) - 1) >> lbn;
    const uint32_t steps = (uint32_t)((p.K + BK - 1) / BK * p.segs), TS = mt * nt1 * p.outs * steps;
    const uint32_t at = (uint32_t)(((n >> lbn) + out * nt1) * mt + (row >> lbm)) * steps;
    const int slots = share_of(at + steps - 1, TS, p.split) - share_of(at, TS, p.split) + 1;
    auto add = [&](int s, F8& fc, F8& uc) {
      const float* q = p.part + ((int64_t)s * rows + mo) * (GATED ? 2 : 1) * p.N + n;
      add_part(fc, q);
      if constexpr (GATED) add_part(uc, q + p.N);
    };
    if (groups > 1) {  // this thread's chain
#pragma unroll 4
      for (int s = k; s < slots; s += kChains) add(s, f[0], u[0]);
    } else {
      for (int s = 0; s < slots; s += kChains) {
#pragma unroll
        for (int c = 0; c < kChains; ++c) {
          if (s + c >= slots) break;
          add(s + c, f[c], u[c]);
        }
      }
    }
  }
  if (groups > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      part[threadIdx.x][e] = f[0].v[e];
      if constexpr (GATED) part[threadIdx.x][8 + e] = u[0].v[e];
    }
    __syncthreads();
    if (k > 0) return;
#pragma unroll
    for (int c = 1; c < kChains; ++c) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[c].v[e] = part[c * per + o][e];
        if constexpr (GATED) u[c].v[e] = part[c * per + o][8 + e];
      }
    }
  }
  if (!in) return;
  if constexpr (GATED) {
    finish_gated<DT>(p, row, n, add_chains(f), add_chains(u));
  } else {
    finish_linear<DT, DT == SA_F16>(p, out, row, n, add_chains(f));
  }
}

// ---- the gradients' elementwise half --------------------------------------------
// d = dy * act'(pre) (linear) or dg = dh u act'(g), du = dh act(g) (gated),
// rounded to the element type for the products, and per strip of rows the
// fp32 column sums of the unrounded d (dbias).  Bound by memory: reads 2 (3)
// values and writes 1 (2) per entry.  A wave takes 512 columns (8 per lane:
// 16-byte accesses) of a quarter of a strip, kDactRows rows at a time so that
// their loads are in flight together; the four waves' sums meet in LDS.
//
// fp16 holds 2^-24 to 65504, d up to 2^49 and far smaller ones, where dx and
// dW may well be ordinary numbers.  So its rows (for dx) and columns (for dW)
// whose largest |d| m lies outside [2^-8, 2^15) are scaled to [2^14, 2^15) by
// a power of two, which the products' epilogues undo in fp32.  A d is rounded
// to half a step or, where it is small, to 2^-17 m (half a subnormal step) at
// worst.  Three launches, as a scale has to be known before a value is
// rounded: kFind writes the unscaled d and the largest |d| of every row and
// column of its block; k_lin_scales finds the scales; kApply returns at once
// if all are 1 (a loss scale keeps d there), or else evaluates d again and
// writes it by rows' scales (another buffer, which dx then reads) and by
// columns' (over the unscaled d).  4096 x 11008, linear (gated): kNone 58 us
// (80), kFind 62 (84), k_lin_scales 5, kApply 5 where it returns at once, else
// 71 (124); 509 x 4096 (gated 300): kFind 7, scales 2-4, kApply 1.6, else 7 (9).
enum Scaling { kNone = 0, kFind = 1, kApply = 2 };
struct DactP {
  const uint16_t *dy, *a, *b;  // a: pre or g; b: u
  int64_t lddy, lda, ldb;
  uint16_t *d0, *d1;           // [T][N] (linear without an activation: none, sums only)
  float* sums;                 // [strips][N] or NULL
  int64_t T, N, strip;
  int act;
  // scaling (fp16); with dx (dW) not wanted the rows' (columns') are NULL
  uint16_t *e0, *e1;           // [T][N]: d by rows' scales
  float *rmax, *cmax;          // [T][column blocks], [strips][outs][N]: largest |d|
  float *rs, *cs;              // [T], [outs][N]: the scales' reciprocals
  uint32_t* scaled;            // not 0: some scale is not 1
};
// The reciprocal of the scale for values up to m.  Rows and columns with Inf
// or NaN have no use for one: all they reach is Inf or NaN.
__device__ __forceinline__ float unscale_of(float m) {
  const int e = (int)(__builtin_bit_cast(uint32_t, m) >> 23) - 127;
  if (m == 0.f || e > 127 || (e >= -8 && e < 15)) return 1.f;
  const int by = 14 - e < 64 ? 14 - e : 64;  // 2^-78 reaches no fp16 output; -35 at least
  return __builtin_bit_cast(float, (uint32_t)(127 - by) << 23);
}
__device__ __forceinline__ float reciprocal_pow2(float u) {
  return __builtin_bit_cast(float, (254u << 23) - __builtin_bit_cast(uint32_t, u));
}
// The largest of the wave's values, none of them negative, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  auto shifted = [&](auto C) {
    const int x = __builtin_bit_cast(int, v);
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, x, decltype(C)::value, 0xf, 0xf, true)));
  };
  shifted(std::integral_constant<int, 0x111>{});  // row_shr:1
  shifted(std::integral_constant<int, 0x112>{});
  shifted(std::integral_constant<int, 0x114>{});
  shifted(std::integral_constant<int, 0x118>{});
  const int x = __builtin_bit_cast(int, v);
  const int r0 = __builtin_amdgcn_readlane(x, 15), r1 = __builtin_amdgcn_readlane(x, 31);
  const int r2 = __builtin_amdgcn_readlane(x, 47), r3 = __builtin_amdgcn_readlane(x, 63);
  return fmaxf(fmaxf(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1)),
               fmaxf(__builtin_bit_cast(float, r2), __builtin_bit_cast(float, r3)));
}
struct DactLane {
  float sum[8];   // column sums
  float m0[8], m1[8];  // kFind: largest |d0|, |d1| of a column; kApply: the columns' scales
};
constexpr int kDactRows = 4;
// `in`: the lane's columns exist; if not it reads column 0 and writes nothing.
template <int DT, bool GATED, int ACT, int SCALING>
__device__ __forceinline__ void dact_rows(const DactP& p, int64_t n, bool in, int64_t t0, int64_t t1,
                                          DactLane& l) {
  constexpr bool map = GATED || ACT != SA_ACT_NONE;
  for (int64_t t = t0; t < t1; t += kDactRows) {
    u16x8 dy[kDactRows], a[kDactRows], b[kDactRows];
#pragma unroll
    for (int r = 0; r < kDactRows; ++r) {
      const int64_t tr = t + r < t1 ? t + r : t1 - 1;
      dy[r] = *reinterpret_cast<const u16x8*>(p.dy + tr * p.lddy + n);
      if constexpr (map) a[r] = *reinterpret_cast<const u16x8*>(p.a + tr * p.lda + n);
      if constexpr (GATED) b[r] = *reinterpret_cast<const u16x8*>(p.b + tr * p.ldb + n);
    }
#pragma unroll
    for (int r = 0; r < kDactRows; ++r) {
      if (t + r >= t1) break;
      u16x8 o0, o1, q0, q1;
      float most = 0.f, by = 1.f;
      if constexpr (SCALING == kApply) by = p.rs ? reciprocal_pow2(p.rs[t + r]) : 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = to_f<DT>(dy[r][e]);
        float f = 0.f, df = 1.f;
        if constexpr (map) act_both<ACT>(to_f<DT>(a[r][e]), f, df);
        float x, y = 0.f;
        if constexpr (GATED) {
          x = v * to_f<DT>(b[r][e]) * df;
          y = v * f;
        } else {
          x = v * df;
          l.sum[e] += x;
        }
        if constexpr (SCALING == kFind) {
          l.m0[e] = fmaxf(l.m0[e], fabsf(x));
          most = fmaxf(most, fabsf(x));
          if constexpr (GATED) {
            l.m1[e] = fmaxf(l.m1[e], fabsf(y));
            most = fmaxf(most, fabsf(y));
          }
        }
        if constexpr (SCALING == kApply) {
          q0[e] = from_f<DT>(x * by);
          x *= l.m0[e];
          if constexpr (GATED) {
            q1[e] = from_f<DT>(y * by);
            y *= l.m1[e];
          }
        }
        o0[e] = from_f<DT>(x);
        if constexpr (GATED) o1[e] = from_f<DT>(y);
      }
      const int64_t at = (t + r) * p.N + n;
      if (in && (SCALING != kApply || p.cs)) {
        if constexpr (map) *reinterpret_cast<u16x8*>(p.d0 + at) = o0;
        if constexpr (GATED) *reinterpret_cast<u16x8*>(p.d1 + at) = o1;
      }
      if constexpr (SCALING == kFind) {
        most = wave_max(in ? most : 0.f);
        if (lane_id() == 0) p.rmax[(t + r) * gridDim.x + blockIdx.x] = most;
      }
      if constexpr (SCALING == kApply) {
        if (in && p.rs) {
          *reinterpret_cast<u16x8*>(p.e0 + at) = q0;
          if constexpr (GATED) *reinterpret_cast<u16x8*>(p.e1 + at) = q1;
        }
      }
    }
  }
}
template <int DT, bool GATED, int SCALING>
__global__ __launch_bounds__(256) void k_lin_dact(DactP p) {
  static_assert(SCALING == kNone || DT == SA_F16, "bf16 has fp32's range");
  __shared__ float part[4][64][9];  // 9: the lanes' rows in different banks
  if constexpr (SCALING == kApply) {
    if (!*p.scaled) return;
  }
  if constexpr (SCALING == kFind) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.scaled = 0;
  }
  const int lane = lane_id(), w = (int)threadIdx.x / kWave;
  int64_t n = ((int64_t)blockIdx.x * 64 + lane) * 8;
  const bool in = n < p.N;
  n = in ? n : 0;
  const int64_t quarter = (p.strip + 3) / 4;
  const int64_t s0 = blockIdx.y * p.strip, send = s0 + p.strip < p.T ? s0 + p.strip : p.T;
  const int64_t t0 = s0 + w * quarter, t1 = t0 + quarter < send ? t0 + quarter : send;
  DactLane l;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    l.sum[e] = 0.f;
    l.m0[e] = SCALING == kApply && p.cs ? reciprocal_pow2(p.cs[n + e]) : 0.f;
    l.m1[e] = SCALING == kApply && GATED && p.cs ? reciprocal_pow2(p.cs[p.N + n + e]) : 0.f;
  }
  with_act(p.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    // the host scales only what an activation or a gate has changed
    if constexpr (SCALING == kNone || GATED || ACT != SA_ACT_NONE)
      dact_rows<DT, GATED, ACT, SCALING>(p, n, in, t0, t1, l);
  });
  // 512 columns by 256 threads, the waves' values in order
  auto columns = [&](const float (&v)[8], float* out, auto&& join) SA_INLINE {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) part[w][lane][e] = v[e];
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = h * 256 + (int)threadIdx.x;
      const int64_t col = (int64_t)blockIdx.x * 512 + c;
      if (col < p.N)
        out[col] = join(join(part[0][c / 8][c % 8], part[1][c / 8][c % 8]),
                        join(part[2][c / 8][c % 8], part[3][c / 8][c % 8]));
    }
  };
  if constexpr (SCALING != kApply && !GATED) {
    if (p.sums) columns(l.sum, p.sums + blockIdx.y * p.N, [](float a, float b) { return a + b; });
  }
  if constexpr (SCALING == kFind) {
    constexpr int outs = GATED ? 2 : 1;
    auto larger = [](float a, float b) { return fmaxf(a, b); };
    columns(l.m0, p.cmax + (int64_t)blockIdx.y * outs * p.N, larger);
    if constexpr (GATED) columns(l.m1, p.cmax + ((int64_t)blockIdx.y * outs + 1) * p.N, larger);
  }
}
// The scales of the rows and columns of d, and dbias.  The first `cblocks`
// workgroups take 64 of the C columns each (wave w strips w, w + 4, ...; sums
// in k_lin_colsum's order), the others a row per wave, of `blocks` maxima.  A
// workgroup stores the flag once, within its XCD: stores of every row and
// column through to memory queued at its address (small d, 509 x 4096: 20 us).
template <bool SUMS>
__global__ __launch_bounds__(256) void k_lin_scales(DactP p, int64_t strips, int64_t C, int cblocks,
                                                    int blocks, uint16_t* dbias) {
  __shared__ float part[4][64], most[4][64];
  const int lane = lane_id(), w = (int)threadIdx.x / kWave;
  bool scaled = false;
  if ((int)blockIdx.x < cblocks) {
    const int64_t n = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f, m = 0.f;
    if (n < C) {
      for (int64_t i = w; i < strips; i += 32) {
        float v[8], q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t k = i + 4 * j < strips ? i + 4 * j : i;
          v[j] = p.cmax[k * C + n];
          q[j] = SUMS ? p.sums[k * C + n] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m = fmaxf(m, v[j]);
          if (SUMS && i + 4 * j < strips) s += q[j];
        }
      }
    }
    part[w][lane] = s;
    most[w][lane] = m;
    __syncthreads();
    if (w == 0 && n < C) {
      if (SUMS)
        dbias[n] = from_f<SA_F16>((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
      if (p.cs) {
        const float u = unscale_of(fmaxf(fmaxf(most[0][lane], most[1][lane]), fmaxf(most[2][lane], most[3][lane])));
        p.cs[n] = u;
        scaled = u != 1.f;
      }
    }
  } else {
    const int64_t step = 4 * (int64_t)((int)gridDim.x - cblocks);
    for (int64_t t = 4 * (int64_t)((int)blockIdx.x - cblocks) + w; t < p.T; t += step) {
      float m = 0.f;
      for (int b = lane; b < blocks; b += 64) m = fmaxf(m, p.rmax[t * blocks + b]);
      const float u = unscale_of(wave_max(m));
      if (lane == 0) p.rs[t] = u;
      scaled |= u != 1.f;
    }
  }
  // read by later launches only: a store that may stay in this XCD's L2
  if (__syncthreads_or(scaled) && threadIdx.x == 0)
    __hip_atomic_store(p.scaled, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
// dbias[n]: the strips' sums.  64 columns per workgroup; wave w adds strips
// w, w + 4, ..., then the waves' four sums are added in order.
template <int DT>
__global__ __launch_bounds__(256) void k_lin_colsum(const float* sums, int64_t strips, int64_t N,
                                                    uint16_t* out) {
  __shared__ float part[4][64];
  const int lane = lane_id(), w = (int)threadIdx.x / kWave;
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int64_t i = w; i < strips; i += 4) s += sums[i * N + n];
  }
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < N)
    out[n] = from_f<DT>((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
}

// ---- plans -----------------------------------------------------------------------
constexpr int64_t kCus = 256;  // compute units of an MI355X

// The compiled tiles: rows and columns (of g and of u each: 128 at most),
// and LDS stages.
constexpr int kTiles = 6;
constexpr int kTileM[kTiles] = {256, 128, 64, 32, 16, 256}, kTileN[kTiles] = {256, 128, 128, 128, 128, 192};
constexpr int kNarrow = 5;  // 256 x 192: whole tiles of plain products only, for another tile count
int g_lin_tile = -1, g_lin_split = -1;  // overrides (linear_set_tuning)

struct Plan {
  int tile, split;  // split: shares, 0 for whole tiles
  int64_t tiles;
};

int64_t tiles_of(int tile, bool gated, int64_t M, int64_t N, int64_t outs) {
  const int64_t bn = gated ? 128 : kTileN[tile];
  return ((M + kTileM[tile] - 1) / kTileM[tile]) * ((N + bn - 1) / bn) * outs;
}

// Largest number of shares that hold part of one tile.
int64_t slots_of(const Plan& pl, int64_t steps) {
  int64_t most = 0;
  for (int64_t t = 0; t < pl.tiles; ++t) {
    const uint32_t at = (uint32_t)(t * steps), TS = (uint32_t)(pl.tiles * steps);
    const int64_t n = share_of(at + (uint32_t)steps - 1, TS, pl.split) - share_of(at, TS, pl.split) + 1;
    most = n > most ? n : most;
  }
  return most;
}

// The tile and split with the smallest estimated time.  Per tile: a step's
// time with one workgroup on a CU (latency) and each workgroup's part of it
// with two (throughput; gated small tiles run alone), in us, measured over
// sweeps of tiles and splits at 1 to 1000 rows; 4 us per round of workgroups;
// 3 us for the reduction's launch (7 with 256 x 256 tiles) and the partials'
// bytes at 4 TB/s; one row tile streams its weights at 26 GB/s per CU at most
// (gated: up to four share them at 40).  Over 180 random shapes (plain, gated,
// dx) the choice took 4 percent longer than the best of a sweep on average,
// but 7 to 13 at 33 to 64 rows and 14 for gated products of 17 to 32, where a
// second row tile of half the height can pay for reading the weights again
// (46 rows, gated 760 x 6584: 19.4 us against 12.7, the largest miss).
Plan lin_plan(int lay, bool gated, int64_t M, int64_t N, int64_t K, int segs, int outs) {
  static const double alone[2][kTiles] = {{1.45, 0.60, 0.45, 0.40, 0.38, 1.15},
                                          {1.45, 0.95, 0.60, 0.55, 0.50, 0}};
  static const double paired[kTiles] = {0, 0.50, 0.36, 0.25, 0.22, 0};
  const int64_t steps = ((K + BK - 1) / BK) * segs;
  Plan best{0, 0, tiles_of(0, gated, M, N, outs)};
  double least = 1e30;
  for (int t = 0; t < kTiles; ++t) {
    if (lay == kDw && t > 1 && t != kNarrow) continue;
    if (t == kNarrow && gated) continue;
    const bool forced = g_lin_tile >= 0 && !(lay == kDw && g_lin_tile > 1 && g_lin_tile != kNarrow) &&
                        !(g_lin_tile == kNarrow && gated);
    if (forced && t != g_lin_tile) continue;
    // up to 64 rows in one row tile, more in tiles of 64 at least (see the
    // misses above)
    if (g_lin_tile < 0 && kTileM[t] < (M < 64 ? M : 64)) continue;
    const int64_t tiles = tiles_of(t, gated, M, N, outs);
    const bool pairs = t > 0 && t != kNarrow && !gated;
    double step = alone[gated][t];
    if (t > 0 && M <= (gated ? 4 : 1) * kTileM[t]) {
      const double stream = (gated ? 32768 : kTileN[t] * 128) / (M <= kTileM[t] ? 26e3 : 40e3) + 0.1 * step;
      step = stream > step ? stream : step;
    }
    // whole tiles
    const int64_t per = pairs ? 2 * kCus : kCus, full = tiles / per, rest = tiles % per;
    const double both = pairs && 2 * paired[t] > step ? 2 * paired[t] : step;
    double whole = full * (steps * (pairs ? both : step) + 4);
    if (rest) whole += steps * (rest > kCus ? both : step) + 4;
    if ((g_lin_split <= 0 || t == kNarrow) && whole < least) {
      least = whole;
      best = Plan{t, 0, tiles};
    }
    // split over one workgroup per CU, of four steps each at least (33 rows of
    // 4096 x 1024 10.1 us, two steps 10.9), down to two for 128 shares (8
    // rows of 880 x 3704, dx: 9.0, four 10.5) and one for 64
    const int64_t TS = tiles * steps;
    int64_t shares = TS / 4 < kCus ? TS / 4 : kCus;
    if (shares < 128) shares = TS / 2 < 128 ? TS / 2 : 128;
    if (shares < 64) shares = TS < 64 ? TS : 64;
    if (g_lin_split > 0) shares = g_lin_split < tiles * steps ? g_lin_split : tiles * steps;
    if (g_lin_split == 0 || t == kNarrow || shares < 1 || tiles * steps >= (1 << 22)) continue;
    while (shares & (shares - 1)) shares &= shares - 1;  // a power of two
    if (g_lin_split < 0 && (tiles >= shares || steps < 2)) continue;
    const double rows = M < kTileM[t] ? M : kTileM[t];
    const double parts = (shares + tiles) * rows * (gated ? 256 : kTileN[t]) * 8.0 / 4e6;
    const double time = (double)tiles * steps / shares * step + (t == 0 ? 11 : 7) + parts;
    if (time < least) {
      least = time;
      best = Plan{t, (int)shares, tiles};
    }
  }
  return best;
}

size_t part_bytes(const Plan& pl, int64_t M, int64_t N, int64_t K, int segs, int outs) {
  if (!pl.split || pl.tiles == 0) return 0;
  return (size_t)(slots_of(pl, (K + BK - 1) / BK * segs) * M * N * outs * 4);
}

template <int DT, int LAY, bool GATED, int EPI, int BM, int BN, int WM, int WN, int NS>
void launch_tile(const LinP& p, int64_t items, hipStream_t s) {  // items: shares or tiles
  constexpr int64_t most = kCus * (160 * 1024 / lin_lds<LAY, BM, BN, NS>());  // workgroups that run at once
  const dim3 grid((unsigned)(p.split || items < most ? items : most));
  hipLaunchKernelGGL((k_lin<DT, LAY, GATED, EPI, BM, BN, WM, WN, NS>), grid, dim3(256), 0, s, p);
}

template <int DT, bool GATED>
hipError_t launch_reduce(const LinP& p, const Plan& pl, hipStream_t s) {
  const int64_t octets = (int64_t)p.M * p.outs * (p.N / 8);
  // a thread per chain while that is less than a workgroup per CU
  const int groups = octets * kChains <= kCus * 256 ? kChains : 1;
  const int64_t n = (octets * groups + 255) / 256;
  if (n > 0x7fffffffLL) return hipErrorNotSupported;
  hipLaunchKernelGGL((k_lin_reduce<DT, GATED>), dim3((unsigned)n), dim3(256), 0, s, p, groups,
                     __builtin_ctz(kTileM[pl.tile]), __builtin_ctz(GATED ? 128 : kTileN[pl.tile]));
  return hipGetLastError();
}

template <int DT, int LAY, bool GATED>
hipError_t launch_lin(LinP p, void* ws, hipStream_t s) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  const Plan pl = lin_plan(LAY, GATED, p.M, p.N, p.K, p.segs, p.outs);
  if (pl.tiles > 0x7fffffffLL) return hipErrorNotSupported;
  const int64_t groups_of_work = pl.split ? pl.split : pl.tiles;
  p.split = pl.split;
  p.part = reinterpret_cast<float*>(ws);
  // One launch where a wave owns its columns, offsets fit 31 bits, and the
  // last wave of a tile adds its partials in at most 4 rounds of loads (one
  // row of 4096 x 4096: 13.5 -> 12.1 us; 33 rows of 4096 x 1024, 24 rounds:
  // 13.8 -> 22.8 us, so those take the second launch).
  const int64_t slots = pl.split ? pl.split / pl.tiles + 2 : 0;
  const int64_t rounds = ((p.M < kTileM[pl.tile] ? p.M : kTileM[pl.tile]) * 4 + 63) / 64 * ((slots + 2) / 4);
  if (!(LAY == kFwd && pl.split && pl.tile >= 2 && pl.tiles <= kTicketTiles && rounds <= 4 &&
        (int64_t)p.M * p.N * (GATED ? 2 : 1) * 4 * slots < 0x7fffffffLL))
    p.tickets = nullptr;
  constexpr int SB = GATED ? 256 : 128;
  constexpr int EPI = LAY == kFwd ? kGeneral : DT == SA_F16 ? kScaled : kPlain;
  if (pl.tile == 0) {
    // split products finish in k_lin_reduce
    if constexpr (LAY != kFwd)
      launch_tile<DT, LAY, GATED, EPI, 256, 256, 2, 2, 2>(p, groups_of_work, s);
    else if (pl.split ||
        (GATED ? !p.pre[0] : !p.bias && !p.pre[0] && p.act == SA_ACT_NONE && !p.res))
      launch_tile<DT, LAY, GATED, kPlain, 256, 256, 2, 2, 2>(p, groups_of_work, s);
    else if (!GATED && !p.bias && !p.pre[0] && p.act == SA_ACT_NONE)
      launch_tile<DT, LAY, GATED, GATED ? EPI : kResidual, 256, 256, 2, 2, 2>(p, groups_of_work, s);
    else
      launch_tile<DT, LAY, GATED, EPI, 256, 256, 2, 2, 2>(p, groups_of_work, s);
  } else if (pl.tile == kNarrow) {
    if constexpr (!GATED) launch_tile<DT, LAY, GATED, EPI, 256, 192, 2, 2, 2>(p, groups_of_work, s);
  } else if (pl.tile == 1) {
    launch_tile<DT, LAY, GATED, EPI, 128, SB, 2, 2, GATED ? 3 : 2>(p, groups_of_work, s);
  } else if constexpr (LAY != kDw) {
    if (pl.tile == 2) launch_tile<DT, LAY, GATED, EPI, 64, SB, 1, 4, 3>(p, groups_of_work, s);
    else if (pl.tile == 3) launch_tile<DT, LAY, GATED, EPI, 32, SB, 1, 4, GATED ? 4 : 3>(p, groups_of_work, s);
    else launch_tile<DT, LAY, GATED, EPI, 16, SB, 1, 4, 4>(p, groups_of_work, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !pl.split || p.tickets) return e;
  return launch_reduce<DT, GATED>(p, pl, s);
}

// dx and dW of one backward call; whichever is split has ws to itself when it runs.
template <int DT>
hipError_t launch_gradients(LinP x, LinP w, void* ws, hipStream_t s) {
  const Plan px = lin_plan(kDx, false, x.M, x.N, x.K, x.segs, x.outs);
  const Plan pw = lin_plan(kDw, false, w.M, w.N, w.K, w.segs, w.outs);
  const bool pair = px.tiles > 0 && (px.tile == 1 || px.tile == 2) && pw.tile == 1 && !pw.split &&
                    (px.split || px.tiles <= kCus) && pw.tiles <= 2 * kCus;
  if (!pair) {
    hipError_t e = launch_lin<DT, kDx, false>(x, ws, s);
    return e != hipSuccess ? e : launch_lin<DT, kDw, false>(w, ws, s);
  }
  x.split = px.split;
  x.part = reinterpret_cast<float*>(ws);
  w.split = 0;
  const int first = px.split ? px.split : (int)px.tiles;
  const dim3 grid((unsigned)(first + pw.tiles));
  if (px.tile == 2) hipLaunchKernelGGL((k_lin_pair<DT, 64>), grid, dim3(256), 0, s, x, w, first);
  else hipLaunchKernelGGL((k_lin_pair<DT, 128>), grid, dim3(256), 0, s, x, w, first);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !px.split ? e : launch_reduce<DT, false>(x, px, s);
}

// Rows per strip of the elementwise kernel (a workgroup's): 16 for small T
// (a latency-bound kernel wants workgroups), 64 from 2048 rows on (fewer
// partial sums), more where that would give over 1024 strips.
int64_t strip_rows(int64_t T) { return T < 2048 ? 16 : T <= 64 * 1024 ? 64 : (T + 1023) / 1024; }
int64_t strips_of(int64_t T) { return (T + strip_rows(T) - 1) / strip_rows(T); }

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

template <int DT>
hipError_t fwd_dt(const LinearCall& c, hipStream_t s) {
  LinP p{};
  p.p[0] = c.x;
  p.ldp = (int)c.ldx;
  p.q[0] = c.w[0];
  p.q[1] = c.w[1];
  p.ldq[0] = (int)c.ldw[0];
  p.ldq[1] = (int)c.ldw[1];
  p.M = (int)c.T;
  p.N = (int)c.d_out;
  p.K = (int)c.d_in;
  p.segs = p.outs = 1;
  p.act = c.act;
  p.bias = c.bias;
  p.res = c.res;
  p.ldr = (int)c.ldr;
  p.y[0] = c.y;
  p.ldy[0] = (int)c.ldy;
  for (int i = 0; i < 2; ++i) {
    p.pre[i] = c.pre[i];
    p.ldpre[i] = (int)c.ldpre[i];
  }
  p.tickets = static_cast<uint32_t*>(c.tickets);
  return c.gated ? launch_lin<DT, kFwd, true>(p, c.ws, s) : launch_lin<DT, kFwd, false>(p, c.ws, s);
}

// The backward calls' scratch, in order; the products' partial sums follow.
struct BwdScratch {
  bool map = false, scaled = false;  // d differs from dy; it is fp16
  size_t d[2] = {}, e[2] = {}, sums = 0, rmax = 0, cmax = 0, rs = 0, cs = 0, flag = 0, end = 0;
};
BwdScratch bwd_scratch(int dtype, bool gated, int64_t T, int64_t d_out, int act, bool dbias) {
  BwdScratch b;
  const int n = gated ? 2 : 1;
  const int64_t strips = strips_of(T), blocks = (d_out + 511) / 512;
  b.map = gated || act != SA_ACT_NONE;
  b.scaled = b.map && dtype == SA_F16;
  auto take = [&](int64_t bytes) {
    const size_t at = b.end;
    b.end += round256((size_t)bytes);
    return at;
  };
  for (int i = 0; i < n && b.map; ++i) b.d[i] = take(T * d_out * 2);
  if (dbias) b.sums = take(strips * d_out * 4);
  if (!b.scaled) return b;
  for (int i = 0; i < n; ++i) b.e[i] = take(T * d_out * 2);
  b.rmax = take(T * blocks * 4);
  b.cmax = take(strips * n * d_out * 4);
  b.rs = take(T * 4);
  b.cs = take(n * d_out * 4);
  b.flag = take(4);
  return b;
}

template <int DT>
hipError_t bwd_dt(const LinearCall& c, hipStream_t s) {
  char* ws = static_cast<char*>(c.ws);
  const BwdScratch b = bwd_scratch(DT, c.gated, c.T, c.d_out, c.act, c.dbias != nullptr);
  const int outs = c.gated ? 2 : 1;
  const uint16_t* d[2] = {c.dy, nullptr};
  int64_t ldd = c.lddy;
  if (b.map) {
    d[0] = reinterpret_cast<uint16_t*>(ws + b.d[0]);
    if (c.gated) d[1] = reinterpret_cast<uint16_t*>(ws + b.d[1]);
    ldd = c.d_out;
  }
  const bool scaled = b.scaled && c.T > 0 && (c.dx || c.dw[0]);
  const int64_t strips = strips_of(c.T);
  DactP a{};
  hipError_t e = hipSuccess;
  a.sums = c.dbias ? reinterpret_cast<float*>(ws + b.sums) : nullptr;
  if (c.T > 0 && (b.map || c.dbias)) {
    a.dy = c.dy;
    a.lddy = c.lddy;
    a.a = c.pre[0];
    a.lda = c.ldpre[0];
    a.b = c.pre[1];
    a.ldb = c.ldpre[1];
    a.d0 = b.map ? const_cast<uint16_t*>(d[0]) : nullptr;
    a.d1 = const_cast<uint16_t*>(d[1]);
    a.T = c.T;
    a.N = c.d_out;
    a.strip = strip_rows(c.T);
    a.act = c.act;
    const dim3 gr((unsigned)((c.d_out + 511) / 512), (unsigned)strips);
    if constexpr (DT == SA_F16) {
      if (scaled) {
        a.rmax = reinterpret_cast<float*>(ws + b.rmax);
        a.cmax = reinterpret_cast<float*>(ws + b.cmax);
        a.scaled = reinterpret_cast<uint32_t*>(ws + b.flag);
        if (c.dx) {
          a.rs = reinterpret_cast<float*>(ws + b.rs);
          a.e0 = reinterpret_cast<uint16_t*>(ws + b.e[0]);
          a.e1 = c.gated ? reinterpret_cast<uint16_t*>(ws + b.e[1]) : nullptr;
        }
        if (c.dw[0]) a.cs = reinterpret_cast<float*>(ws + b.cs);
        if (c.gated) hipLaunchKernelGGL((k_lin_dact<DT, true, kFind>), gr, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((k_lin_dact<DT, false, kFind>), gr, dim3(256), 0, s, a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t C = outs * c.d_out;
        const int cblocks = a.cs || c.dbias ? (int)((C + 63) / 64) : 0;
        const int64_t rows = c.dx ? (c.T + 3) / 4 : 0;
        const dim3 gs((unsigned)(cblocks + (rows < 1024 ? rows : 1024)));
        if (c.dbias) hipLaunchKernelGGL((k_lin_scales<true>), gs, dim3(256), 0, s, a, strips, C, cblocks, (int)gr.x, c.dbias);
        else hipLaunchKernelGGL((k_lin_scales<false>), gs, dim3(256), 0, s, a, strips, C, cblocks, (int)gr.x, c.dbias);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (c.gated) hipLaunchKernelGGL((k_lin_dact<DT, true, kApply>), gr, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((k_lin_dact<DT, false, kApply>), gr, dim3(256), 0, s, a);
      }
    }
    if (!scaled) {
      if (c.gated) hipLaunchKernelGGL((k_lin_dact<DT, true, kNone>), gr, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((k_lin_dact<DT, false, kNone>), gr, dim3(256), 0, s, a);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (c.dbias && !scaled) {
    hipLaunchKernelGGL((k_lin_colsum<DT>), dim3((unsigned)((c.d_out + 63) / 64)), dim3(256), 0, s,
                       a.sums, strips, c.d_out, c.dbias);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  ws += b.end;
  LinP x{}, w{};
  x.p[0] = d[0];
  x.p[1] = d[1];
  x.ldp = (int)ldd;
  w.p[0] = c.x;
  w.ldp = (int)c.ldx;
  for (int i = 0; i < 2; ++i) {
    x.q[i] = c.w[i];
    x.ldq[i] = (int)c.ldw[i];
    w.q[i] = d[i];
    w.ldq[i] = (int)ldd;
    w.y[i] = c.dw[i];
    w.ldy[i] = (int)c.lddw[i];
  }
  x.y[0] = c.dx;
  x.ldy[0] = (int)c.lddx;
  x.M = (int)c.T;
  x.N = (int)c.d_in;
  x.K = (int)c.d_out;
  x.segs = c.gated ? 2 : 1;
  x.outs = 1;
  w.M = (int)c.d_in;
  w.N = (int)c.d_out;
  w.K = (int)c.T;
  w.segs = 1;
  w.outs = outs;
  if (scaled) {
    x.rs = a.rs;
    x.scaled = a.scaled;
    x.alt[0] = a.e0;
    x.alt[1] = a.e1;
    w.cs = a.cs;
  }
  if (c.dx && c.dw[0]) return launch_gradients<DT>(x, w, ws, s);
  if (c.dx) return launch_lin<DT, kDx, false>(x, ws, s);
  if (c.dw[0]) return launch_lin<DT, kDw, false>(w, ws, s);
  return e;
}

}  // namespace

size_t linear_workspace_bytes(bool gated, int64_t T, int64_t d_in, int64_t d_out) {
  return part_bytes(lin_plan(kFwd, gated, T, d_out, d_in, 1, 1), T, d_out, d_in, 1, gated ? 2 : 1);
}

size_t linear_backward_workspace_bytes(int dtype, bool gated, int64_t T, int64_t d_in, int64_t d_out,
                                       int act, bool dbias) {
  const int n = gated ? 2 : 1;
  const size_t b = bwd_scratch(dtype, gated, T, d_out, act, dbias).end;
  const size_t px = part_bytes(lin_plan(kDx, false, T, d_in, d_out, n, 1), T, d_in, d_out, n, 1);
  const size_t pw = part_bytes(lin_plan(kDw, false, d_in, d_out, T, 1, n), d_in, d_out, T, 1, n);
  return b + (px > pw ? px : pw);
}

int linear_set_tuning(int tile, int split) {
  if (tile < -1 || tile >= kTiles || split < -1 || split > 2 * kCus) return 1;
  g_lin_tile = tile;
  g_lin_split = split;
  return 0;
}

int linear_plan(int op, int64_t T, int64_t d_in, int64_t d_out, int* rows, int* cols, int* split,
                int64_t* tiles) {
  Plan pl;
  switch (op) {
    case SA_LINEAR_FORWARD: pl = lin_plan(kFwd, false, T, d_out, d_in, 1, 1); break;
    case SA_LINEAR_GATED: pl = lin_plan(kFwd, true, T, d_out, d_in, 1, 1); break;
    case SA_LINEAR_DX: pl = lin_plan(kDx, false, T, d_in, d_out, 1, 1); break;
    case SA_LINEAR_DW: pl = lin_plan(kDw, false, d_in, d_out, T, 1, 1); break;
    case SA_LINEAR_GATED_DX: pl = lin_plan(kDx, false, T, d_in, d_out, 2, 1); break;
    case SA_LINEAR_GATED_DW: pl = lin_plan(kDw, false, d_in, d_out, T, 1, 2); break;
    default: return 1;
  }
  *rows = kTileM[pl.tile];
  *cols = op == SA_LINEAR_GATED ? 128 : kTileN[pl.tile];
  *split = pl.split;
  *tiles = pl.tiles;
  return 0;
}

hipError_t launch_linear(const LinearCall& c, hipStream_t s) {
  return c.dtype == SA_F16 ? fwd_dt<SA_F16>(c, s) : fwd_dt<SA_BF16>(c, s);
}

hipError_t launch_linear_backward(const LinearCall& c, hipStream_t s) {
  return c.dtype == SA_F16 ? bwd_dt<SA_F16>(c, s) : bwd_dt<SA_BF16>(c, s);
}

}  // namespace sa
