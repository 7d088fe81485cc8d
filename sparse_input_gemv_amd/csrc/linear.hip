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
// Every product is one kernel, k_lin<DT, LAY, ...>: C[m][n] = sum_k P[m][k]
// Q[k][n] for a row operand P and a column operand Q, each stored with k
// contiguous ("KC") or with m or n contiguous ("NC"):
//   forward  P = x  [T][d_in]  KC,  Q = WT [d_in][d_out] NC;
//   dx       P = d  [T][d_out] KC,  Q = WT, read as n = d_in, k = d_out: KC;
//   dWT      P = x, read as m = d_in, k = T: NC,  Q = d [T][d_out]: NC.
#include <hip/hip_runtime.h>

#include "../../include/sparse_act.h"
#include "common.hpp"
#include "launch.hpp"

namespace sa {
namespace {

typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
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
template <int DT>
__device__ __forceinline__ f4v mfma16(s8v a, s8v b, f4v c) {
  if constexpr (DT == SA_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a),
                                                   __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
}

// ---- activations and their slopes (fp32) -------------------------------------
// sigma(z) = 1 / (1 + e^-z).  gelu's normal distribution function goes
// through erfc, which keeps its relative accuracy in the lower tail.
constexpr float kTanhA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}
__device__ __forceinline__ float act_value(int act, float v) {
  switch (act) {
    case SA_ACT_RELU: return v > 0.f ? v : 0.f;
    case SA_ACT_RELU2: return v > 0.f ? v * v : 0.f;
    case SA_ACT_SILU: return v * sigmoid(v);
    case SA_ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case SA_ACT_GELU_TANH: return v * sigmoid(2.f * kTanhA * (v + kTanhB * v * v * v));
    default: return v;
  }
}
__device__ __forceinline__ float act_slope(int act, float v) {
  switch (act) {
    case SA_ACT_RELU: return v > 0.f ? 1.f : 0.f;
    case SA_ACT_RELU2: return v > 0.f ? 2.f * v : 0.f;
    case SA_ACT_SILU: {
      const float s = sigmoid(v);
      return s * (1.f + v * (1.f - s));
    }
    case SA_ACT_GELU:
      return 0.5f * erfcf(-0.70710678118654752f * v) +
             v * 0.3989422804014327f * __expf(-0.5f * v * v);
    case SA_ACT_GELU_TANH: {
      const float s = sigmoid(2.f * kTanhA * (v + kTanhB * v * v * v));
      return s + 2.f * kTanhA * v * s * (1.f - s) * (1.f + 3.f * kTanhB * v * v);
    }
    default: return 1.f;
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
__device__ __forceinline__ i4v make_rsrc(const void* base, int64_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  if (bytes < 0) bytes = 0;
  if (bytes > 0x7fffffffLL) bytes = 0x7fffffffLL;
  i4v r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu));
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}
constexpr uint32_t kOutOfRange = 0x80000000u;  // past every resource
__device__ __forceinline__ void load_lds16(uint32_t voff, i4v rsrc, uint32_t lds) {
  asm volatile(
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, 0 offen lds"
      :
      : "v"(voff), "s"(rsrc), "{m0}"(lds)
      : "memory");
}

// Waits until at most VM loads and no LDS reads are outstanding, then the
// workgroup barrier.  s_waitcnt encoding: vmcnt bits 3:0 and 15:14, expcnt
// 6:4 (7: no wait), lgkmcnt 11:8.
template <int VM>
__device__ __forceinline__ void stage_barrier() {
  static_assert(VM >= 0 && VM < 64, "vmcnt range");
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
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

#define SA_LDS(T, a) ((const __attribute__((address_space(3))) T*)(uintptr_t)(a))

__device__ __forceinline__ s8v read_kc(uint32_t a) { return *SA_LDS(s8v, a); }
__device__ __forceinline__ s8v read_nc(uint32_t a) {
  typedef __attribute__((address_space(3))) s4v* lp;
  const s4v q0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)a);
  const s4v q1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)(a + 4 * 256));
  return s8v{q0[0], q0[1], q0[2], q0[3], q1[0], q1[1], q1[2], q1[3]};
}

enum Layout { kFwd = 0, kDx = 1, kDw = 2 };

struct LinP {
  const uint16_t* p[2];  // row operand (per K segment)
  const uint16_t* q[2];  // column operand (per K segment, gated half or output)
  int64_t ldp, ldq[2];
  int64_t M, N, K;       // K per segment
  int segs;              // K segments (dx of the gated pair: 2)
  int outs;              // outputs side by side (dW of the gated pair: 2)
  int slices;            // split of the K steps over workgroups
  float* part;           // [slices][M][N * (gated ? 2 : 1)] when slices > 1
  // epilogue
  int act;
  const uint16_t* bias;
  const uint16_t* res;
  int64_t ldr;
  uint16_t* y[2];        // output (per outs)
  int64_t ldy[2];
  uint16_t* pre[2];      // pre-activation, or g and u
  int64_t ldpre[2];
};

template <int DT>
__device__ __forceinline__ void store4(uint16_t* p, f4v v) {
  u16x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = from_f<DT>(v[i]);
  *reinterpret_cast<u16x4*>(p) = o;
}

// Four outputs of row m from column n on (all within N).
template <int DT>
__device__ __forceinline__ void finish_linear(const LinP& p, int o, int64_t m, int64_t n, f4v v) {
  if (p.bias) {
    const u16x4 b = *reinterpret_cast<const u16x4*>(p.bias + n);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += to_f<DT>(b[i]);
  }
  if (p.pre[0]) store4<DT>(p.pre[0] + m * p.ldpre[0] + n, v);
  if (p.act != SA_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_value(p.act, v[i]);
  }
  if (p.res) {
    const u16x4 r = *reinterpret_cast<const u16x4*>(p.res + m * p.ldr + n);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += to_f<DT>(r[i]);
  }
  store4<DT>(p.y[o] + m * p.ldy[o] + n, v);
}
template <int DT>
__device__ __forceinline__ void finish_gated(const LinP& p, int64_t m, int64_t n, f4v g, f4v u) {
  if (p.pre[0]) {
    store4<DT>(p.pre[0] + m * p.ldpre[0] + n, g);
    store4<DT>(p.pre[1] + m * p.ldpre[1] + n, u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = act_value(p.act, g[i]) * u[i];
  store4<DT>(p.y[0] + m * p.ldy[0] + n, g);
}

// The tile of workgroup b: the hardware deals workgroups over the 8 XCDs in
// turn, so each XCD takes a contiguous run of a grouped order (kGroupM row
// tiles across all column tiles); tiles that run together on one XCD share
// their operands in its L2.  A bijection.
constexpr int kGroupM = 4;
__device__ __forceinline__ void tile_of(int64_t b, int64_t total, int64_t mt, int64_t nt,
                                        int64_t& m, int64_t& n, int64_t& slice) {
  const int64_t x = b % 8, l = b / 8;
  const int64_t per = total / 8, rem = total % 8;
  int64_t t = x * per + (x < rem ? x : rem) + l;
  slice = t / (mt * nt);
  t %= mt * nt;
  const int64_t gsz = kGroupM * nt;
  const int64_t first = (t / gsz) * kGroupM;
  const int64_t gm = (mt - first < kGroupM) ? mt - first : kGroupM;
  m = first + (t % gsz) % gm;
  n = (t % gsz) / gm;
}

// One operand's tile: R rows (KC) or columns (NC) by 64 k, loaded by four
// waves with I instructions of 1 KB each.
template <bool NC, int R>
struct Operand {
  static constexpr int kRows = NC ? R : (R < 32 ? 32 : R);
  static constexpr int kBytes = kRows * BK * 2;
  static constexpr int I = kBytes / 1024 / 4;
  static_assert(!NC || R % 128 == 0, "NC tiles come in halves of 128 columns");
  static_assert(I >= 1, "one load per wave at least");
  uint32_t voff[I];
  __device__ __forceinline__ void init(int w, int64_t ld) {
    const int lane = lane_id();
#pragma unroll
    for (int j = 0; j < I; ++j) {
      const int id = w * I + j;
      if constexpr (NC) {
        const int k = (id % 16) * 4 + lane / 16;
        const int c = (lane % 16) ^ swz_nc(k);
        voff[j] = (uint32_t)(k * ld * 2 + c * 16);
      } else {
        const int r = id * 8 + lane / 8;
        const int c = (lane % 8) ^ swz_kc(r);
        voff[j] = (uint32_t)(r * ld * 2 + c * 16);
      }
    }
  }
  // K step starting at k0 (k0 >= K: zeros) of the operand whose tile starts
  // at row or column r0 of `rows` (KC: rows; NC: columns).
  __device__ __forceinline__ void issue(const uint16_t* base, int64_t ld, int64_t r0, int64_t rows,
                                        int64_t k0, int64_t K, uint32_t lds, int w) const {
    if constexpr (NC) {
      // the wave's loads lie in one half tile
      const int64_t c0 = r0 + 128 * ((w * I) / 16);
      int64_t left = K - k0;
      if (left > BK) left = BK;
      const int64_t bytes = (left > 0 && c0 < rows) ? ((left - 1) * ld + (rows - c0)) * 2 : 0;
      const i4v rs = make_rsrc(base + k0 * ld + c0, bytes);
#pragma unroll
      for (int j = 0; j < I; ++j) load_lds16(voff[j], rs, lds + (w * I + j) * 1024);
    } else {
      int64_t left = rows - r0;
      if (left > R) left = R;
      const int64_t bytes = (left > 0 && k0 < K) ? ((left - 1) * ld + (K - k0)) * 2 : 0;
      const i4v rs = make_rsrc(base + r0 * ld + k0, bytes);
      if (K - k0 >= BK) {
#pragma unroll
        for (int j = 0; j < I; ++j) load_lds16(voff[j], rs, lds + (w * I + j) * 1024);
      } else {
        // the row's end lies inside the step: chunks past it are zeros, not
        // the next row
        const int lane = lane_id();
#pragma unroll
        for (int j = 0; j < I; ++j) {
          const int r = (w * I + j) * 8 + lane / 8;
          const int c = (lane % 8) ^ swz_kc(r);
          load_lds16(k0 + 8 * c < K ? voff[j] : kOutOfRange, rs, lds + (w * I + j) * 1024);
        }
      }
    }
  }
};

// C tile of BM x BN (gated: BN / 2 columns of g and of u), 256 threads as WM
// x WN waves.  The K loop steps through NS LDS stages; operands are double
// buffered in registers by half steps of 32 k: while the MFMAs of one half
// run, the reads of the next half are in flight.  One barrier per step, in
// its middle: every wave has then read all of stage t, so its buffer takes
// the loads of stage t + NS; and stage t + 1 is complete.  Loads past the
// last step read zeros, so the load count per step never changes.
template <int DT, int LAY, bool GATED, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(256, 1) void k_lin(LinP p) {
  constexpr bool PNC = LAY == kDw, QNC = LAY != kDx;
  constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
  static_assert(WM * WN == 4 && MB >= 1 && NB >= 1, "four waves");
  using OP = Operand<PNC, BM>;
  using OQ = Operand<QNC, BN>;
  constexpr int L = OP::I + OQ::I;
  constexpr int kStage = OP::kBytes + OQ::kBytes;
  __shared__ __align__(16) uint8_t S[NS * kStage];
  const uint32_t lp = lds_addr(S), lq = lp + NS * OP::kBytes;

  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wm = w / WN, wn = w % WN;
  constexpr int BNO = GATED ? BN / 2 : BN;  // output columns per tile
  const int64_t mt = (p.M + BM - 1) / BM, nt1 = (p.N + BNO - 1) / BNO;
  const int64_t nt = nt1 * p.outs;
  int64_t mi, ni, slice;
  tile_of(blockIdx.x, gridDim.x, mt, nt, mi, ni, slice);
  const int out = ni >= nt1;
  const int64_t m0 = mi * BM, n0 = (ni - (out ? nt1 : 0)) * BNO;

  const int64_t ks = (p.K + BK - 1) / BK;  // steps per segment
  const int64_t steps = ks * p.segs;
  const int64_t s0 = steps * slice / p.slices, s1 = steps * (slice + 1) / p.slices;

  OP op;
  OQ oq;
  op.init(w, p.ldp);
  // gated: the waves of the second half load u's weight
  const int qh = GATED ? (w * OQ::I) / 16 : 0;
  oq.init(w, (LAY == kFwd && GATED && qh) ? p.ldq[1] : LAY == kDw ? p.ldq[out] : p.ldq[0]);
  auto issue = [&](int64_t t, int buf) {
    const int seg = t >= ks;
    const int64_t k0 = t < s1 ? (t - (seg ? ks : 0)) * BK : p.K;
    if constexpr (LAY == kFwd) {
      op.issue(p.p[0], p.ldp, m0, p.M, k0, p.K, lp + buf * OP::kBytes, w);
      // gated: half 0 is g's columns, half 1 u's, both from n0 on
      const int64_t c0 = GATED ? n0 - 128 * qh : n0;
      oq.issue(p.q[qh], p.ldq[qh], c0, p.N, k0, p.K, lq + buf * OQ::kBytes, w);
    } else if constexpr (LAY == kDx) {
      op.issue(p.p[seg], p.ldp, m0, p.M, k0, p.K, lp + buf * OP::kBytes, w);
      oq.issue(p.q[seg], p.ldq[seg], n0, p.N, k0, p.K, lq + buf * OQ::kBytes, w);
    } else {
      op.issue(p.p[0], p.ldp, m0, p.M, k0, p.K, lp + buf * OP::kBytes, w);
      oq.issue(p.q[out], p.ldq[out], n0, p.N, k0, p.K, lq + buf * OQ::kBytes, w);
    }
  };

  // LDS addresses of a lane's operands: KC one per half step (blocks are 16
  // rows, a constant apart), NC one per block of 16 columns (the swizzle
  // acts on the block's bits; half steps are a constant apart).
  const int g = lane / 16, i = lane % 16;
  auto kc_addr = [&](int row0, int kk) {
    return (uint32_t)((row0 + i) * 128 + (((4 * kk + g) ^ swz_kc(i)) * 16));
  };
  auto nc_addr = [&](int blk) {  // block of 16 columns
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
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[a][b] = f4v{0.f, 0.f, 0.f, 0.f};
  s8v fp[2][MB], fq[2][NB];
  auto read_half = [&](int kk, int buf) {
    const uint32_t po = buf * OP::kBytes, qo = buf * OQ::kBytes;
#pragma unroll
    for (int a = 0; a < MB; ++a)
      fp[kk][a] = PNC ? read_nc(pa[PNC ? a : 0] + po + kk * 32 * 256)
                      : read_kc(pa[PNC ? 0 : kk] + po + a * 16 * 128);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      fq[kk][b] = QNC ? read_nc(qa[QNC ? b : 0] + qo + kk * 32 * 256)
                      : read_kc(qa[QNC ? 0 : kk] + qo + b * 16 * 128);
  };
  auto mma_half = [&](int kk) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = mfma16<DT>(fq[kk][b], fp[kk][a], acc[a][b]);
  };

  if (s0 < s1) {
#pragma unroll
    for (int j = 0; j < NS; ++j) issue(s0 + j, j);
    stage_barrier<(NS - 1) * L>();
    read_half(0, 0);
    int buf = 0;
    for (int64_t t = s0; t < s1; ++t) {
      read_half(1, buf);
      mma_half(0);
      stage_barrier<(NS - 2) * L>();
      issue(t + NS, buf);
      buf = buf + 1 == NS ? 0 : buf + 1;
      read_half(0, buf);
      mma_half(1);
    }
    stage_barrier<0>();  // no load may land in LDS after the workgroup's end
  }

  // lane: row 16 a + i, columns 16 b + 4 g .. + 3
#pragma unroll
  for (int a = 0; a < MB; ++a) {
    const int64_t m = m0 + (wm * MB + a) * 16 + i;
    if (m >= p.M) continue;
    if constexpr (GATED) {
#pragma unroll
      for (int b = 0; b < NB / 2; ++b) {
        const int64_t n = n0 + (wn * (NB / 2) + b) * 16 + 4 * g;
        if (n >= p.N) continue;
        if (p.slices > 1) {
          float* q = p.part + ((slice * p.M + m) * 2) * p.N + n;
          *reinterpret_cast<f4v*>(q) = acc[a][b];
          *reinterpret_cast<f4v*>(q + p.N) = acc[a][b + NB / 2];
        } else {
          finish_gated<DT>(p, m, n, acc[a][b], acc[a][b + NB / 2]);
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int64_t n = n0 + (wn * NB + b) * 16 + 4 * g;
        if (n >= p.N) continue;
        if (p.slices > 1)
          *reinterpret_cast<f4v*>(p.part + ((slice * p.outs + out) * p.M + m) * p.N + n) = acc[a][b];
        else
          finish_linear<DT>(p, out, m, n, acc[a][b]);
      }
    }
  }
}

// Sums the slices' partials in slice order and finishes the outputs: one
// thread per 4 columns of a row.
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void k_lin_reduce(LinP p) {
  const int64_t n4 = p.N / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= p.M * p.outs * n4) return;
  const int64_t n = (id % n4) * 4, mo = id / n4;
  if constexpr (GATED) {
    f4v gs = {0.f, 0.f, 0.f, 0.f}, us = gs;
    for (int s = 0; s < p.slices; ++s) {
      const float* q = p.part + ((s * p.M + mo) * 2) * p.N + n;
      gs += *reinterpret_cast<const f4v*>(q);
      us += *reinterpret_cast<const f4v*>(q + p.N);
    }
    finish_gated<DT>(p, mo, n, gs, us);
  } else {
    f4v v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.slices; ++s)
      v += *reinterpret_cast<const f4v*>(p.part + ((int64_t)s * p.outs * p.M + mo) * p.N + n);
    const int o = mo >= p.M;
    finish_linear<DT>(p, o, mo - (o ? p.M : 0), n, v);
  }
}

// ---- the gradients' elementwise half --------------------------------------------
// d = dy * act'(pre) (linear) or dg = dh u act'(g), du = dh act(g) (gated),
// rounded to the element type for the products, and per strip of rows the
// fp32 column sums of the unrounded d (dbias).  A thread owns 8 columns of a
// strip.  Bound by memory: reads 2 (3) values and writes 1 (2) per entry.
struct DactP {
  const uint16_t *dy, *a, *b;  // a: pre or g; b: u
  int64_t lddy, lda, ldb;
  uint16_t *d0, *d1;           // [T][N]; d0 NULL: sums only
  float* sums;                 // [strips][N] or NULL
  int64_t T, N, strip;
  int act;
};
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void k_lin_dact(DactP p) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (n >= p.N) return;
  const int64_t t0 = blockIdx.y * p.strip;
  const int64_t t1 = t0 + p.strip < p.T ? t0 + p.strip : p.T;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const u16x8 dy = *reinterpret_cast<const u16x8*>(p.dy + t * p.lddy + n);
    u16x8 a = {}, b = {}, o0, o1;
    if (p.a) a = *reinterpret_cast<const u16x8*>(p.a + t * p.lda + n);
    if constexpr (GATED) b = *reinterpret_cast<const u16x8*>(p.b + t * p.ldb + n);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = to_f<DT>(dy[e]), z = to_f<DT>(a[e]);
      if constexpr (GATED) {
        o0[e] = from_f<DT>(v * to_f<DT>(b[e]) * act_slope(p.act, z));
        o1[e] = from_f<DT>(v * act_value(p.act, z));
      } else {
        const float d = p.a ? v * act_slope(p.act, z) : v;
        sum[e] += d;
        o0[e] = from_f<DT>(d);
      }
    }
    if (p.d0) *reinterpret_cast<u16x8*>(p.d0 + t * p.N + n) = o0;
    if constexpr (GATED) *reinterpret_cast<u16x8*>(p.d1 + t * p.N + n) = o1;
  }
  if constexpr (!GATED) {
    if (p.sums) {
      float* s = p.sums + blockIdx.y * p.N + n;
      *reinterpret_cast<f4v*>(s) = f4v{sum[0], sum[1], sum[2], sum[3]};
      *reinterpret_cast<f4v*>(s + 4) = f4v{sum[4], sum[5], sum[6], sum[7]};
    }
  }
}
// dbias[n] = the strips' sums, in strip order.
template <int DT>
__global__ __launch_bounds__(256) void k_lin_colsum(const float* sums, int64_t strips, int64_t N,
                                                    uint16_t* out) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.f;
  for (int64_t i = 0; i < strips; ++i) s += sums[i * N + n];
  out[n] = from_f<DT>(s);
}

// ---- plans -----------------------------------------------------------------------
constexpr int64_t kCus = 256;  // compute units of an MI355X

struct Plan {
  int tile;    // index into the compiled tiles (0: 256 x 256, 1: 128 x 128, 2: 16 rows)
  int slices;
};
constexpr int kTileM[3] = {256, 128, 16}, kTileN[3] = {256, 128, 128};

int64_t tiles_of(int tile, bool gated, int64_t M, int64_t N, int64_t outs) {
  // the gated small tiles hold 128 columns of g and of u
  const int64_t bn = gated ? 128 : kTileN[tile];
  return ((M + kTileM[tile] - 1) / kTileM[tile]) * ((N + bn - 1) / bn) * outs;
}

Plan lin_plan(int lay, bool gated, int64_t M, int64_t N, int64_t K, int segs, int outs) {
  Plan pl{0, 1};
  const int64_t steps = ((K + BK - 1) / BK) * segs;
  if (lay != kDw && M <= 16) pl.tile = 2;
  else if (tiles_of(0, gated, M, N, outs) < kCus) pl.tile = 1;
  const int64_t tiles = tiles_of(pl.tile, gated, M, N, outs);
  const int64_t want = pl.tile == 0 ? 1 : (2 * kCus) / (tiles > 0 ? tiles : 1);
  int64_t s = want < 1 ? 1 : want;
  if (s > steps / 2) s = steps / 2;
  if (s > 64) s = 64;
  pl.slices = s < 1 ? 1 : (int)s;
  return pl;
}

size_t part_bytes(const Plan& pl, int64_t M, int64_t N, int outs) {
  return pl.slices > 1 ? (size_t)pl.slices * M * N * outs * 4 : 0;
}

template <int DT, int LAY, bool GATED>
hipError_t launch_lin(LinP p, void* ws, hipStream_t s) {
  const Plan pl = lin_plan(LAY, GATED, p.M, p.N, p.K, p.segs, p.outs);
  if (p.M == 0 || p.N == 0) return hipSuccess;
  p.slices = pl.slices;
  p.part = reinterpret_cast<float*>(ws);
  const int64_t grid = tiles_of(pl.tile, GATED, p.M, p.N, p.outs) * pl.slices;
  if (grid > 0x7fffffffLL) return hipErrorNotSupported;
  const dim3 gr((unsigned)grid), th(256);
  constexpr int SB = GATED ? 256 : 128;
  if (pl.tile == 0) {
    hipLaunchKernelGGL((k_lin<DT, LAY, GATED, 256, 256, 2, 2, 2>), gr, th, 0, s, p);
  } else if (pl.tile == 1) {
    hipLaunchKernelGGL((k_lin<DT, LAY, GATED, 128, SB, 2, 2, 2>), gr, th, 0, s, p);
  } else {
    if constexpr (LAY != kDw)
      hipLaunchKernelGGL((k_lin<DT, LAY, GATED, 16, SB, 1, 4, 3>), gr, th, 0, s, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.slices == 1) return e;
  const int64_t n = (p.M * p.outs * (p.N / 4) + 255) / 256;
  if (n > 0x7fffffffLL) return hipErrorNotSupported;
  hipLaunchKernelGGL((k_lin_reduce<DT, GATED>), dim3((unsigned)n), th, 0, s, p);
  return hipGetLastError();
}

// Rows per strip of the elementwise kernel: 64, more where that would give
// over 1024 strips.
int64_t strip_rows(int64_t T) { return T <= 64 * 1024 ? 64 : (T + 1023) / 1024; }
int64_t strips_of(int64_t T) { return (T + strip_rows(T) - 1) / strip_rows(T); }

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

template <int DT>
hipError_t fwd_dt(const LinearCall& c, hipStream_t s) {
  LinP p{};
  p.p[0] = c.x;
  p.ldp = c.ldx;
  p.q[0] = c.w[0];
  p.q[1] = c.w[1];
  p.ldq[0] = c.ldw[0];
  p.ldq[1] = c.ldw[1];
  p.M = c.T;
  p.N = c.d_out;
  p.K = c.d_in;
  p.segs = p.outs = 1;
  p.act = c.act;
  p.bias = c.bias;
  p.res = c.res;
  p.ldr = c.ldr;
  p.y[0] = c.y;
  p.ldy[0] = c.ldy;
  for (int i = 0; i < 2; ++i) {
    p.pre[i] = c.pre[i];
    p.ldpre[i] = c.ldpre[i];
  }
  return c.gated ? launch_lin<DT, kFwd, true>(p, c.ws, s) : launch_lin<DT, kFwd, false>(p, c.ws, s);
}

template <int DT>
hipError_t bwd_dt(const LinearCall& c, hipStream_t s) {
  char* ws = static_cast<char*>(c.ws);
  const size_t dbytes = round256((size_t)c.T * c.d_out * 2);
  const bool map = c.gated || c.act != SA_ACT_NONE;  // d differs from dy
  const uint16_t* d[2] = {c.dy, nullptr};
  int64_t ldd = c.lddy;
  if (map) {
    d[0] = reinterpret_cast<uint16_t*>(ws);
    ws += dbytes;
    if (c.gated) {
      d[1] = reinterpret_cast<uint16_t*>(ws);
      ws += dbytes;
    }
    ldd = c.d_out;
  }
  const int64_t strips = strips_of(c.T);
  float* sums = nullptr;
  if (c.dbias) {
    sums = reinterpret_cast<float*>(ws);
    ws += round256((size_t)strips * c.d_out * 4);
  }
  hipError_t e = hipSuccess;
  if (c.T > 0 && (map || c.dbias)) {
    DactP a{};
    a.dy = c.dy;
    a.lddy = c.lddy;
    a.a = map ? c.pre[0] : nullptr;
    a.lda = c.ldpre[0];
    a.b = c.pre[1];
    a.ldb = c.ldpre[1];
    a.d0 = map ? const_cast<uint16_t*>(d[0]) : nullptr;
    a.d1 = const_cast<uint16_t*>(d[1]);
    a.sums = sums;
    a.T = c.T;
    a.N = c.d_out;
    a.strip = strip_rows(c.T);
    a.act = c.act;
    const dim3 gr((unsigned)((c.d_out / 8 + 255) / 256), (unsigned)strips);
    if (c.gated)
      hipLaunchKernelGGL((k_lin_dact<DT, true>), gr, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((k_lin_dact<DT, false>), gr, dim3(256), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (c.dbias) {
    hipLaunchKernelGGL((k_lin_colsum<DT>), dim3((unsigned)((c.d_out + 255) / 256)), dim3(256), 0, s,
                       sums, strips, c.d_out, c.dbias);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (c.dx) {
    LinP p{};
    p.p[0] = d[0];
    p.p[1] = d[1];
    p.ldp = ldd;
    for (int i = 0; i < 2; ++i) {
      p.q[i] = c.w[i];
      p.ldq[i] = c.ldw[i];
    }
    p.M = c.T;
    p.N = c.d_in;
    p.K = c.d_out;
    p.segs = c.gated ? 2 : 1;
    p.outs = 1;
    p.y[0] = c.dx;
    p.ldy[0] = c.lddx;
    e = launch_lin<DT, kDx, false>(p, ws, s);
    if (e != hipSuccess) return e;
  }
  if (c.dw[0]) {
    LinP p{};
    p.p[0] = c.x;
    p.ldp = c.ldx;
    for (int i = 0; i < 2; ++i) {
      p.q[i] = d[i];
      p.ldq[i] = ldd;
      p.y[i] = c.dw[i];
      p.ldy[i] = c.lddw[i];
    }
    p.M = c.d_in;
    p.N = c.d_out;
    p.K = c.T;
    p.segs = 1;
    p.outs = c.gated ? 2 : 1;
    e = launch_lin<DT, kDw, false>(p, ws, s);
  }
  return e;
}

}  // namespace

size_t linear_workspace_bytes(bool gated, int64_t T, int64_t d_in, int64_t d_out) {
  return part_bytes(lin_plan(kFwd, gated, T, d_out, d_in, 1, 1), T, d_out, gated ? 2 : 1);
}

size_t linear_backward_workspace_bytes(bool gated, int64_t T, int64_t d_in, int64_t d_out, int act,
                                       bool dbias) {
  const int n = gated ? 2 : 1;
  size_t b = 0;
  if (gated || act != SA_ACT_NONE) b += n * round256((size_t)T * d_out * 2);
  if (dbias) b += round256((size_t)strips_of(T) * d_out * 4);
  const size_t px = part_bytes(lin_plan(kDx, false, T, d_in, d_out, n, 1), T, d_in, 1);
  const size_t pw = part_bytes(lin_plan(kDw, false, d_in, d_out, T, 1, n), d_in, d_out, n);
  return b + (px > pw ? px : pw);
}

hipError_t launch_linear(const LinearCall& c, hipStream_t s) {
  return c.dtype == SA_F16 ? fwd_dt<SA_F16>(c, s) : fwd_dt<SA_BF16>(c, s);
}

hipError_t launch_linear_backward(const LinearCall& c, hipStream_t s) {
  return c.dtype == SA_F16 ? bwd_dt<SA_F16>(c, s) : bwd_dt<SA_BF16>(c, s);
}

}  // namespace sa
