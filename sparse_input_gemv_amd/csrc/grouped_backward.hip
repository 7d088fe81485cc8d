// Linear layers grouped by expert for gfx950: the gradients.
//
//   d = dy act'(pre) (gated: dg = dh u act'(g), du = dh act(g));
//   dx = d We by rows' experts, dWe^T = x_e^T d_e, dbias_e = sum of d's rows.
//
// dW's K is the expert's rows, so its tiles differ in steps (none for an
// expert without rows: its gradient is written as zeros).  The elementwise
// half and its scales are the dense layers' (linear.hip), on strips of
// rows that end with their expert: column sums and scales are the expert's.
//
// d is rounded to 16 bits between the two halves, as the products take 16-bit
// operands: the gradients' error is 1.4 times that of one rounding at the end (bf16
// 2.3e-3 against 1.7e-3, fp16 2.9e-4 against 2.1e-4, relative).
//
// What bounds it, measured on MI355X: gate and up 4096 -> 11008 of 8 experts, 4096
// rows, bf16, 1680-1750 us: elementwise 115, dx 730, dW 900; ungated 930 (dx 470).
// dW writes 1.44 GB of gradients (4.65 TB/s) and its products wait for the stores;
// non-temporal stores, another order over the dies, staggered starts and later waits
// gave nothing (a tile of fewer stages, so that two workgroups share a CU, was not
// tried).  16 experts 1024 -> 4096, fp16: 509 rows 91-103 us in five launches, dx 40,
// dW 35 (one launch for both took as long); gated, 300 rows, 128.
#include "grouped_launch.hpp"

namespace sa {
namespace {

int strip_lg(int64_t T) {  // strips are powers of two here
  int lg = 4;
  while ((1 << lg) < strip_rows(T)) ++lg;
  return lg;
}
int64_t grp_strips(int64_t T, int64_t E) { return (T >> strip_lg(T)) + (E < T ? E : T); }  // at most

struct GrpDactP : DactP {
  const int32_t* offsets;
  int E;
};

template <int DT, bool GATED, int SCALING>
__global__ __launch_bounds__(256) void k_grp_dact(GrpDactP p, int lg) {
  __shared__ float part[4][64][9];
  __shared__ GroupTab tab;
  if constexpr (SCALING == kApply) {
    if (!*p.scaled) return;
  }
  if constexpr (SCALING == kFind) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.scaled = 0;
  }
  group_table(p.offsets, p.E, (int)p.T, lg, 1, tab);
  const int strip = (int)blockIdx.y;
  if (strip >= tab.first[p.E]) return;
  const int e = group_of(tab, p.E, strip);
  const int s0 = tab.row[e] + ((strip - tab.first[e]) << lg), last = tab.row[e + 1];
  const int send = s0 + (1 << lg) < last ? s0 + (1 << lg) : last;
  const float* cs = p.cs ? p.cs + (int64_t)e * (GATED ? 2 : 1) * p.N : nullptr;
  dact_strip<DT, GATED, SCALING>(p, s0, send, strip, cs, part);
}

// As k_lin_scales: the first `groups` workgroups take 64 of an expert's C columns
// at a time, the others a row of any expert per wave.
template <bool SUMS>
__global__ __launch_bounds__(256) void k_grp_scales(GrpDactP p, int lg, int64_t C, int cblocks, int groups,
                                                    int blocks, uint16_t* dbias) {
  __shared__ float part[4][64], most[4][64];
  __shared__ GroupTab tab;
  group_table(p.offsets, p.E, (int)p.T, lg, 1, tab);
  bool scaled = false;
  if ((int)blockIdx.x < groups) {
    for (int i = (int)blockIdx.x; i < cblocks * p.E; i += groups) {
      const int e = i / cblocks, b = i - e * cblocks;
      if (i >= groups) __syncthreads();  // the columns before are read
      scaled |= scale_columns<SUMS>(p, tab.first[e], tab.first[e + 1], C, (int64_t)b * 64,
                                    p.cs ? p.cs + e * C : nullptr, SUMS ? dbias + e * C : nullptr, part, most);
    }
  } else {
    const int64_t step = 4 * (int64_t)((int)gridDim.x - groups);
    const int64_t t0 = tab.row[0] + 4 * (int64_t)((int)blockIdx.x - groups) + (int)threadIdx.x / kWave;
    for (int64_t t = t0; t < tab.row[p.E]; t += step) scaled |= scale_row(p, t, blocks);
  }
  // read by later launches only: a store that may stay in this XCD's L2
  if (__syncthreads_or(scaled) && threadIdx.x == 0)
    __hip_atomic_store(p.scaled, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// dbias[blockIdx.y][64 columns].
template <int DT>
__global__ __launch_bounds__(256) void k_grp_colsum(GrpDactP p, int lg, uint16_t* dbias) {
  __shared__ float part[4][64];
  __shared__ GroupTab tab;
  group_table(p.offsets, p.E, (int)p.T, lg, 1, tab);
  const int e = (int)blockIdx.y;
  sum_columns<DT>(p.sums, tab.first[e], tab.first[e + 1], p.N, (int64_t)blockIdx.x * 64, dbias + e * p.N, part);
}

// dW: whole tiles, 256 x 256, or 128 x 128 where those take less time.  A round of
// either writes its outputs at 4.65 TB/s (7.2 us, 3.6 for 512 tiles of 32 KB),
// and that does not overlap its products: the CUs' stores are backed up while
// they are issued.
template <int DT>
hipError_t launch_dw(const GroupP& p, hipStream_t s) {
  constexpr int EPI = DT == SA_F16 ? kScaled : kPlain;
  int tile, split;
  linear_tuning(&tile, &split);
  const int64_t per = (int64_t)p.E * p.outs;
  const int64_t big = per * ((p.M + 255) / 256) * ((p.N + 255) / 256);
  const int64_t small = per * ((p.M + 127) / 128) * ((p.N + 127) / 128);
  if (small > 0x7fffffffLL) return hipErrorNotSupported;
  const double steps = (double)p.T / p.E / BK;
  const double tb = ((big + kCus - 1) / kCus) * (steps * 1.45 + 7.2);
  const double ts = ((small + 2 * kCus - 1) / (2 * kCus)) * (steps * (small > kCus ? 1.0 : 0.6) + 3.6);
  if (tile == 0 || (tile != 1 && tb <= ts)) grp_tile<DT, kDw, false, EPI, 256, 256, 2, 2, 2>(p, big, s);
  else grp_tile<DT, kDw, false, EPI, 128, 128, 2, 2, 2>(p, small, s);
  return hipGetLastError();
}

// The calls' scratch, in order; dx's partial sums follow.
struct Scratch {
  bool map = false, scaled = false;
  size_t d[2] = {}, e[2] = {}, sums = 0, rmax = 0, cmax = 0, rs = 0, cs = 0, flag = 0, end = 0;
};
Scratch scratch_of(int dtype, bool gated, int64_t T, int64_t E, int64_t d_out, int act, bool dbias) {
  Scratch b;
  const int n = gated ? 2 : 1;
  const int64_t strips = grp_strips(T, E), blocks = (d_out + 511) / 512;
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
  b.cs = take(E * n * d_out * 4);
  b.flag = take(4);
  return b;
}

template <int DT>
hipError_t bwd_dt(const GroupedCall& c, hipStream_t s) {
  char* ws = static_cast<char*>(c.ws);
  const Scratch b = scratch_of(DT, c.gated, c.T, c.experts, c.d_out, c.act, c.dbias != nullptr);
  const int outs = c.gated ? 2 : 1, lg = strip_lg(c.T);
  const uint16_t* d[2] = {c.dy, nullptr};
  int64_t ldd = c.lddy;
  if (b.map) {
    d[0] = reinterpret_cast<uint16_t*>(ws + b.d[0]);
    if (c.gated) d[1] = reinterpret_cast<uint16_t*>(ws + b.d[1]);
    ldd = c.d_out;
  }
  const bool scaled = b.scaled && c.T > 0 && (c.dx || c.dw[0]);
  GrpDactP a{};
  hipError_t e = hipSuccess;
  a.offsets = c.offsets;
  a.E = (int)c.experts;
  a.T = c.T;
  a.N = c.d_out;
  a.strip = 1 << lg;
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
    a.act = c.act;
    const int64_t strips = grp_strips(c.T, c.experts);
    if (strips > 65535) return hipErrorNotSupported;
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
        if (c.gated) hipLaunchKernelGGL((k_grp_dact<DT, true, kFind>), gr, dim3(256), 0, s, a, lg);
        else hipLaunchKernelGGL((k_grp_dact<DT, false, kFind>), gr, dim3(256), 0, s, a, lg);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t C = outs * c.d_out;
        const int cblocks = a.cs || c.dbias ? (int)((C + 63) / 64) : 0;
        const int64_t rows = c.dx ? (c.T + 3) / 4 : 0;
        // one block of columns each, but for wide outputs of many experts: a launch
        // holds fewer than 2^24 workgroups of 256 threads
        const int64_t columns = cblocks * c.experts;
        const int groups = columns < (1 << 23) ? (int)columns : 1 << 23;
        const dim3 gs((unsigned)(groups + (rows < 1024 ? rows : 1024)));
        if (c.dbias) hipLaunchKernelGGL((k_grp_scales<true>), gs, dim3(256), 0, s, a, lg, C, cblocks, groups, (int)gr.x, c.dbias);
        else hipLaunchKernelGGL((k_grp_scales<false>), gs, dim3(256), 0, s, a, lg, C, cblocks, groups, (int)gr.x, c.dbias);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (c.gated) hipLaunchKernelGGL((k_grp_dact<DT, true, kApply>), gr, dim3(256), 0, s, a, lg);
        else hipLaunchKernelGGL((k_grp_dact<DT, false, kApply>), gr, dim3(256), 0, s, a, lg);
      }
    }
    if (!scaled) {
      if (c.gated) hipLaunchKernelGGL((k_grp_dact<DT, true, kNone>), gr, dim3(256), 0, s, a, lg);
      else hipLaunchKernelGGL((k_grp_dact<DT, false, kNone>), gr, dim3(256), 0, s, a, lg);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (c.dbias && !scaled) {
    hipLaunchKernelGGL((k_grp_colsum<DT>), dim3((unsigned)((c.d_out + 63) / 64), (unsigned)c.experts), dim3(256),
                       0, s, a, lg, c.dbias);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  ws += b.end;
  GroupP x{}, w{};
  x.offsets = w.offsets = c.offsets;
  x.E = w.E = (int)c.experts;
  x.T = w.T = (int)c.T;
  x.p[0] = d[0];
  x.p[1] = d[1];
  x.ldp = (int)ldd;
  w.p[0] = c.x;
  w.ldp = (int)c.ldx;
  for (int i = 0; i < 2; ++i) {
    x.q[i] = c.w[i];
    x.ldq[i] = (int)c.ldw[i];
    x.sq[i] = c.sw[i];
    w.q[i] = d[i];
    w.ldq[i] = (int)ldd;
    w.y[i] = c.dw[i];
    w.ldy[i] = (int)c.lddw[i];
    w.sy[i] = c.sdw[i];
  }
  x.y[0] = c.dx;
  x.ldy[0] = (int)c.lddx;
  x.M = (int)c.T;
  x.N = (int)c.d_in;
  x.K = (int)c.d_out;
  x.segs = outs;
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
  // One after the other: in one launch, a workgroup of each on a CU, they take
  // as long (509 rows, 16 experts of 1024 x 4096: 74 us, 40 + 35 apart), as both
  // are bound by memory.
  if (c.dx) e = launch_grp<DT, kDx, false>(x, ws, s);
  if (e == hipSuccess && c.dw[0]) e = launch_dw<DT>(w, s);
  return e;
}

}  // namespace

size_t grouped_backward_workspace_bytes(int dtype, bool gated, int64_t T, int64_t experts, int64_t d_in,
                                        int64_t d_out, int act, bool dbias) {
  const size_t b = scratch_of(dtype, gated, T, experts, d_out, act, dbias).end;
  return b + (T ? grp_part_bytes(grp_plan(false, T, experts, d_in, d_out, gated ? 2 : 1), false) : 0);
}

hipError_t launch_grouped_backward(const GroupedCall& c, hipStream_t s) {
  return c.dtype == SA_F16 ? bwd_dt<SA_F16>(c, s) : bwd_dt<SA_BF16>(c, s);
}

}  // namespace sa
