// Linear layers grouped by expert for gfx950, forward: rows offsets[e] ..
// offsets[e + 1] - 1 of x through expert e's weights, fp16 or bf16 with fp32
// sums.
//
//   grouped_linear        y = act(x We^T + be) + residual
//   grouped_gated_linear  h = act(x Wge^T) * (x Wue^T)
//
// What bounds it: many rows per expert, the matrix cores' power, as in the
// dense layers; few rows, the weights' stream of the experts that have rows.
// Measured on MI355X, bf16: gate and up 4096 -> 14336 of 8 experts, 16 rows 202-254
// us, by how many experts have rows (6.5-6.9 TB/s of weights read; a large copy runs
// at 4.8-5.1); 64 experts 1024 -> 4096, 1000 rows, fp16, 97-105 us; down 14336 ->
// 4096, 8192 rows over 8 experts 805-877 us: 1.1-1.2 PFLOP/s of existing rows.  The
// tiles that an expert's last rows leave part empty cost the rest (4096 ragged rows
// over 8 experts fill about 4 of 5).
#include "grouped_launch.hpp"

namespace sa {
namespace {

template <int DT>
hipError_t fwd_dt(const GroupedCall& c, hipStream_t s) {
  GroupP p{};
  p.p[0] = c.x;
  p.ldp = (int)c.ldx;
  for (int i = 0; i < 2; ++i) {
    p.q[i] = c.w[i];
    p.ldq[i] = (int)c.ldw[i];
    p.sq[i] = c.sw[i];
    p.pre[i] = c.pre[i];
    p.ldpre[i] = (int)c.ldpre[i];
  }
  p.M = p.T = (int)c.T;
  p.N = (int)c.d_out;
  p.K = (int)c.d_in;
  p.segs = p.outs = 1;
  p.act = c.act;
  p.bias = c.bias;
  p.res = c.res;
  p.ldr = (int)c.ldr;
  p.y[0] = c.y;
  p.ldy[0] = (int)c.ldy;
  p.offsets = c.offsets;
  p.E = (int)c.experts;
  return c.gated ? launch_grp<DT, kFwd, true>(p, c.ws, s) : launch_grp<DT, kFwd, false>(p, c.ws, s);
}

}  // namespace

size_t grouped_workspace_bytes(bool gated, int64_t T, int64_t experts, int64_t d_in, int64_t d_out) {
  return T ? grp_part_bytes(grp_plan(gated, T, experts, d_out, d_in, 1), gated) : 0;
}

hipError_t launch_grouped(const GroupedCall& c, hipStream_t s) {
  return c.dtype == SA_F16 ? fwd_dt<SA_F16>(c, s) : fwd_dt<SA_BF16>(c, s);
}

int grouped_plan(int op, int64_t T, int64_t experts, int64_t d_in, int64_t d_out, int* rows, int* split) {
  GrpPlan pl;
  switch (op) {
    case SA_LINEAR_FORWARD: pl = grp_plan(false, T, experts, d_out, d_in, 1); break;
    case SA_LINEAR_GATED: pl = grp_plan(true, T, experts, d_out, d_in, 1); break;
    case SA_LINEAR_DX: pl = grp_plan(false, T, experts, d_in, d_out, 1); break;
    case SA_LINEAR_GATED_DX: pl = grp_plan(false, T, experts, d_in, d_out, 2); break;
    default: return 1;
  }
  *rows = kGrpM[pl.tile];
  *split = pl.split;
  return 0;
}

}  // namespace sa
