// Launches of the products grouped by expert, which grouped.hip (forward) and
// grouped_backward.hip share.  The kernel is the dense layers' (lin_run) on
// items that carry their expert: every workgroup first turns the offsets,
// which the host never sees, into a table of row tiles in its LDS.
//
// A split deals the steps of the last round of tiles (of all, where they are
// fewer than the workgroups) evenly over the workgroups, as in the dense layers,
// but the tiles' number is known on the device only.  So partial sums belong to
// shares, not tiles: a share can hold part of two tiles at most, its first and
// its last, and those it holds whole it finishes.  The share that begins a tile
// it does not end writes the tile down for k_grp_reduce.  (Decoding, 16 rows over
// 8 experts, gated 4096 -> 14336, bf16: whole tiles 257 us, split 242, 6.8 TB/s.)
#pragma once

#define SA_LINEAR_ENGINE_ONLY
#include "linear.hip"

namespace sa {
namespace {

template <int LAY, int BM>
constexpr int table_lg() {  // dW: the table's rows alone are used
  return LAY == kDw ? 6 : __builtin_ctz(BM);
}
template <int DT, int LAY, bool GATED, int EPI, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(256, 1) void k_grp(GroupP p) {
  __shared__ __align__(16) uint8_t S[lin_lds<LAY, BM, BN, NS>()];
  __shared__ GroupTab tab;
  constexpr int BNO = GATED ? BN / 2 : BN;
  group_table(p.offsets, p.E, p.T, table_lg<LAY, BM>(), LAY == kDw ? 1 : (p.N + BNO - 1) / BNO, tab);
  lin_run<DT, LAY, GATED, EPI, BM, BN, WM, WN, NS>(p, blockIdx.x, gridDim.x, S, &tab);
}

// Sums the partials of the tile that share blockIdx.x begins and does not end
// (if any) and finishes 2048 of its outputs, 8 columns of a row per thread.
template <int DT, bool GATED, int BN>
__global__ __launch_bounds__(256) void k_grp_reduce(GroupP p, int lbm) {
  constexpr int OCT = (GATED ? BN / 2 : BN) / 8, ROWS = 256 / OCT;
  const CutTile c = p.cut[blockIdx.x];
  const int row = (int)blockIdx.y * ROWS + (int)threadIdx.x / OCT, col = (int)threadIdx.x % OCT * 8;
  const int n = c.n0 + col;
  if (c.shares == 0 || row >= c.rows || n >= p.N) return;
  const float* const at = p.part + row * BN + col;
  const int64_t tile = (int64_t)BN << lbm;
  F8 f[kChains] = {}, u[kChains] = {};
  for (int s = 0; s < c.shares; s += kChains) {
#pragma unroll
    for (int k = 0; k < kChains; ++k) {
      if (s + k >= c.shares) break;
      const float* q = at + (((int64_t)blockIdx.x + s + k) * 2 + (s + k == 0)) * tile;
      add_part(f[k], q);
      if constexpr (GATED) add_part(u[k], q + BN / 2);
    }
  }
  LinP l = p;
  if (l.bias) l.bias += c.e * (int64_t)p.N;
  if constexpr (GATED) finish_gated<DT>(l, c.m0 + row, n, add_chains(f), add_chains(u));
  else finish_linear<DT, DT == SA_F16>(l, 0, c.m0 + row, n, add_chains(f));
}

// The compiled tiles: 256 x 256, and 128, 64, 32 or 16 rows x 128 (gated: 128
// of g and of u).
constexpr int kGrpTiles = 5;
constexpr int kGrpM[kGrpTiles] = {256, 128, 64, 32, 16}, kGrpN[kGrpTiles] = {256, 128, 128, 128, 128};

struct GrpPlan {
  int tile, split;  // split: shares, 0 for whole tiles
  int64_t tiles;    // at most
};

inline int64_t grp_row_tiles(int tile, int64_t T, int64_t E) {  // at most
  return T / kGrpM[tile] + (E < T ? E : T);
}

// The tile and split with the smallest estimated time, for rows spread evenly
// over the experts (the host knows no more).  An expert's rows fill tiles of
// BM rows but for half of the last one.  A step takes what it does in the dense
// plan, and tiles of up to 64 rows as long as a CU needs to read their weights
// at 40 GB/s; together they read them at 6.6 TB/s, each for itself, as they run
// far apart (larger ones share them).  A round of workgroups costs 4 us more, a
// split 8 (5 where only the last of several rounds is) and its partial sums.
// Over 22 random shapes (forward, gated, dx; 1 to 3924 rows, 1 to 124 experts)
// the choice took 2 percent longer than the best of a sweep on average, 25 at
// most (108 rows of 14 experts, gated 992 -> 312: 18.5 against 14.8 us).
inline GrpPlan grp_plan(bool gated, int64_t T, int64_t E, int64_t N, int64_t K, int segs) {
  static const double alone[2][kGrpTiles] = {{1.45, 0.60, 0.45, 0.41, 0.41}, {1.45, 0.95, 0.82, 0.82, 0.82}};
  static const double paired[kGrpTiles] = {0, 0.50, 0.36, 0.25, 0.22};
  const int64_t steps = ((K + BK - 1) / BK) * segs;
  const double used = (double)(E < T ? E : T), mean = used > 0 ? T / used : 0;
  int tuned_tile, tuned_split;
  linear_tuning(&tuned_tile, &tuned_split);
  if (tuned_tile >= kGrpTiles) tuned_tile = -1;
  GrpPlan best{kGrpTiles - 1, 0, 0};
  double least = 1e30;
  for (int t = kGrpTiles - 1; t >= 0; --t) {
    if (tuned_tile >= 0 && t != tuned_tile) continue;
    const int64_t nt = (N + (gated ? 128 : kGrpN[t]) - 1) / (gated ? 128 : kGrpN[t]);
    const int64_t most = grp_row_tiles(t, T, E) * nt;
    const double per = mean <= kGrpM[t] / 2 ? 1 : mean / kGrpM[t] + 0.5;  // row tiles of an expert
    const double tiles = used * per * nt;
    const bool pairs = t > 0 && !gated;
    const double step = alone[gated][t];
    const double both = pairs && 2 * paired[t] > step ? 2 * paired[t] : step;
    const double read = (t >= 2 ? tiles : used * nt) * steps * (gated || t == 0 ? 32768 : 16384) / 6.6e6 + 4;
    const int64_t cus = pairs ? 2 * kCus : kCus;
    const double rounds = tiles <= cus ? 1 : (int64_t)(tiles / cus) + 1;
    double whole = rounds * (steps * (tiles > kCus ? both : step) + 4);
    whole = whole > 1.08 * read ? whole : 1.08 * read;  // whole tiles end unevenly
    // even shares, one workgroup per CU; positions times shares fit 31 bits
    int64_t shares = tuned_split > 0 ? tuned_split : kCus;
    while (shares & (shares - 1)) shares &= shares - 1;
    if (t == 0) {  // the last round alone is shared, where the device finds that it pays: from 24 steps on
      if (shares > kCus) shares = kCus;
      const bool rest = tuned_split != 0 && (tuned_split > 0 || steps >= 24) &&
                        kCus * steps * shares < 0x7fffffffLL && most < 0x3fffffffLL;
      if (whole < least) {
        least = whole;
        best = GrpPlan{t, rest ? (int)shares : 0, most};
      }
      continue;
    }
    if (tuned_split <= 0 && whole < least) {
      least = whole;
      best = GrpPlan{t, 0, most};
    }
    if (tuned_split == 0 || most * steps * shares >= 0x7fffffffLL) continue;
    // not tiles of 128 rows: their shares took 1.65 us a step in dx (509 rows,
    // 16 experts of 1024 x 4096: 53 us, whole tiles of 64 rows 40)
    if (tuned_split < 0 && t < 2) continue;
    const double parts = shares * 2.0 * (mean < kGrpM[t] ? mean : kGrpM[t]) * (gated ? 256 : 128) * 8 / 4e6;
    const double shared = tiles * steps / shares * step;
    const double time = (shared > read ? shared : read) + (tiles > shares ? 5 : 8) + parts;
    if (time < least) {
      least = time;
      best = GrpPlan{t, (int)shares, most};
    }
  }
  if (best.tiles == 0) best.tiles = grp_row_tiles(best.tile, T, E) * ((N + 127) / 128);
  return best;
}

inline size_t grp_part_bytes(const GrpPlan& pl, bool gated) {
  if (!pl.split) return 0;
  return round256(pl.split * sizeof(CutTile)) + (size_t)pl.split * 2 * kGrpM[pl.tile] * (gated ? 256 : kGrpN[pl.tile]) * 4;
}

template <int DT, int LAY, bool GATED, int EPI, int BM, int BN, int WM, int WN, int NS>
void grp_tile(const GroupP& p, int64_t items, hipStream_t s) {  // items: shares or tiles
  constexpr int64_t most = kCus * (160 * 1024 / (lin_lds<LAY, BM, BN, NS>() + (int)sizeof(GroupTab)));
  const dim3 grid((unsigned)(p.split || items < most ? items : most));
  hipLaunchKernelGGL((k_grp<DT, LAY, GATED, EPI, BM, BN, WM, WN, NS>), grid, dim3(256), 0, s, p);
}

template <int DT, bool GATED>
hipError_t launch_grp_reduce(const GroupP& p, const GrpPlan& pl, hipStream_t s) {
  const int rows = kGrpM[pl.tile] < p.T ? kGrpM[pl.tile] : p.T, lbm = __builtin_ctz(kGrpM[pl.tile]);
  if (!GATED && pl.tile == 0)
    hipLaunchKernelGGL((k_grp_reduce<DT, GATED, 256>), dim3(pl.split, (rows + 7) / 8), dim3(256), 0, s, p, lbm);
  else
    hipLaunchKernelGGL((k_grp_reduce<DT, GATED, GATED ? 256 : 128>), dim3(pl.split, (rows + 15) / 16), dim3(256), 0,
                       s, p, lbm);
  return hipGetLastError();
}

// Forward and dx.
template <int DT, int LAY, bool GATED>
hipError_t launch_grp(GroupP p, void* ws, hipStream_t s) {
  static_assert(LAY != kDw, "rows are grouped");
  if (p.T == 0 || p.N == 0) return hipSuccess;
  const GrpPlan pl = grp_plan(GATED, p.T, p.E, p.N, p.K, p.segs);
  if (pl.tiles > 0x7fffffffLL) return hipErrorNotSupported;
  p.split = pl.split;
  p.cut = reinterpret_cast<CutTile*>(ws);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + round256(pl.split * sizeof(CutTile)));
  const int64_t items = pl.split ? pl.split : pl.tiles;
  constexpr int SB = GATED ? 256 : 128;
  constexpr int EPI = LAY == kFwd ? kGeneral : DT == SA_F16 ? kScaled : kPlain;
  if (pl.tile == 0) {
    if (LAY == kFwd && (GATED ? !p.pre[0] : !p.bias && !p.pre[0] && p.act == SA_ACT_NONE && !p.res))
      grp_tile<DT, LAY, GATED, LAY == kFwd ? kPlain : EPI, 256, 256, 2, 2, 2>(p, items, s);
    else
      grp_tile<DT, LAY, GATED, EPI, 256, 256, 2, 2, 2>(p, items, s);
  } else if (pl.tile == 1) {
    grp_tile<DT, LAY, GATED, EPI, 128, SB, 2, 2, GATED ? 3 : 2>(p, items, s);
  } else if (pl.tile == 2) {
    grp_tile<DT, LAY, GATED, EPI, 64, SB, 1, 4, 3>(p, items, s);
  } else if (pl.tile == 3) {
    grp_tile<DT, LAY, GATED, EPI, 32, SB, 1, 4, GATED ? 4 : 3>(p, items, s);
  } else {
    grp_tile<DT, LAY, GATED, EPI, 16, SB, 1, 4, GATED ? 4 : 3>(p, items, s);
  }
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !pl.split ? e : launch_grp_reduce<DT, GATED>(p, pl, s);
}

}  // namespace
}  // namespace sa
