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
#include "linear_engine.hpp"

namespace sa {
namespace {

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
