// The gated projections of one tile, for 16-bit weights (gated_kernels.hip) and
// 4-bit ones (w4_kernels.hip): a wave's columns are half gates and half the ups
// beside them, so g and u of an output meet in one lane's registers and the
// activation and the product are the epilogue.
#pragma once

#include "gated_act.h"
#include "tile16.h"

namespace fp8blk {
namespace t16 {

// A row of saved factors: both halves, four outputs' in 12 bytes.
__host__ __device__ inline int64_t factor_half(int64_t I) { return (I + 3) / 4 * 12; }
__host__ __device__ inline int64_t factor_row(int64_t I) { return 2 * factor_half(I); }

struct GluArgs {
  const uint16_t *x;
  int64_t ldx, M, I, K;
  int64_t first, outs;            // of the I outputs, those of this launch
  int tiles_m, tiles_n;
  int steps, ranges;              // of K
  float *parts;                   // [ranges][M][2 outs], ranges > 1
  int act;
  uint16_t *h;                    // forward
  uint8_t *factors;               // rows of factor_row(I) bytes, or NULL
  const uint16_t *dh;             // gradient: dgu = d_h times the factors
  uint16_t *dgu;
  int64_t ld_dgu;                 // >= 2I; the rows end in zeros
};

// Row of W (counted in its half's rows from the tile's first output) and half of
// row `row` of the tile: of each wave's rows, first the gates', then the ups'.
template <typename S>
struct PairRow {
  int half, c;
  __device__ __forceinline__ explicit PairRow(int row) {
    constexpr int kHalf = S::kWaveN / 2;
    const int in = row % (2 * kHalf);
    half = in / kHalf;
    c = row / (2 * kHalf) * kHalf + in % kHalf;
  }
};

// What becomes of a g and its u: forward h (and the saved factors), or from the
// gradient d of h those of g and u.
template <int ACT>
__device__ __forceinline__ void glu(v4f g, v4f u, float (&h)[4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = act_value<ACT>(g[r]) * u[r];
}
template <int ACT>
__device__ __forceinline__ void glu_factors(v4f g, v4f u, float (&f)[4], float (&a)[4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float slope;
    act_both<ACT>(g[r], a[r], slope);
    f[r] = u[r] * slope;
  }
}
__device__ __forceinline__ void save_factors(const GluArgs &p, int64_t m, int64_t n,
                                             const float (&f)[4], const float (&a)[4]) {
  uint8_t *row = p.factors + m * factor_row(p.I) + n * 3;
  store_24(row, f);      // (past the last output: of zero sums)
  store_24(row + factor_half(p.I), a);
}

// The tile's outputs from (m0, n0) on; the wave's begin row, col further.
template <typename T, typename S, int ACT, bool GRAD>
__device__ __forceinline__ void glu_store(const GluArgs &p, const typename S::Acc &acc, int64_t m0,
                                          int64_t n0, int row, int col, uint8_t *lds) {
  constexpr int kHalf = S::kFN / 2, kCols = S::TN / 2;
  static_assert(!(S::kAcross && GRAD), "factors and d_h are taken four columns at a time");
  const int lane = threadIdx.x & 63;
  __syncthreads();      // every wave is past its last stage
#pragma unroll
  for (int i = 0; i < S::kFM; ++i)
#pragma unroll
    for (int j = 0; j < kHalf; ++j) {
      const v4f g = acc[i][j], u = acc[i][j + kHalf];
      const int64_t m = m0 + row + S::row(i, 0, lane), n = n0 + col + S::col(j, 0, lane);
      const bool in = m < p.M && n < p.I;
      if constexpr (GRAD) {
        float d[4] = {0, 0, 0, 0}, f[4], a[4];
        if (in) load4<T>(p.dh + m * p.I + n, d, p.I - n);
        glu_factors<ACT>(g, u, f, a);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          f[r] *= d[r];
          a[r] *= d[r];
        }
        stage4<T, S, kCols>(lds, row, col, i, j, f, lane);
        stage4<T, S, kCols>(lds + S::TM * kCols * 2, row, col, i, j, a, lane);
      } else {
        float h[4];
        glu<ACT>(g, u, h);
        stage4<T, S, kCols>(lds, row, col, i, j, h, lane);
        if constexpr (!S::kAcross) {
          if (p.factors && in) {
            float f[4], a[4];
            glu_factors<ACT>(g, u, f, a);
            save_factors(p, m, n, f, a);
          }
        }
      }
    }
  __syncthreads();
  const int64_t rows = p.M - m0, cols = p.I - n0;
  if constexpr (GRAD) {
    uint16_t *out = p.dgu + m0 * p.ld_dgu + n0;
    store_staged<S::kThreads, S::TM, kCols>(lds, out, p.ld_dgu, rows, cols);
    store_staged<S::kThreads, S::TM, kCols>(lds + S::TM * kCols * 2, out + p.I, p.ld_dgu, rows,
                                            cols);
    if (cols <= kCols)      // the rows end in zeros
      for (int r = threadIdx.x; r < S::TM && r < rows; r += S::kThreads)
        for (int64_t c = 2 * p.I; c < p.ld_dgu; ++c) p.dgu[(m0 + r) * p.ld_dgu + c] = 0;
  } else {
    store_staged<S::kThreads, S::TM, kCols>(lds, p.h + m0 * p.I + n0, p.I, rows, cols);
  }
}

// W::Pair<T, S> loads the tile's rows of the weights (init(w, p, n0, wave, lane)),
// W::multiply<T, S> forms the tile's sums with it, in W::Smem<S>, placed as W::Place<S>.
template <typename T, typename Tile, bool GRAD, typename W>
__global__ __launch_bounds__(Tile::kThreads) void glu_kernel(GluArgs p, W w) {
  using S = typename W::template Place<Tile>;
  __shared__ typename W::template Smem<S> sm;
  const int tiles = p.tiles_m * p.tiles_n, range = blockIdx.x / tiles;
  int tm, tn;
  tile_of(blockIdx.x - range * tiles, p.tiles_m, p.tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m = (int64_t)tm * S::TM, n = p.first + (int64_t)tn * (S::TN / 2);
  Loader<kRows, S::TM, S::kWaves> la;
  la.init(Operand{p.x + m * p.ldx, p.ldx, min(p.M - m, (int64_t)S::TM), p.K}, wave, lane);
  typename W::template Pair<T, S> lb;
  lb.init(w, p, n, wave, lane);
  const int s0 = (int)((int64_t)p.steps * range / p.ranges);
  const int s1 = (int)((int64_t)p.steps * (range + 1) / p.ranges);
  typename S::Acc acc;
  W::template multiply<T, S>(la, lb, s0, s1 - s0, sm, acc);
  const int row = wave_row<S>(), col = wave_col<S>() / 2;
  if (p.ranges > 1) {
    constexpr int kHalf = S::kFN / 2;
    float *parts = p.parts + ((int64_t)range * p.M + m + row) * 2 * p.outs + n - p.first + col;
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
      for (int j = 0; j < S::kFN; ++j)
        store_part<S>(parts + i * 32 * p.outs + (j >= kHalf ? p.outs : 0) + j % kHalf * 16,
                      2 * p.outs, p.M - m - row - i * 16,
                      p.first + p.outs - n - col - j % kHalf * 16, acc[i][j], lane);
    return;
  }
  uint8_t *lds = reinterpret_cast<uint8_t *>(&sm);
  if (p.act == kSilu) glu_store<T, S, kSilu, GRAD>(p, acc, m, n, row, col, lds);
  else if (p.act == kGelu) glu_store<T, S, kGelu, GRAD>(p, acc, m, n, row, col, lds);
  else glu_store<T, S, kGeluTanh, GRAD>(p, acc, m, n, row, col, lds);
}

// The outputs of parts, four a thread.
template <typename T, int ACT, bool GRAD>
__device__ __forceinline__ void glu_store4(const GluArgs &p, int64_t m, int64_t n, v4f g, v4f u) {
  const int64_t left = p.I - n;
  float a[4], f[4];
  if constexpr (GRAD) {
    float d[4];
    load4<T>(p.dh + m * p.I + n, d, left);
    glu_factors<ACT>(g, u, f, a);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f[r] *= d[r];
      a[r] *= d[r];
    }
    uint16_t *row = p.dgu + m * p.ld_dgu;
    store4<T>(row + n, f, left);
    store4<T>(row + p.I + n, a, left);
    if (left <= 4)
      for (int64_t c = 2 * p.I; c < p.ld_dgu; ++c) row[c] = 0;
  } else {
    glu<ACT>(g, u, a);
    store4<T>(p.h + m * p.I + n, a, left);
    if (p.factors) {
      glu_factors<ACT>(g, u, f, a);
      save_factors(p, m, n, f, a);
    }
  }
}
template <typename T, bool GRAD>
__global__ __launch_bounds__(256) void glu_join_kernel(GluArgs p) {
  const int64_t quads = (p.outs + 3) / 4, step = p.M * 2 * p.outs;
  for (int64_t at = first_item(); at < p.M * quads; at += all_threads()) {
    const int64_t m = at / quads, c = (at - m * quads) * 4, left = p.outs - c, n = p.first + c;
    const float *q = p.parts + m * 2 * p.outs + c;
    const v4f g = join4(q, p.ranges, step, left), u = join4(q + p.outs, p.ranges, step, left);
    if (p.act == kSilu) glu_store4<T, kSilu, GRAD>(p, m, n, g, u);
    else if (p.act == kGelu) glu_store4<T, kGelu, GRAD>(p, m, n, g, u);
    else glu_store4<T, kGeluTanh, GRAD>(p, m, n, g, u);
  }
}

// Launches by plan; p's sizes, pointers and act are set.
template <typename T, bool GRAD, typename W>
hipError_t launch_glu(GluArgs p, const W &w, hipStream_t stream) {
  hipError_t e = hipSuccess;
  each_launch(cut_of(p.M, 2 * p.I, p.K, W::kFourBits), 2 * p.I,
              [&](int64_t first, int64_t cols, const Plan &plan) {
    if (e != hipSuccess) return;
    p.first = first / 2;      // (whole tiles, half of them gates)
    p.outs = cols / 2;
    p.steps = (int)tiles(p.K, kK);
    p.ranges = plan.ranges;
    with_shape(plan.shape, [&](auto shape) {
      using S = decltype(shape);
      p.tiles_m = (int)tiles(p.M, S::TM);
      p.tiles_n = (int)tiles(p.outs, S::TN / 2);
      glu_kernel<T, S, GRAD, W>
          <<<dim3((unsigned)p.tiles_m * p.tiles_n * p.ranges), S::kThreads, 0, stream>>>(p, w);
    });
    e = hipGetLastError();
    if (e == hipSuccess && p.ranges > 1) {
      glu_join_kernel<T, GRAD><<<groups(p.M * tiles(p.outs, 4)), 256, 0, stream>>>(p);
      e = hipGetLastError();
    }
  });
  return e;
}

}  // namespace t16
}  // namespace fp8blk
