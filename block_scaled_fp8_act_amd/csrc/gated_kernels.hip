// The gated projections of a feed-forward block and their gradients, for gfx950:
//   g = x Wg^T, u = x Wu^T, h = act(g) * u,
// x [M, K], W [2I, K] (gate rows first), h [M, I] in bf16 or fp16, sums in fp32.
//   f = (u act'(g), act(g)),  dgu = (d_h f_gate, d_h f_up)   [M, 2I]
//   d_x = dgu W,  d_W = dgu^T x.
//
// One kernel does both projections, the activation and the product (glu_tile.h);
// the gradients are two more products on the same tiles (tile16.h), whose operands are
// read where they lie, with the sum along rows or columns.
//
// Measured on one MI355X, on which a large 16-bit library product runs at 1.39 to 1.53
// PFLOP/s and a large copy at 5.0 TB/s:
//   4096 x 7168 -> 18432        1.63 ms, 1.33 PFLOP/s: matrix instructions at the 1.5 GHz
//                               that they leave the chip, then the operands' way into LDS
//   4096 x 4096 -> 14336, all   forward 795 us (with factors), factors 118, d_x 714
//                               (1.35 PFLOP/s), d_W 770 (1.25)
//   1003 x 1536 -> 4099, all    177 us: each product one partly empty round of tiles
//   515 x 1000 -> 2731          20.6 us: 16 steps' latency and the copy of x to a 16-byte
//                               pitch (3 us)
//   1 x 4096 -> 14336           33.7 us: W at 7.0 TB/s
// The factors are saved rather than g and u, so that the gradient needs no activation;
// without them the first product runs again with the gradient's epilogue (1003 rows:
// 60 us).
//
// dgu is rounded to 16 bits once, as the matrix instructions take it.  With that and their
// own rounding d_x and d_W are 1.41 times as far from binary64 as fp32 sums of an unrounded
// dgu (bf16 0.0023 against 0.0017, fp16 0.00029 against 0.00021, relative).  A second 16-bit
// part of it would take the difference away and run both products again (at 4096 x 4096 ->
// 14336 another 714 and 770 us beside the step's 2400).
#include <algorithm>

#include "glu_tile.h"

namespace fp8blk {

using namespace t16;

namespace {

__global__ __launch_bounds__(256) void align_rows_kernel(const uint16_t *in, int64_t ld,
                                                         int64_t rows, int64_t cols,
                                                         uint16_t *out, int64_t ldo) {
  align_rows(in, ld, rows, cols, out, ldo);
}

// 16-bit weights [2I, K], rows ld apart (whole 16-byte chunks).
struct Dense {
  const uint16_t *w;
  int64_t ld;
  static constexpr bool kFourBits = false;
  template <typename S>
  using Place = S;
  template <typename S>
  using Smem = typename S::Smem;
  template <typename T, typename S, typename LA, typename LB>
  static __device__ __forceinline__ void multiply(const LA &la, const LB &lb, int step0, int steps,
                                                  typename S::Smem &sm, typename S::Acc &acc) {
    t16::multiply<T, S, kRows, kRows>(la, lb, step0, steps, sm, acc);
  }
  template <typename T, typename S>
  struct Pair : Loader<kRows, S::TN, S::kWaves> {
    __device__ __forceinline__ void init(const Dense &d, const GluArgs &p, int64_t n0, int wave_,
                                         int lane) {
      using L = Loader<kRows, S::TN, S::kWaves>;
      static_assert(S::kWaveN / 2 == L::kDma * 8, "a wave loads its half's rows, gates or ups");
      const int half = PairRow<S>(8 * L::kDma * wave_).half;
      const int64_t left = p.I - n0;
      this->place(Operand{d.w + (half * p.I + n0) * d.ld, d.ld, min(left, (int64_t)S::TN / 2), p.K},
                  wave_);
#pragma unroll
      for (int i = 0; i < L::kDma; ++i) {
        const int row = 8 * (L::kDma * wave_ + i) + (lane >> 3);
        const int c = PairRow<S>(row).c;
        this->chunk[i] = (lane & 7) ^ swz_f(row);
        this->off[i] = c < left ? c * (uint32_t)d.ld * 2 + this->chunk[i] * 16 : kOut;
      }
    }
  };
};

// ---------------------------------------------------------------------------
// One or two rows of x (single decoding sequences): W streams past once, 8 values a lane
// and row, 512 of K at a time; a lane's products are summed
// by the two-element dot product and the lanes' sums joined at the end.  Rows of any
// width: 16 bytes at any even address, the last few of K one by one.  Bound: HBM
// traffic of W, which is loaded past the caches.
template <typename T>
struct Dot;
template <>
struct Dot<Bf16> {
  typedef __bf16 V __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ float two(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c,
                                           false);
  }
};
template <>
struct Dot<F16> {
  typedef _Float16 V __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ float two(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, false);
  }
};

__device__ __forceinline__ v4u load8(const uint16_t *p, int64_t left) {
  if (left >= 8) return *reinterpret_cast<const v4u_any *>(p);
  v4u v = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < left) v[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
  return v;
}

struct FewArgs {
  const uint16_t *x, *w;
  int64_t ldx, K, I;
  int M, act;
  uint16_t *h;
  uint8_t *factors;
};

// R outputs a wave, MT rows of x (M of them there), the K range shared by KS waves.
template <typename T, int R, int MT, int KS>
__global__ __launch_bounds__(256) void few_kernel(FewArgs p) {
  constexpr int kRows = 2 * R, kOuts = 4 / KS * R;
  __shared__ float red[4][kRows * MT];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kOuts;
  const uint16_t *w[kRows], *x[MT];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    w[i] = p.w + (min(n0 + wave / KS * R + i % R, p.I - 1) + (i >= R ? p.I : 0)) * p.K + lane * 8;
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = p.x + min(m, p.M - 1) * p.ldx + lane * 8;
  float acc[kRows * MT];
#pragma unroll
  for (int i = 0; i < kRows * MT; ++i) acc[i] = 0.0f;
  auto add = [&](const v4u (&wv)[kRows], const v4u (&xv)[MT]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i * MT + m] = Dot<T>::two(wv[i][e], xv[m][e], acc[i * MT + m]);
  };
  const int64_t whole = p.K / 512 * 512;
  v4u wv[kRows], xv[MT];
#pragma unroll 2
  for (int64_t k = (int64_t)(wave % KS) * 512; k < whole; k += KS * 512) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      wv[i] = __builtin_nontemporal_load(reinterpret_cast<const v4u_any *>(w[i] + k));
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = *reinterpret_cast<const v4u_any *>(x[m] + k);
    add(wv, xv);
  }
  if (whole < p.K && wave % KS == KS - 1) {
    const int64_t left = p.K - whole - lane * 8;
#pragma unroll
    for (int i = 0; i < kRows; ++i) wv[i] = load8(w[i] + whole, left);
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = load8(x[m] + whole, left);
    add(wv, xv);
  }
  wave_sums<kRows * MT>(acc, red[wave], lane);
  __syncthreads();
  // a thread an output
  if ((int)threadIdx.x >= kOuts * MT) return;
  const int m = threadIdx.x % MT, o = threadIdx.x / MT, r = o % R, w0 = o / R * KS;
  const int64_t n = n0 + o;
  if (m >= p.M || n >= p.I) return;
  float g = 0.0f, u = 0.0f;
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    g += red[w0 + i][r * MT + m];
    u += red[w0 + i][(R + r) * MT + m];
  }
  float a, slope;
  both_any(p.act, g, a, slope);
  p.h[m * p.I + n] = (uint16_t)T::bits(a * u);
  if (p.factors) {
    uint8_t *f = p.factors + m * factor_row(p.I) + n * 3;
    store_24_one(f, u * slope);
    store_24_one(f + factor_half(p.I), a);
  }
}

template <typename T, int MT>
hipError_t few(const FewArgs &p, hipStream_t stream) {
  // an output a wave and K shared by four (4096 -> 14336: 33.9 us for a row, 41.3 for
  // two; two outputs 34.9 and 49.1, four and all of K a wave 48.9), but not pieces of a
  // few loads
  constexpr int R = 1;
  if (p.K < 1024)
    few_kernel<T, R, MT, 1><<<dim3((unsigned)tiles(p.I, 4 * R)), 256, 0, stream>>>(p);
  else
    few_kernel<T, R, MT, 4><<<dim3((unsigned)tiles(p.I, R)), 256, 0, stream>>>(p);
  return hipGetLastError();
}

// dgu from the saved factors, 4 outputs a thread.  Bound: HBM traffic (4096 x 14336:
// 118 us, 704 MB, 6.0 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void factors_kernel(const uint16_t *dh, const uint8_t *factors,
                                                      int64_t M, int64_t I, uint16_t *dgu,
                                                      int64_t ld_dgu) {
  const int64_t quads = (I + 3) / 4;
  for (int64_t at = first_item(); at < M * quads; at += all_threads()) {
    const int64_t m = at / quads, n = (at - m * quads) * 4, left = I - n;
    float d[4], f[4], a[4];
    load4<T>(dh + m * I + n, d, left);
    const uint8_t *p = factors + m * factor_row(I) + n * 3;
    load_24(p, f);
    load_24(p + factor_half(I), a);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f[r] *= d[r];
      a[r] *= d[r];
    }
    uint16_t *row = dgu + m * ld_dgu;
    store4<T>(row + n, f, left);
    store4<T>(row + I + n, a, left);
    if (left <= 4)
      for (int64_t c = 2 * I; c < ld_dgu; ++c) row[c] = 0;
  }
}

// ---------------------------------------------------------------------------
// The products of the gradients: out [rows, cols] = A B^T, in ranges of K where
// the tiles alone leave the chip idle (fp32 parts, added in order afterwards).

template <typename T, typename S, Kind KA, Kind KB>
__global__ __launch_bounds__(S::kThreads) void product_kernel(Operand a, Operand b, Out p) {
  __shared__ typename S::Smem sm;
  const int tiles = p.tiles_m * p.tiles_n, range = blockIdx.x / tiles;
  int tm, tn;
  tile_of(blockIdx.x - range * tiles, p.tiles_m, p.tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)tm * S::TM, n0 = (int64_t)tn * S::TN;
  a.p += m0 * (KA == kRows ? a.ld : 1);
  b.p += n0 * (KB == kRows ? b.ld : 1);
  a.rows = min(a.rows - m0, (int64_t)S::TM);
  b.rows = min(b.rows - n0, (int64_t)S::TN);
  Loader<KA, S::TM, S::kWaves> la;
  Loader<KB, S::TN, S::kWaves> lb;
  la.init(a, wave, lane);
  lb.init(b, wave, lane);
  const int s0 = p.first_step(range);
  typename S::Acc acc;
  multiply<T, S, KA, KB>(la, lb, s0, p.first_step(range + 1) - s0, sm, acc);
  store_tile<T, S>(p, acc, m0, n0, range, reinterpret_cast<uint8_t *>(&sm));
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t *out, int64_t n) {
  for (int64_t i = first_item(); i < n; i += all_threads()) out[i] = 0;
}

// ---------------------------------------------------------------------------
// Host side.

hipError_t align(const uint16_t *in, int64_t ld, int64_t rows, int64_t cols, uint16_t *out,
                 hipStream_t stream) {
  const int64_t ldo = up(cols, 8);
  align_rows_kernel<<<groups(rows * (ldo / 8)), 256, 0, stream>>>(in, ld, rows, cols, out, ldo);
  return hipGetLastError();
}

// out [rows, cols] = A B^T.
template <typename T, Kind KA, Kind KB>
hipError_t product(const Operand &a, const Operand &b, void *out, int64_t rows, int64_t cols,
                   float *parts, hipStream_t stream) {
  hipError_t e = hipSuccess;
  each_launch(cut_of(rows, cols, a.k), cols, [&](int64_t first, int64_t n, const Plan &plan) {
    if (e != hipSuccess) return;
    Operand part = b;
    part.p += first * (KB == kRows ? b.ld : 1);
    part.rows -= first;
    Out p{rows, n, static_cast<uint16_t *>(out) + first, cols, parts};
    with_shape(plan.shape, [&](auto shape) {
      using S = decltype(shape);
      const dim3 grid = p.tile<S>(plan, a.k);
      product_kernel<T, S, KA, KB><<<grid, S::kThreads, 0, stream>>>(a, part, p);
    });
    e = hipGetLastError();
    if (e == hipSuccess && p.ranges > 1) e = join<T>(p, stream);
  });
  return e;
}

hipError_t zero(void *out, int64_t n, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  zero_kernel<<<groups(n), 256, 0, stream>>>(static_cast<uint16_t *>(out), n);
  return hipGetLastError();
}

// x and W with rows on 16 bytes: themselves, or copies in the workspace.
struct Inputs {
  const uint16_t *x, *w;
  int64_t ldx, ldw;
};

void inputs_space(int64_t M, int64_t I, int64_t K, int64_t ldx, Space &s) {
  if (ldx % 8 || K % 8) s.take((size_t)M * up(K, 8) * 2);
  if (K % 8) s.take((size_t)2 * I * up(K, 8) * 2);
}

hipError_t lay_inputs(const GatedCall &c, Inputs &in, Space &s, hipStream_t stream) {
  in = {static_cast<const uint16_t *>(c.x), static_cast<const uint16_t *>(c.w), c.ldx, c.K};
  const int64_t kp = up(c.K, 8);
  if (c.ldx % 8 || c.K % 8) {
    uint16_t *x = reinterpret_cast<uint16_t *>(s.take((size_t)c.M * kp * 2));
    if (hipError_t e = align(in.x, in.ldx, c.M, c.K, x, stream)) return e;
    in.x = x;
    in.ldx = kp;
  }
  if (c.K % 8) {
    uint16_t *w = reinterpret_cast<uint16_t *>(s.take((size_t)2 * c.I * kp * 2));
    if (hipError_t e = align(in.w, in.ldw, 2 * c.I, c.K, w, stream)) return e;
    in.w = w;
    in.ldw = kp;
  }
  return hipSuccess;
}

GluArgs glu_args(const GatedCall &c, const Inputs &in, const Space &s) {
  GluArgs p{};
  p.x = in.x;
  p.ldx = in.ldx;
  p.M = c.M;
  p.I = c.I;
  p.K = up(c.K, 8);
  p.act = c.act;
  p.parts = reinterpret_cast<float *>(s.base + s.used);
  return p;
}

// More rows take longer here (3 rows of 4096 -> 14336: 71 us) than on tiles (58).
constexpr int64_t kFewRows = 2;

template <typename T>
hipError_t forward(const GatedCall &c, void *h, void *factors, void *work, hipStream_t stream) {
  if (c.M <= kFewRows) {
    const FewArgs p{static_cast<const uint16_t *>(c.x), static_cast<const uint16_t *>(c.w), c.ldx,
                    c.K, c.I, (int)c.M, c.act, static_cast<uint16_t *>(h),
                    static_cast<uint8_t *>(factors)};
    return c.M == 1 ? few<T, 1>(p, stream) : few<T, 2>(p, stream);
  }
  Space s{static_cast<uint8_t *>(work), 0};
  Inputs in;
  if (hipError_t e = lay_inputs(c, in, s, stream)) return e;
  GluArgs p = glu_args(c, in, s);
  p.h = static_cast<uint16_t *>(h);
  p.factors = static_cast<uint8_t *>(factors);
  return launch_glu<T, false>(p, Dense{in.w, in.ldw}, stream);
}

template <typename T>
hipError_t backward(const GatedCall &c, const void *dh, const void *factors, void *dx, void *dw,
                    void *work, hipStream_t stream) {
  Space s{static_cast<uint8_t *>(work), 0};
  Inputs in;
  if (hipError_t e = lay_inputs(c, in, s, stream)) return e;
  const int64_t ld = up(2 * c.I, 8), kp = up(c.K, 8);
  uint16_t *dgu = reinterpret_cast<uint16_t *>(s.take((size_t)c.M * ld * 2));
  // the parts of one product after the other
  float *parts = reinterpret_cast<float *>(s.base + s.used);
  if (factors) {
    factors_kernel<T><<<groups(c.M * tiles(c.I, 4)), 256, 0, stream>>>(
        static_cast<const uint16_t *>(dh), static_cast<const uint8_t *>(factors), c.M, c.I, dgu, ld);
    if (hipError_t e = hipGetLastError()) return e;
  } else {
    GluArgs p = glu_args(c, in, s);
    p.dh = static_cast<const uint16_t *>(dh);
    p.dgu = dgu;
    p.ld_dgu = ld;
    if (hipError_t e = launch_glu<T, true>(p, Dense{in.w, in.ldw}, stream)) return e;
  }
  if (dx)
    if (hipError_t e = product<T, kRows, kCols>(Operand{dgu, ld, c.M, ld},
                                                Operand{in.w, in.ldw, kp, 2 * c.I}, dx, c.M, c.K,
                                                parts, stream))
      return e;
  if (dw)
    if (hipError_t e = product<T, kCols, kCols>(Operand{dgu, ld, ld, c.M},
                                                Operand{in.x, in.ldx, kp, c.M}, dw, 2 * c.I, c.K,
                                                parts, stream))
      return e;
  return hipSuccess;
}

}  // namespace

bool gated_fits(int64_t M, int64_t I, int64_t K) {
  return grid_fits(M, 2 * I) && grid_fits(M, K) && grid_fits(2 * I, K);
}

size_t gated_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t ldx) {
  if (M <= kFewRows) return 0;
  Space s{nullptr, 0};
  inputs_space(M, I, K, ldx, s);
  return s.used + part_bytes(M, 2 * I, up(K, 8));
}

hipError_t launch_gated(const GatedCall &c, void *h, void *factors, void *work,
                        hipStream_t stream) {
  return c.bf16 ? forward<Bf16>(c, h, factors, work, stream)
                : forward<F16>(c, h, factors, work, stream);
}

// (sized for the projections computed again, whether they are or not)
size_t gated_backward_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t ldx, bool dx,
                                      bool dw) {
  Space s{nullptr, 0};
  inputs_space(M, I, K, ldx, s);
  s.take((size_t)M * up(2 * I, 8) * 2);
  return s.used + std::max({part_bytes(M, 2 * I, up(K, 8)),
                            dx ? part_bytes(M, K, up(2 * I, 8)) : 0,
                            dw ? part_bytes(2 * I, K, M) : 0});
}

hipError_t launch_gated_backward(const GatedCall &c, const void *dh, const void *factors, void *dx,
                                 void *dw, void *work, hipStream_t stream) {
  if (c.M == 0) return dw ? zero(dw, 2 * c.I * c.K, stream) : hipSuccess;
  if (c.I == 0) return dx ? zero(dx, c.M * c.K, stream) : hipSuccess;
  return c.bf16 ? backward<Bf16>(c, dh, factors, dx, dw, work, stream)
                : backward<F16>(c, dh, factors, dx, dw, work, stream);
}

}  // namespace fp8blk
