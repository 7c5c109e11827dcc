// The gated projections of a feed-forward block and their gradients, for gfx950:
//   g = x Wg^T, u = x Wu^T, h = act(g) * u,
// x [M, K], W [2I, K] (gate rows first), h [M, I] in bf16 or fp16, sums in fp32.
//   f = (u act'(g), act(g)),  dgu = (d_h f_gate, d_h f_up)   [M, 2I]
//   d_x = dgu W,  d_W = dgu^T x.
//
// One kernel does both projections, the activation and the product (glu_tile.h);
// the gradients are two more products on the same tiles (tile16.h).
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
  template <typename T, typename S>
  struct Pair : Loader<kRows, S::TN, S::kWaves> {
    __device__ __forceinline__ void init(const Dense &d, const GluArgs &p, int64_t n0, int wave_,
                                         int lane) {
      using L = Loader<kRows, S::TN, S::kWaves>;
      static_assert(S::kFN * 8 == L::kDma * 8, "a wave loads its half's rows, gates or ups");
      this->wave = wave_;
      const int half = PairRow<S>(8 * L::kDma * wave_).half;
      const int64_t left = p.I - n0;
      this->o = Operand{d.w + (half * p.I + n0) * d.ld, d.ld, min(left, (int64_t)S::TN / 2), p.K};
#pragma unroll
      for (int i = 0; i < L::kDma; ++i) {
        const int row = 8 * (L::kDma * wave_ + i) + (lane >> 3);
        const int c = PairRow<S>(row).c;
        this->chunk[i] = (lane & 7) ^ swz_f(row);
        this->off[i] = c < left ? (uint32_t)(c * d.ld * 2) + this->chunk[i] * 16 : kOut;
      }
    }
  };
};

// dgu from the saved factors, 8 outputs a thread.
template <typename T>
__global__ __launch_bounds__(256) void factors_kernel(const uint16_t *dh, const uint16_t *factors,
                                                      int64_t M, int64_t I, uint16_t *dgu,
                                                      int64_t ld_dgu) {
  const int64_t chunks = (I + 7) / 8;
  for (int64_t at = first_item(); at < M * chunks; at += all_threads()) {
    const int64_t m = at / chunks, n = (at - m * chunks) * 8;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint16_t *f = factors + (m * 2 + half) * I + n;
      uint16_t *out = dgu + m * ld_dgu + half * I + n;
      if (n + 8 <= I) {
        const v4u dv = *reinterpret_cast<const v4u_any *>(dh + m * I + n);
        const v4u fv = *reinterpret_cast<const v4u_any *>(f);
        v4u o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = pack2<T>(T::value(dv[j] & 0xffff) * T::value(fv[j] & 0xffff),
                          T::value(dv[j] >> 16) * T::value(fv[j] >> 16));
        *reinterpret_cast<v4u_any *>(out) = o;
      } else {
        for (int j = 0; n + j < I; ++j)
          out[j] = (uint16_t)T::bits(T::value(dh[m * I + n + j]) * T::value(f[j]));
      }
    }
    if (n + 8 >= I)
      for (int64_t c = 2 * I; c < ld_dgu; ++c) dgu[m * ld_dgu + c] = 0;
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
  v4f acc[S::kFM][S::kFN];
  multiply<T, S, KA, KB>(la, lb, s0, p.first_step(range + 1) - s0, sm, acc);
  store_tile<T, S>(p, acc, m0, n0, range);
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

template <typename T, Kind KA, Kind KB>
hipError_t product(const Operand &a, const Operand &b, Out p, hipStream_t stream) {
  const Plan plan = plan_of(p.rows, p.cols, a.k);
  p.steps = (int)tiles(a.k, kK);
  p.ranges = plan.ranges;
  p.tiles_m = (int)tiles(p.rows, plan.large ? Large::TM : Small::TM);
  p.tiles_n = (int)tiles(p.cols, plan.large ? Large::TN : Small::TN);
  const dim3 grid((unsigned)p.tiles_m * p.tiles_n * p.ranges);
  if (plan.large) product_kernel<T, Large, KA, KB><<<grid, Large::kThreads, 0, stream>>>(a, b, p);
  else product_kernel<T, Small, KA, KB><<<grid, Small::kThreads, 0, stream>>>(a, b, p);
  if (p.ranges > 1) {
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<T><<<groups(tiles(p.rows * p.cols, 4)), 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

size_t part_bytes(int64_t rows, int64_t cols, int64_t k) {
  const int r = plan_of(rows, cols, k).ranges;
  return r == 1 ? 0 : (size_t)r * rows * cols * sizeof(float);
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

template <typename T>
hipError_t forward(const GatedCall &c, void *h, void *factors, void *work, hipStream_t stream) {
  Space s{static_cast<uint8_t *>(work), 0};
  Inputs in;
  if (hipError_t e = lay_inputs(c, in, s, stream)) return e;
  GluArgs p = glu_args(c, in, s);
  p.h = static_cast<uint16_t *>(h);
  p.factors = static_cast<uint16_t *>(factors);
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
    factors_kernel<T><<<groups(c.M * tiles(c.I, 8)), 256, 0, stream>>>(
        static_cast<const uint16_t *>(dh), static_cast<const uint16_t *>(factors), c.M, c.I, dgu,
        ld);
    if (hipError_t e = hipGetLastError()) return e;
  } else {
    GluArgs p = glu_args(c, in, s);
    p.dh = static_cast<const uint16_t *>(dh);
    p.dgu = dgu;
    p.ld_dgu = ld;
    if (hipError_t e = launch_glu<T, true>(p, Dense{in.w, in.ldw}, stream)) return e;
  }
  if (dx) {
    const Out o{c.M, c.K, static_cast<uint16_t *>(dx), parts};
    if (hipError_t e = product<T, kRows, kCols>(Operand{dgu, ld, c.M, ld},
                                                Operand{in.w, in.ldw, kp, 2 * c.I}, o, stream))
      return e;
  }
  if (dw) {
    const Out o{2 * c.I, c.K, static_cast<uint16_t *>(dw), parts};
    if (hipError_t e = product<T, kCols, kCols>(Operand{dgu, ld, ld, c.M},
                                                Operand{in.x, in.ldx, kp, c.M}, o, stream))
      return e;
  }
  return hipSuccess;
}

}  // namespace

bool gated_fits(int64_t M, int64_t I, int64_t K) {
  const int64_t most = (int64_t(1) << 32) / Large::kThreads;   // workgroups of a grid
  return grid_of<Large>(M, 2 * I) < most && grid_of<Large>(M, K) < most &&
         grid_of<Large>(2 * I, K) < most;
}

size_t gated_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t ldx) {
  Space s{nullptr, 0};
  inputs_space(M, I, K, ldx, s);
  return s.used + glu_part_bytes(M, I, up(K, 8));
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
  return s.used + std::max({glu_part_bytes(M, I, up(K, 8)),
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
