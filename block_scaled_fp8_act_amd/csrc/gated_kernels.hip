// The gated projections of a feed-forward block and their gradients, for gfx950:
//   g = x Wg^T, u = x Wu^T, h = act(g) * u,
// x [M, K], W [2I, K] (gate rows first), h [M, I] in bf16 or fp16, sums in fp32.
//   f = (u act'(g), act(g)),  dgu = (d_h f_gate, d_h f_up)   [M, 2I]
//   d_x = dgu W,  d_W = dgu^T x.
//
// One kernel does both projections, the activation and the product: a wave's 64
// columns of W are 32 gates and the 32 ups beside them, so g and u of an output
// meet in one lane's registers.
#include <algorithm>

#include "gated_act.h"
#include "tile16.h"

namespace fp8blk {

using namespace t16;

namespace {

// Element-wise kernels: as many workgroups as the work has, up to a grid that HIP
// runs whole, whose threads then take several items each.
constexpr int64_t kMostGroups = 1 << 20;
__device__ __forceinline__ int64_t first_item() {
  return (int64_t)blockIdx.x * 256 + threadIdx.x;
}
__device__ __forceinline__ int64_t all_threads() { return (int64_t)gridDim.x * 256; }

// ---------------------------------------------------------------------------
// Rows brought to a 16-byte pitch, for inputs whose rows are not (an odd width or
// stride); what is past a row's end reads as zeros.

__global__ __launch_bounds__(256) void align_rows_kernel(const uint16_t *in, int64_t ld,
                                                         int64_t rows, int64_t cols,
                                                         uint16_t *out, int64_t ldo) {
  const int64_t chunks = ldo / 8;
  for (int64_t at = first_item(); at < rows * chunks; at += all_threads()) {
    const int64_t r = at / chunks, c = (at - r * chunks) * 8;
    const uint16_t *p = in + r * ld + c;
    v4u v;
    if (c + 8 <= cols) {
      v = *reinterpret_cast<const v4u_any *>(p);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = c + j < cols ? p[j] : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = e[2 * j] | (e[2 * j + 1] << 16);
    }
    *reinterpret_cast<v4u *>(out + r * ldo + c) = v;
  }
}

// ---------------------------------------------------------------------------
// Stores of four neighbouring columns.

template <typename T>
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4], int64_t left) {
  if (left >= 4) {
    v2u u = {pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
    *reinterpret_cast<v2u_any *>(p) = u;
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < left) p[r] = (uint16_t)T::bits(v[r]);
  }
}
template <typename T>
__device__ __forceinline__ void load4(const uint16_t *p, float (&v)[4], int64_t left) {
  if (left >= 4) {
    const v2u u = *reinterpret_cast<const v2u_any *>(p);
    v[0] = T::value(u[0] & 0xffff);
    v[1] = T::value(u[0] >> 16);
    v[2] = T::value(u[1] & 0xffff);
    v[3] = T::value(u[1] >> 16);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = r < left ? T::value(p[r]) : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Both projections.

// W's rows of a tile of TN / 2 outputs: of each wave's 64, first 32 gates, then
// the ups of the same outputs.
template <int kDma>
struct GateUpLoader : Loader<kRows, kDma * 8, kDma> {
  __device__ __forceinline__ void init_pair(const uint16_t *w, int64_t K, int64_t ld, int64_t I,
                                            int64_t n0, int wave_, int lane) {
    static_assert(kDma == 4, "a wave loads 32 rows, all gates or all ups");
    this->wave = wave_;
    const int half = wave_ & 1;
    this->o = Operand{w + (half * I + n0) * ld, ld, I - n0, K};
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int row = 8 * (kDma * wave_ + i) + (lane >> 3);
      const int c = (row >> 6) * 32 + (row & 31);
      this->chunk[i] = (lane & 7) ^ swz_f(row);
      this->off[i] = c < I - n0 ? (uint32_t)(c * ld * 2) + this->chunk[i] * 16 : kOut;
    }
    // rows of the resource: those of the tile at most
    this->o.rows = min(I - n0, (int64_t)128);
  }
};

struct GluArgs {
  const uint16_t *x, *w;
  int64_t ldx, ldw, M, I, K;
  int tiles_m, tiles_n;
  int act;
  uint16_t *h, *factors;          // forward: factors may be NULL
  const uint16_t *dh;             // gradient: dgu = d_h times the factors
  uint16_t *dgu;
  int64_t ld_dgu;
};

template <typename T, int ACT, bool GRAD, int FM>
__device__ __forceinline__ void glu_store(const GluArgs &p, const v4f (&acc)[FM][4], int64_t m0,
                                          int64_t n0, int lane) {
  const int r16 = lane & 15, q = lane >> 4;
#pragma unroll
  for (int mi = 0; mi < FM; ++mi) {
    const int64_t m = m0 + mi * 16 + r16;
    if (m >= p.M) continue;
#pragma unroll
    for (int ni = 0; ni < 2; ++ni) {
      const int64_t n = n0 + ni * 16 + 4 * q;
      const int64_t left = p.I - n;
      if (left <= 0) continue;
      float a[4], f[4];
      if constexpr (GRAD) {
        float d[4];
        load4<T>(p.dh + m * p.I + n, d, left);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g = acc[mi][ni][r], u = acc[mi][ni + 2][r];
          f[r] = d[r] * (u * act_slope<ACT>(g));
          a[r] = d[r] * act_value<ACT>(g);
        }
        uint16_t *row = p.dgu + m * p.ld_dgu;
        store4<T>(row + n, f, left);
        store4<T>(row + p.I + n, a, left);
      } else {
        float hv[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float g = acc[mi][ni][r], u = acc[mi][ni + 2][r];
          a[r] = act_value<ACT>(g);
          hv[r] = a[r] * u;
          f[r] = u;
        }
        store4<T>(p.h + m * p.I + n, hv, left);
        if (p.factors) {
#pragma unroll
          for (int r = 0; r < 4; ++r) f[r] *= act_slope<ACT>(acc[mi][ni][r]);
          uint16_t *row = p.factors + m * 2 * p.I;
          store4<T>(row + n, f, left);
          store4<T>(row + p.I + n, a, left);
        }
      }
    }
  }
}

template <typename T, typename S, bool GRAD>
__global__ __launch_bounds__(S::kThreads) void glu_kernel(GluArgs p) {
  __shared__ typename S::Smem sm;
  int tm, tn;
  tile_of(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)tm * S::TM, n0 = (int64_t)tn * (S::TN / 2);
  Loader<kRows, S::TM, S::kDmaA> la;
  la.init(Operand{p.x + m0 * p.ldx, p.ldx, min(p.M - m0, (int64_t)S::TM), p.K}, wave, lane);
  GateUpLoader<S::kDmaB> lb;
  lb.init_pair(p.w, p.K, p.ldw, p.I, n0, wave, lane);
  v4f acc[S::kFM][4];
  multiply<T, S, kRows, kRows>(la, lb, 0, (int)((p.K + kK - 1) / kK), sm, acc);
  const int64_t m = m0 + wave / S::kWN * (S::kFM * 16), n = n0 + wave % S::kWN * 32;
  if (p.act == kSilu) glu_store<T, kSilu, GRAD>(p, acc, m, n, lane);
  else if (p.act == kGelu) glu_store<T, kGelu, GRAD>(p, acc, m, n, lane);
  else glu_store<T, kGeluTanh, GRAD>(p, acc, m, n, lane);
  if constexpr (GRAD) {    // dgu's rows end in zeros
    if (tn == p.tiles_n - 1 && (int)threadIdx.x < S::TM && m0 + threadIdx.x < p.M)
      for (int64_t c = 2 * p.I; c < p.ld_dgu; ++c) p.dgu[(m0 + threadIdx.x) * p.ld_dgu + c] = 0;
  }
}

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

struct ProductArgs {
  Operand a, b;
  int64_t rows, cols;     // of the output
  int tiles_m, tiles_n;
  int steps, ranges;
  uint16_t *out;          // [rows, cols]
  float *parts;           // [ranges][rows][cols], ranges > 1
};

template <typename T, typename S, Kind KA, Kind KB>
__global__ __launch_bounds__(S::kThreads) void product_kernel(ProductArgs p) {
  __shared__ typename S::Smem sm;
  const int tiles = p.tiles_m * p.tiles_n;
  const int range = blockIdx.x / tiles;
  int tm, tn;
  tile_of(blockIdx.x - range * tiles, p.tiles_m, p.tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)tm * S::TM, n0 = (int64_t)tn * S::TN;
  Operand a = p.a, b = p.b;
  a.p += m0 * (KA == kRows ? a.ld : 1);
  b.p += n0 * (KB == kRows ? b.ld : 1);
  a.rows = min(a.rows - m0, (int64_t)S::TM);
  b.rows = min(b.rows - n0, (int64_t)S::TN);
  Loader<KA, S::TM, S::kDmaA> la;
  Loader<KB, S::TN, S::kDmaB> lb;
  la.init(a, wave, lane);
  lb.init(b, wave, lane);
  const int s0 = (int)((int64_t)p.steps * range / p.ranges);
  const int s1 = (int)((int64_t)p.steps * (range + 1) / p.ranges);
  v4f acc[S::kFM][4];
  multiply<T, S, KA, KB>(la, lb, s0, s1 - s0, sm, acc);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t mw = m0 + wave / S::kWN * (S::kFM * 16), nw = n0 + wave % S::kWN * 64;
#pragma unroll
  for (int mi = 0; mi < S::kFM; ++mi) {
    const int64_t m = mw + mi * 16 + r16;
    if (m >= p.rows) continue;
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) {
      const int64_t n = nw + ni * 16 + 4 * q;
      const int64_t left = p.cols - n;
      if (left <= 0) continue;
      if (p.ranges == 1) {
        const float v[4] = {acc[mi][ni][0], acc[mi][ni][1], acc[mi][ni][2], acc[mi][ni][3]};
        store4<T>(p.out + m * p.cols + n, v, left);
      } else {
        float *o = p.parts + ((int64_t)range * p.rows + m) * p.cols + n;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r < left) o[r] = acc[mi][ni][r];
      }
    }
  }
}

// out = the sum of `ranges` parts, in order.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(const float *parts, int ranges, int64_t n,
                                                   uint16_t *out) {
  for (int64_t i = first_item() * 4; i < n; i += all_threads() * 4) {
    const int64_t left = n - i;
    float v[4] = {0, 0, 0, 0};
    for (int s = 0; s < ranges; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) v[r] += parts[s * n + i + r];
    store4<T>(out + i, v, left);
  }
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t *out, int64_t n) {
  for (int64_t i = first_item(); i < n; i += all_threads()) out[i] = 0;
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int kCUs = 256;

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }
dim3 groups(int64_t items) { return dim3((unsigned)std::min(tiles(items, 256), kMostGroups)); }

template <typename S>
int64_t grid_of(int64_t rows, int64_t cols) {
  return tiles(rows, S::TM) * tiles(cols, S::TN);
}

// 256 x 256 tiles where they fill most of the chip.
bool use_large(int64_t rows, int64_t cols) { return grid_of<Large>(rows, cols) >= 192; }

// Ranges of K: enough workgroups for two a compute unit, at least 8 stages each.
int ranges_of(int64_t rows, int64_t cols, int64_t k) {
  if (use_large(rows, cols)) return 1;
  const int64_t grid = grid_of<Small>(rows, cols), steps = tiles(k, kK);
  const int64_t r = std::min<int64_t>(2 * kCUs / grid, steps / 8);
  return (int)std::max<int64_t>(r, 1);
}

hipError_t align_rows(const uint16_t *in, int64_t ld, int64_t rows, int64_t cols, uint16_t *out,
                      hipStream_t stream) {
  const int64_t ldo = up(cols, 8), n = rows * (ldo / 8);
  align_rows_kernel<<<groups(n), 256, 0, stream>>>(in, ld, rows, cols, out,
                                                                       ldo);
  return hipGetLastError();
}

template <typename T, bool GRAD>
hipError_t glu(GluArgs p, hipStream_t stream) {
  if (use_large(p.M, 2 * p.I)) {
    p.tiles_m = (int)tiles(p.M, Large::TM);
    p.tiles_n = (int)tiles(p.I, Large::TN / 2);
    glu_kernel<T, Large, GRAD>
        <<<dim3(p.tiles_m * p.tiles_n), Large::kThreads, 0, stream>>>(p);
  } else {
    p.tiles_m = (int)tiles(p.M, Small::TM);
    p.tiles_n = (int)tiles(p.I, Small::TN / 2);
    glu_kernel<T, Small, GRAD>
        <<<dim3(p.tiles_m * p.tiles_n), Small::kThreads, 0, stream>>>(p);
  }
  return hipGetLastError();
}

template <typename T, Kind KA, Kind KB>
hipError_t product(ProductArgs p, hipStream_t stream) {
  const bool large = use_large(p.rows, p.cols);
  p.steps = (int)tiles(p.a.k, kK);
  p.ranges = ranges_of(p.rows, p.cols, p.a.k);
  p.tiles_m = (int)tiles(p.rows, large ? Large::TM : Small::TM);
  p.tiles_n = (int)tiles(p.cols, large ? Large::TN : Small::TN);
  const unsigned grid = (unsigned)p.tiles_m * p.tiles_n * p.ranges;
  if (large) product_kernel<T, Large, KA, KB><<<dim3(grid), Large::kThreads, 0, stream>>>(p);
  else product_kernel<T, Small, KA, KB><<<dim3(grid), Small::kThreads, 0, stream>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  if (p.ranges == 1) return hipSuccess;
  const int64_t n = p.rows * p.cols;
  join_kernel<T><<<groups(tiles(n, 4)), 256, 0, stream>>>(p.parts, p.ranges, n, p.out);
  return hipGetLastError();
}

hipError_t zero(void *out, int64_t n, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  zero_kernel<<<groups(n), 256, 0, stream>>>(static_cast<uint16_t *>(out), n);
  return hipGetLastError();
}

size_t part_bytes(int64_t rows, int64_t cols, int64_t k) {
  const int r = ranges_of(rows, cols, k);
  return r == 1 ? 0 : (size_t)r * rows * cols * sizeof(float);
}

// Workspace parts start at multiples of 256 bytes.
struct Space {
  uint8_t *base;
  size_t used;
  uint8_t *take(size_t n) {
    uint8_t *at = base + used;
    used += (n + 255) / 256 * 256;
    return at;
  }
};

bool odd_rows(int64_t ld) { return ld % 8 != 0; }

// x and W with rows on 16 bytes: themselves, or copies in the workspace.
struct Inputs {
  const uint16_t *x, *w;
  int64_t ldx, ldw;
};

size_t inputs_bytes(int64_t M, int64_t I, int64_t K, int64_t ldx) {
  Space s{nullptr, 0};
  if (odd_rows(ldx) || K % 8) s.take((size_t)M * up(K, 8) * 2);
  if (K % 8) s.take((size_t)2 * I * up(K, 8) * 2);
  return s.used;
}

hipError_t lay_inputs(Inputs &in, int64_t M, int64_t I, int64_t K, Space &s, hipStream_t stream) {
  const int64_t kp = up(K, 8);
  if (odd_rows(in.ldx) || K % 8) {
    uint16_t *x = reinterpret_cast<uint16_t *>(s.take((size_t)M * kp * 2));
    if (hipError_t e = align_rows(in.x, in.ldx, M, K, x, stream)) return e;
    in.x = x;
    in.ldx = kp;
  }
  if (K % 8) {
    uint16_t *w = reinterpret_cast<uint16_t *>(s.take((size_t)2 * I * kp * 2));
    if (hipError_t e = align_rows(in.w, in.ldw, 2 * I, K, w, stream)) return e;
    in.w = w;
    in.ldw = kp;
  }
  return hipSuccess;
}

template <typename T>
hipError_t forward(const GatedCall &c, void *h, void *factors, void *work, hipStream_t stream) {
  Space s{static_cast<uint8_t *>(work), 0};
  Inputs in{static_cast<const uint16_t *>(c.x), static_cast<const uint16_t *>(c.w), c.ldx, c.K};
  if (hipError_t e = lay_inputs(in, c.M, c.I, c.K, s, stream)) return e;
  GluArgs p{};
  p.x = in.x; p.w = in.w; p.ldx = in.ldx; p.ldw = in.ldw;
  p.M = c.M; p.I = c.I; p.K = up(c.K, 8); p.act = c.act;
  p.h = static_cast<uint16_t *>(h);
  p.factors = static_cast<uint16_t *>(factors);
  return glu<T, false>(p, stream);
}

template <typename T>
hipError_t backward(const GatedCall &c, const void *dh, const void *factors, void *dx, void *dw,
                    void *work, hipStream_t stream) {
  Space s{static_cast<uint8_t *>(work), 0};
  Inputs in{static_cast<const uint16_t *>(c.x), static_cast<const uint16_t *>(c.w), c.ldx, c.K};
  if (hipError_t e = lay_inputs(in, c.M, c.I, c.K, s, stream)) return e;
  const int64_t ld = up(2 * c.I, 8), kp = up(c.K, 8);
  uint16_t *dgu = reinterpret_cast<uint16_t *>(s.take((size_t)c.M * ld * 2));
  if (factors) {
    factors_kernel<T><<<groups(c.M * tiles(c.I, 8)), 256, 0, stream>>>(
        static_cast<const uint16_t *>(dh), static_cast<const uint16_t *>(factors), c.M, c.I, dgu,
        ld);
    if (hipError_t e = hipGetLastError()) return e;
  } else {
    GluArgs p{};
    p.x = in.x; p.w = in.w; p.ldx = in.ldx; p.ldw = in.ldw;
    p.M = c.M; p.I = c.I; p.K = kp; p.act = c.act;
    p.dh = static_cast<const uint16_t *>(dh);
    p.dgu = dgu;
    p.ld_dgu = ld;
    if (hipError_t e = glu<T, true>(p, stream)) return e;
  }
  ProductArgs p{};
  p.parts = reinterpret_cast<float *>(s.base + s.used);   // one product after the other
  if (dx) {
    p.a = Operand{dgu, ld, c.M, ld};
    p.b = Operand{in.w, in.ldw, kp, 2 * c.I};
    p.rows = c.M; p.cols = c.K;
    p.out = static_cast<uint16_t *>(dx);
    if (hipError_t e = product<T, kRows, kCols>(p, stream)) return e;
  }
  if (dw) {
    p.a = Operand{dgu, ld, ld, c.M};
    p.b = Operand{in.x, in.ldx, kp, c.M};
    p.rows = 2 * c.I; p.cols = c.K;
    p.out = static_cast<uint16_t *>(dw);
    if (hipError_t e = product<T, kCols, kCols>(p, stream)) return e;
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
  return inputs_bytes(M, I, K, ldx);
}

hipError_t launch_gated(const GatedCall &c, void *h, void *factors, void *work,
                        hipStream_t stream) {
  return c.bf16 ? forward<Bf16>(c, h, factors, work, stream)
                : forward<F16>(c, h, factors, work, stream);
}

size_t gated_backward_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t ldx, bool dx,
                                      bool dw) {
  Space s{nullptr, inputs_bytes(M, I, K, ldx)};
  s.take((size_t)M * up(2 * I, 8) * 2);
  return s.used + std::max(dx ? part_bytes(M, K, up(2 * I, 8)) : 0,
                           dw ? part_bytes(2 * I, K, M) : 0);
}

hipError_t launch_gated_backward(const GatedCall &c, const void *dh, const void *factors, void *dx,
                                 void *dw, void *work, hipStream_t stream) {
  if (c.M == 0) return dw ? zero(dw, 2 * c.I * c.K, stream) : hipSuccess;
  if (c.I == 0) return dx ? zero(dx, c.M * c.K, stream) : hipSuccess;
  return c.bf16 ? backward<Bf16>(c, dh, factors, dx, dw, work, stream)
                : backward<F16>(c, dh, factors, dx, dw, work, stream);
}

}  // namespace fp8blk
