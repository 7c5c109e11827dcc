// 4-bit weights with a scale, and if wanted a zero point, per group of K, for gfx950:
//   W[n, k] = (q[n, k] - z[n, k / group]) * s[n, k / group],   q in 0..15,
// z = 8 where no zero points are kept.  Two codes a byte, even k in the low half;
// scales in the activations' type (bf16 or fp16), zero points a byte each.
#include "glu_tile.h"

namespace fp8blk {

using namespace t16;

namespace {

struct W4 {
  const uint8_t *codes;      // [rows, K / 2]
  const uint16_t *scale;     // [rows, K >> shift]
  const uint8_t *zeros;      // [rows, K >> shift] or NULL (8)
  int shift;                 // log2 of the group

  template <typename T, typename S>
  struct Pair;
};

// ---------------------------------------------------------------------------
// Quantization.  K is whole groups, so the codes, scales and zero points of a
// matrix are those of its groups one after another; GROUP / 8 neighbouring lanes
// hold a group, 8 weights each.
//
//   with zero points: s = T(fl32((hi - lo) / 15)), lo and hi its least and largest
//     weight with 0 among them; z = clamp(rint(-lo / s), 0, 15)
//   without: s = T(fl32(max |w| / 7)), z = 8
//   q = clamp(rint(w / s) + z, 0, 15);  s = 0: q = z (0 or 8).
// w and s are 16-bit floats: a quotient that is not half a whole number itself is
// far further from one than fp32's rounding, so rint of the fp32 quotient is that
// of the exact one.
//
// fl32(w / s): the product with the reciprocal, corrected once by its exact
// residual.  For tiny s both are scaled by 2^100 first (exactly), so that neither
// the reciprocal overflows nor the residual underflows.
struct Quotient {
  float f, s, y;
  __device__ __forceinline__ explicit Quotient(float step) {
    f = step < 0x1p-64f ? 0x1p100f : 1.0f;
    s = step * f;
    y = step > 0.0f ? 1.0f / s : 0.0f;
  }
  __device__ __forceinline__ float operator()(float w) const {
    const float v = w * f, q = v * y;
    return __builtin_fmaf(__builtin_fmaf(-q, s, v), y, q);
  }
};

template <typename T, int GROUP>
__global__ __launch_bounds__(256) void w4_quant_kernel(const uint16_t *w, int64_t chunks,
                                                       uint32_t *codes, uint16_t *scale,
                                                       uint8_t *zeros) {
  constexpr int kLanes = GROUP / 8;
  // chunks is whole groups, and a group's lanes share a wave: they run together
  for (int64_t at = first_item(); at < chunks; at += all_threads()) {
    const v4u v = *reinterpret_cast<const v4u *>(w + at * 8);
    float e[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e[2 * j] = T::value(v[j] & 0xffff);
      e[2 * j + 1] = T::value(v[j] >> 16);
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo = fminf(lo, e[j]);
      hi = fmaxf(hi, e[j]);
    }
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) {
      lo = fminf(lo, __shfl_xor(lo, d));
      hi = fmaxf(hi, __shfl_xor(hi, d));
    }
    const float range = zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
    const uint32_t bits = T::bits(range);
    const Quotient over(T::value(bits));
    const float z = zeros ? fminf(fmaxf(rintf(over(-lo)), 0.0f), 15.0f) : 8.0f;
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      c |= (uint32_t)fminf(fmaxf(rintf(over(e[j])) + z, 0.0f), 15.0f) << (4 * j);
    codes[at] = c;
    if (at % kLanes == 0) {
      scale[at / kLanes] = (uint16_t)bits;
      if (zeros) zeros[at / kLanes] = (uint8_t)z;
    }
  }
}

// Eight codes of a dword as fp32 weights, (q - z) s = q s - z s: both products have
// at most 4 + 11 bits, so each is exact and the sum rounds at most once (never in
// bf16's or fp16's range of scales: it has 5 + 11 bits).
__device__ __forceinline__ void decode8(uint32_t c, float s, float zs, float (&w)[8]) {
  const uint32_t even = c & 0x0f0f0f0fu, odd = (c >> 4) & 0x0f0f0f0fu;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[2 * j] = __builtin_fmaf((float)((even >> (8 * j)) & 0xffu), s, zs);
    w[2 * j + 1] = __builtin_fmaf((float)((odd >> (8 * j)) & 0xffu), s, zs);
  }
}
template <typename T>
__device__ __forceinline__ v4u decode16(uint32_t c, float s, float zs) {
  float w[8];
  decode8(c, s, zs, w);
  return v4u{pack2<T>(w[0], w[1]), pack2<T>(w[2], w[3]), pack2<T>(w[4], w[5]),
             pack2<T>(w[6], w[7])};
}

template <typename T>
__global__ __launch_bounds__(256) void w4_dequant_kernel(W4 p, int64_t chunks, uint16_t *w) {
  for (int64_t at = first_item(); at < chunks; at += all_threads()) {
    const int64_t g = at * 8 >> p.shift;
    const float s = T::value(p.scale[g]), z = p.zeros ? (float)p.zeros[g] : 8.0f;
    *reinterpret_cast<v4u *>(w + at * 8) =
        decode16<T>(reinterpret_cast<const uint32_t *>(p.codes)[at], s, -z * s);
  }
}

// ---------------------------------------------------------------------------
// Batches: the tiled product, the codes decoded on their way into LDS, once a
// workgroup.  A weight enters the product rounded to the activations' type, as
// fp8blk_w4_dequant gives it: at most half a step, an error of the size of the
// inputs' own rounding, for a product whose matrix instructions run as with 16-bit
// weights.
//
// A thread decodes half a stage of one row of W (32 codes, 16 bytes).
template <typename T, typename S>
struct W4Loader {
  static constexpr bool kRegs = true;
  static_assert(S::kThreads == 2 * S::TN, "two threads a row");
  const uint8_t *codes;
  const uint16_t *scale;
  const uint8_t *zeros;
  int row, half, shift;
  int64_t K;
  v4u c;
  float s, zs;

  // This thread's row of the tile is row `n` of the weights.
  __device__ __forceinline__ void at(const W4 &w, int64_t k, int64_t n) {
    K = k;
    shift = w.shift;
    row = threadIdx.x >> 1;
    half = threadIdx.x & 1;
    codes = w.codes + n * (K / 2) + half * 16;
    scale = w.scale + n * (K >> shift);
    zeros = w.zeros ? w.zeros + n * (K >> shift) : nullptr;
  }
  __device__ __forceinline__ void fetch(int step) {
    const int64_t k = (int64_t)step * kK + half * 32;
    const bool in = k < K;       // (K is a multiple of 32)
    const int64_t at = in ? (int64_t)step * 32 : 0, g = in ? k >> shift : 0;
    c = *reinterpret_cast<const v4u *>(codes + (in ? at : -half * 16));
    s = in ? T::value(scale[g]) : 0.0f;
    zs = -(zeros ? (float)zeros[g] : 8.0f) * s;
  }
  __device__ __forceinline__ void put(uint8_t *stage) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<v4u *>(stage + row * 128 + (((half * 4 + j) ^ swz_f(row)) << 4)) =
          decode16<T>(c[j], s, zs);
  }
};

}  // namespace

template <typename T, typename S>
struct W4::Pair : W4Loader<T, S> {
  __device__ __forceinline__ void init(const W4 &w, const GluArgs &p, int64_t n0, int, int) {
    const PairRow<S> r(threadIdx.x >> 1);
    this->at(w, p.K, r.half * p.I + min(n0 + r.c, p.I - 1));
  }
};

namespace {

template <typename T, typename S>
__global__ __launch_bounds__(S::kThreads) void w4_product_kernel(Operand a, W4 w, Out p) {
  __shared__ typename S::Smem sm;
  const int tiles = p.tiles_m * p.tiles_n, range = blockIdx.x / tiles;
  int tm, tn;
  tile_of(blockIdx.x - range * tiles, p.tiles_m, p.tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)tm * S::TM, n0 = (int64_t)tn * S::TN;
  a.p += m0 * a.ld;
  a.rows = min(a.rows - m0, (int64_t)S::TM);
  Loader<kRows, S::TM, S::kWaves> la;
  W4Loader<T, S> lb;
  la.init(a, wave, lane);
  lb.at(w, a.k, min(n0 + (int64_t)(threadIdx.x >> 1), p.cols - 1));
  const int s0 = p.first_step(range);
  v4f acc[S::kFM][S::kFN];
  multiply<T, S, kRows, kRows>(la, lb, s0, p.first_step(range + 1) - s0, sm, acc);
  store_tile<T, S>(p, acc, m0, n0, range);
}

__global__ __launch_bounds__(256) void align_x_kernel(const uint16_t *in, int64_t ld, int64_t rows,
                                                      int64_t cols, uint16_t *out) {
  align_rows(in, ld, rows, cols, out, cols);
}

// ---------------------------------------------------------------------------
// Host side.

W4 weights(const W4Call &c) {
  return {static_cast<const uint8_t *>(c.codes), static_cast<const uint16_t *>(c.scale),
          static_cast<const uint8_t *>(c.zeros), c.group == 32 ? 5 : c.group == 64 ? 6 : 7};
}

// x with rows on 16 bytes: itself, or a copy in the workspace (K is whole chunks).
void x_space(int64_t M, int64_t K, int64_t ldx, Space &s) {
  if (ldx % 8) s.take((size_t)M * K * 2);
}
hipError_t lay_x(const W4Call &c, Operand &a, Space &s, hipStream_t stream) {
  a = Operand{static_cast<const uint16_t *>(c.x), c.ldx, c.M, c.K};
  if (c.ldx % 8 == 0) return hipSuccess;
  uint16_t *x = reinterpret_cast<uint16_t *>(s.take((size_t)c.M * c.K * 2));
  align_x_kernel<<<groups(c.M * (c.K / 8)), 256, 0, stream>>>(a.p, a.ld, c.M, c.K, x);
  a.p = x;
  a.ld = c.K;
  return hipGetLastError();
}

template <typename T>
hipError_t linear(const W4Call &c, void *y, void *work, hipStream_t stream) {
  Space s{static_cast<uint8_t *>(work), 0};
  Operand a;
  if (hipError_t e = lay_x(c, a, s, stream)) return e;
  const Plan plan = plan_of(c.M, c.rows, c.K);
  Out p{c.M, c.rows, static_cast<uint16_t *>(y), reinterpret_cast<float *>(s.base + s.used)};
  p.steps = (int)tiles(c.K, kK);
  p.ranges = plan.ranges;
  p.tiles_m = (int)tiles(p.rows, plan.large ? Large::TM : Small::TM);
  p.tiles_n = (int)tiles(p.cols, plan.large ? Large::TN : Small::TN);
  const dim3 grid((unsigned)p.tiles_m * p.tiles_n * p.ranges);
  if (plan.large) w4_product_kernel<T, Large><<<grid, Large::kThreads, 0, stream>>>(a, weights(c), p);
  else w4_product_kernel<T, Small><<<grid, Small::kThreads, 0, stream>>>(a, weights(c), p);
  if (p.ranges > 1) {
    if (hipError_t e = hipGetLastError()) return e;
    join_kernel<T><<<groups(tiles(p.rows * p.cols, 4)), 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t gated(const W4Call &c, int act, void *h, void *work, hipStream_t stream) {
  Space s{static_cast<uint8_t *>(work), 0};
  Operand a;
  if (hipError_t e = lay_x(c, a, s, stream)) return e;
  GluArgs p{};
  p.x = a.p;
  p.ldx = a.ld;
  p.M = c.M;
  p.I = c.rows / 2;
  p.K = c.K;
  p.act = act;
  p.h = static_cast<uint16_t *>(h);
  p.parts = reinterpret_cast<float *>(s.base + s.used);
  return launch_glu<T, false>(p, weights(c), stream);
}

template <typename T>
hipError_t quant(const void *w, int64_t chunks, int group, void *codes, void *scale, void *zeros,
                 hipStream_t stream) {
  const uint16_t *in = static_cast<const uint16_t *>(w);
  uint32_t *q = static_cast<uint32_t *>(codes);
  uint16_t *s = static_cast<uint16_t *>(scale);
  uint8_t *z = static_cast<uint8_t *>(zeros);
  if (group == 32) w4_quant_kernel<T, 32><<<groups(chunks), 256, 0, stream>>>(in, chunks, q, s, z);
  else if (group == 64) w4_quant_kernel<T, 64><<<groups(chunks), 256, 0, stream>>>(in, chunks, q, s, z);
  else w4_quant_kernel<T, 128><<<groups(chunks), 256, 0, stream>>>(in, chunks, q, s, z);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_quant(const void *w, bool bf16, int64_t rows, int64_t K, int group,
                           void *codes, void *scale, void *zeros, hipStream_t stream) {
  const int64_t chunks = rows * (K / 8);
  return bf16 ? quant<Bf16>(w, chunks, group, codes, scale, zeros, stream)
              : quant<F16>(w, chunks, group, codes, scale, zeros, stream);
}

hipError_t launch_w4_dequant(const W4Call &c, void *w, hipStream_t stream) {
  const int64_t chunks = c.rows * (c.K / 8);
  uint16_t *out = static_cast<uint16_t *>(w);
  if (c.bf16) w4_dequant_kernel<Bf16><<<groups(chunks), 256, 0, stream>>>(weights(c), chunks, out);
  else w4_dequant_kernel<F16><<<groups(chunks), 256, 0, stream>>>(weights(c), chunks, out);
  return hipGetLastError();
}

bool w4_fits(int64_t M, int64_t rows) {
  return grid_of<Large>(M, rows) < (int64_t(1) << 32) / Large::kThreads;
}

size_t w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t ldx) {
  Space s{nullptr, 0};
  x_space(M, K, ldx, s);
  const int r = plan_of(M, N, K).ranges;
  return s.used + (r == 1 ? 0 : (size_t)r * M * N * sizeof(float));
}

size_t w4_gated_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t ldx) {
  Space s{nullptr, 0};
  x_space(M, K, ldx, s);
  return s.used + glu_part_bytes(M, I, K);
}

hipError_t launch_w4_linear(const W4Call &c, void *y, void *work, hipStream_t stream) {
  return c.bf16 ? linear<Bf16>(c, y, work, stream) : linear<F16>(c, y, work, stream);
}

hipError_t launch_w4_gated(const W4Call &c, int act, void *h, void *work, hipStream_t stream) {
  return c.bf16 ? gated<Bf16>(c, act, h, work, stream) : gated<F16>(c, act, h, work, stream);
}

}  // namespace fp8blk
