// 4-bit weights with a scale, and if wanted a zero point, per group of K, for gfx950:
//   W[n, k] = (q[n, k] - z[n, k / group]) * s[n, k / group],   q in 0..15,
// z = 8 where no zero points are kept.  Two codes a byte, even k in the low half;
// scales in the activations' type (bf16 or fp16), zero points a byte each.
//
// Measured on one MI355X:
//   quantizer, 18432 x 7168          57 us, and back 48: HBM (0.33 GB: 5.9, 6.9 TB/s)
//   1 x 14336 -> 4096                9.1 us: four waves' two rounds of 2048 of K, the second
//                                    loaded behind the first's products
//   1 x 4096 -> 14336, gated         14.2 us: HBM
//   37 x 7168 -> 2111                16.5 us: the loads' latency, 7 chunks a wave
//   128 x 4096 -> 14336, gated       61 us: a stage's latency and its decoding
//   2048 x 7168 -> 18432             560 us, 0.97 PFLOP/s: vector instructions (69 % of the
//                                    busy cycles: decoding, and the multiply-adds that scale
//                                    each group's sum) beside the matrix ones (48 %); LDS
//                                    bank conflicts (18 %, their source not found)
#include "glu_tile.h"

namespace fp8blk {

using namespace t16;

namespace {

struct Weights {
  const uint8_t *codes;      // [rows, K / 2]
  const uint16_t *scale;     // [rows, K >> shift]
  const uint8_t *zeros;      // [rows, K >> shift] or NULL (8)
  int shift;                 // log2 of the group
};

// ---------------------------------------------------------------------------
// Quantization.  K is whole groups, so the codes, scales and zero points of a
// matrix are those of its groups one after another; GROUP / 8 neighbouring lanes
// hold a group, 8 weights each.
//
//   with zero points: s = T(fl32((hi - lo) / 15)), lo and hi its least and largest
//     weight with 0 among them; z = clamp(rint(-lo / s), 0, 15)
//   without: s = T(fl32(max |w| / 7)), z = 8
//   q = clamp(rint(w / s) + z, 0, 15);  s = 0, infinite or NaN: q = z (0 or 8).
// A NaN in a group makes s NaN, an infinity makes it infinite (both maxima and minima
// hand NaN on), so that neither is taken for a weight.
// w and s are 16-bit floats: a quotient that is not half a whole number itself is
// far further from one than fp32's rounding, so rint of the fp32 quotient is that
// of the exact one.
//
// The quotient w / s: the product with the reciprocal, corrected once by its exact
// residual, which makes it exact where it is representable (half whole numbers, ties,
// are).  For tiny s both are scaled by 2^100 first (exactly), so that neither the
// reciprocal overflows nor the residual underflows.
struct Quotient {
  float f, s, y;
  __device__ __forceinline__ explicit Quotient(float step) {
    f = step < 0x1p-64f ? 0x1p100f : 1.0f;
    s = step * f;
    y = step > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
  }
  // rint(w / s), of quotients far below 2^22: 1.5 2^23 + it, whose low bits it is.
  __device__ __forceinline__ int operator()(float w) const {
    const float v = w * f, q = v * y;
    return __float_as_int(__builtin_fmaf(__builtin_fmaf(-q, s, v), y, q) + 0x1.8p23f) - 0x4b400000;
  }
};
// fl32(a / D) of a small odd D.  What the one correction leaves wrong is below 2^-24
// of the last place, and a / D lies 1 / (2 D) of a place off any tie.  An infinity has no
// residual and stays one.
template <int D>
__device__ __forceinline__ float over(float a) {
  constexpr float kInverse = 1.0f / D;
  const float q = a * kInverse;
  return a < __builtin_inff() ? __builtin_fmaf(__builtin_fmaf(-q, (float)D, a), kInverse, q) : a;
}
// f over the LANES (4, 8 or 16) neighbouring lanes of a group: lanes trade 1 and 2 apart,
// then halves of 8 and of 16 mirrored, equal within themselves by then.
template <int LANES, typename V, typename F>
__device__ __forceinline__ V over_lanes(V v, F f) {
  static_assert(sizeof(V) == 4 && (LANES == 4 || LANES == 8 || LANES == 16), "");
  auto from = [](V u, auto ctrl) {
    return __builtin_bit_cast(
        V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, u), ctrl.value, 0xf, 0xf, true));
  };
  v = f(v, from(v, std::integral_constant<int, 0xb1>{}));      // 1 0 3 2
  v = f(v, from(v, std::integral_constant<int, 0x4e>{}));      // 2 3 0 1
  if constexpr (LANES >= 8) v = f(v, from(v, std::integral_constant<int, 0x141>{}));
  if constexpr (LANES >= 16) v = f(v, from(v, std::integral_constant<int, 0x140>{}));
  return v;
}

// Chunks a thread loads ahead (18432 x 7168: one 61 us, two 57, four 55 to quantize; back,
// two 47, four 55), w past the caches (back by plain stores: 60).
constexpr int kAhead = 2;

// Bound: HBM, with about as much time in vector instructions, hence the reciprocals and
// lane exchanges above (divisions and shuffles: 76 us at 18432 x 7168, 66 without them and
// one chunk a thread, now 57).
template <typename T, int GROUP, bool ZEROS>
__global__ __launch_bounds__(256) void w4_quant_kernel(const uint16_t *w, int64_t chunks,
                                                       uint32_t *codes, uint16_t *scale,
                                                       uint8_t *zeros) {
  constexpr int kLanes = GROUP / 8;
  auto one = [&](int64_t at, v4u v) {
    float e[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e[2 * j] = T::value(v[j] & 0xffff);
      e[2 * j + 1] = T::value(v[j] >> 16);
    }
    float range, lo = 0.0f;
    if constexpr (ZEROS) {
      float hi = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo = __builtin_elementwise_minimum(lo, e[j]);
        hi = __builtin_elementwise_maximum(hi, e[j]);
      }
      lo = over_lanes<kLanes>(lo, [](float a, float b) { return __builtin_elementwise_minimum(a, b); });
      hi = over_lanes<kLanes>(hi, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
      range = over<15>(hi - lo);
    } else {
      // magnitudes are ordered as their bits are
      typedef unsigned short v2us __attribute__((ext_vector_type(2)));
      auto larger = [](v2us a, v2us b) { return __builtin_elementwise_max(a, b); };
      v2us m = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = larger(m, __builtin_bit_cast(v2us, v[j] & 0x7fff7fffu));
      m = over_lanes<kLanes>(m, larger);
      range = over<7>(T::value(m[0] > m[1] ? m[0] : m[1]));
    }
    const uint32_t bits = T::bits(range);
    const float step = T::value(bits);
    const Quotient quotient(step);
    const bool finite = step < __builtin_inff();      // (not of NaN)
    const int z = ZEROS ? (finite ? min(max(quotient(-lo), 0), 15) : 0) : 8;
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) c |= (uint32_t)min(max(quotient(e[j]) + z, 0), 15) << (4 * j);
    if (!finite) c = ZEROS ? 0u : 0x88888888u;
    __builtin_nontemporal_store(c, codes + at);
    if (at % kLanes == 0) {
      scale[at / kLanes] = (uint16_t)bits;
      if constexpr (ZEROS) zeros[at / kLanes] = (uint8_t)z;
    }
  };
  // chunks is whole groups, and a group's lanes share a wave: they run together
  for (int64_t at = (int64_t)blockIdx.x * (256 * kAhead) + threadIdx.x; at < chunks;
       at += (int64_t)gridDim.x * (256 * kAhead)) {
    v4u v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      v[i] = __builtin_nontemporal_load(
          reinterpret_cast<const v4u *>(w + min(at + i * 256, chunks - 1) * 8));
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (at + i * 256 < chunks) one(at + i * 256, v[i]);
  }
}

// Eight codes of a dword less their zero point, as fp32: whole numbers from -15
// to 15.
__device__ __forceinline__ void decode8(uint32_t c, float z, float (&w)[8]) {
  const uint32_t even = c & 0x0f0f0f0fu, odd = (c >> 4) & 0x0f0f0f0fu;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[2 * j] = (float)((even >> (8 * j)) & 0xffu) - z;
    w[2 * j + 1] = (float)((odd >> (8 * j)) & 0xffu) - z;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void w4_dequant_kernel(Weights p, int64_t chunks, uint16_t *w) {
  for (int64_t from = (int64_t)blockIdx.x * (256 * kAhead) + threadIdx.x; from < chunks;
       from += (int64_t)gridDim.x * (256 * kAhead)) {
    uint32_t c[kAhead];
    float s[kAhead], z[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = min(from + i * 256, chunks - 1), g = at * 8 >> p.shift;
      c[i] = reinterpret_cast<const uint32_t *>(p.codes)[at];
      s[i] = T::value(p.scale[g]);
      z[i] = p.zeros ? (float)p.zeros[g] : 8.0f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = from + i * 256;
      float v[8];     // (the products are exact in fp32: at most 5 + 11 bits)
      decode8(c[i], z[i], v);
      if (at < chunks)
        __builtin_nontemporal_store(
            v4u{pack2<T>(v[0] * s[i], v[1] * s[i]), pack2<T>(v[2] * s[i], v[3] * s[i]),
                pack2<T>(v[4] * s[i], v[5] * s[i]), pack2<T>(v[6] * s[i], v[7] * s[i])},
            reinterpret_cast<v4u *>(w + at * 8));
    }
  }
}

// ---------------------------------------------------------------------------
// Batches: the tiled product, the codes decoded on their way into LDS, once a
// workgroup, as whole numbers (q - z), which bf16 and fp16 hold exactly.  The
// matrix instructions form a group's sum (or 64 of a longer one's), and one fp32
// multiply-add an output puts it on the accumulator with its scale.  Weights
// rounded to 16 bits instead, with the scale, would take no such multiply-adds and
// carry an error as large as the result's own rounding into it.

// Eight codes less their zero point as 16-bit floats, in the order of k: in bf16 the
// upper halves of the fp32 values (exact), in fp16 by 1024 + q, whose low bits are q,
// less 1024 + z.
template <typename T>
__device__ __forceinline__ v4u whole16(uint32_t c, float z);
template <>
__device__ __forceinline__ v4u whole16<Bf16>(uint32_t c, float z) {
  float w[8];
  decode8(c, z, w);
  v4u out;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    out[j] = __builtin_amdgcn_perm(__float_as_uint(w[2 * j + 1]), __float_as_uint(w[2 * j]),
                                   0x07060302u);
  return out;
}
template <>
__device__ __forceinline__ v4u whole16<F16>(uint32_t c, float z) {
  const _Float16 bias = (_Float16)(1024.0f + z);
  uint32_t p[4];      // codes j and j + 4
#pragma unroll
  for (int j = 0; j < 4; ++j)
    p[j] = __builtin_bit_cast(
        uint32_t, __builtin_bit_cast(F16::Pair, ((c >> (4 * j)) & 0x000f000fu) | 0x64006400u) -
                      F16::Pair{bias, bias});
  return v4u{__builtin_amdgcn_perm(p[1], p[0], 0x05040100u),
             __builtin_amdgcn_perm(p[3], p[2], 0x05040100u),
             __builtin_amdgcn_perm(p[1], p[0], 0x07060302u),
             __builtin_amdgcn_perm(p[3], p[2], 0x07060302u)};
}

template <typename S>
struct W4Smem : S::Smem {
  float scale[2][2][S::TN];      // by stage and half of its K
};

// A thread decodes half a stage of one row of W (32 codes, 16 bytes); neighbouring
// lanes take neighbouring rows, whose chunks fall into different banks.
template <typename T, typename S>
struct W4Loader {
  static_assert(S::kThreads == 2 * S::TN, "two threads a row");
  const uint8_t *codes;
  const uint16_t *scale;
  const uint8_t *zeros;
  int row, half, shift;
  int64_t K;
  v4u next;              // fetched
  uint32_t next_s, next_z;
  bool in, has_zeros;
  v4u c;                 // taken
  float s, z;

  static __device__ __forceinline__ int tile_row() {
    return (threadIdx.x >> 6) * 32 + (threadIdx.x & 31);
  }
  // This thread's row of the tile is row `n` of the weights.
  __device__ __forceinline__ void at(const Weights &w, int64_t k, int64_t n) {
    K = k;
    shift = w.shift;
    row = tile_row();
    half = (threadIdx.x >> 5) & 1;
    codes = w.codes + n * (K / 2) + half * 16;
    scale = w.scale + n * (K >> shift);
    has_zeros = w.zeros != nullptr;
    // (without zero points their loads bring bytes of the scales, not used)
    zeros = (has_zeros ? w.zeros : reinterpret_cast<const uint8_t *>(w.scale)) + n * (K >> shift);
  }
  // Loads without branches, which the unrolled loop around them would pay for.
  __device__ __forceinline__ void fetch(int step) {
    const int64_t k = (int64_t)step * kK + half * 32;
    in = k < K;       // (K is a multiple of 32; past it the scale is zero)
    const int64_t at = in ? (int64_t)step * 32 : -half * 16, g = in ? k >> shift : 0;
    next = *reinterpret_cast<const v4u *>(codes + at);
    next_s = scale[g];
    next_z = zeros[g];
  }
  __device__ __forceinline__ void take() {
    c = next;
    s = in ? T::value(next_s) : 0.0f;
    z = has_zeros ? (float)next_z : 8.0f;
  }
  // Quarter j of the codes taken into a stage.
  __device__ __forceinline__ void put(W4Smem<S> &sm, int stage, int j) const {
    *reinterpret_cast<v4u *>(sm.b[stage] + row * 128 + (((half * 4 + j) ^ swz_f(row)) << 4)) =
        whole16<T>(c[j], z);
    if (j == 0) sm.scale[stage][half][row] = s;
  }
};

// G32: groups of 32, two a stage; else a stage lies within a group.
template <bool G32>
struct W4 : Weights {
  static constexpr bool kFourBits = true;
  // (a lane then holds outputs of one column of each fragment: one scale)
  template <typename S>
  using Place = typename S::Across;
  template <typename S>
  using Smem = W4Smem<S>;
  template <typename T, typename S>
  struct Pair : W4Loader<T, S> {
    __device__ __forceinline__ void init(const W4 &w, const GluArgs &p, int64_t n0, int, int) {
      const PairRow<S> r(W4Loader<T, S>::tile_row());
      this->at(w, p.K, r.half * p.I + min(n0 + r.c, p.I - 1));
    }
  };

  // As t16::multiply, with the groups' scales: the multiply-adds of a row of
  // fragments follow the next row's matrix instructions, whose results they do not
  // wait for.  The codes of the stage after next are fetched at a step's start and
  // taken at its barrier, to be decoded into the stage just read among the next step's
  // rows of fragments.
  // Past the last step the last stage is brought again, and not read.
  template <typename T, typename S, typename LA, typename LB>
  static __device__ __forceinline__ void multiply(const LA &la, LB &lb, int step0, int steps,
                                                  W4Smem<S> &sm, typename S::Acc &acc) {
    const int lane = threadIdx.x & 63;
    constexpr int FM = S::kFM, FN = S::kFN, kParts = G32 ? 2 : 1, kUnits = FM * kParts;
    const int arow = wave_row<S>(), brow = wave_col<S>();
#pragma unroll
    for (int mi = 0; mi < FM; ++mi)
#pragma unroll
      for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = v4f{0, 0, 0, 0};
    auto at = [&](int s) { return step0 + min(s, steps - 1); };
    auto read_a = [&](int st, int mi) {
      return read_frag<kRows, S::TM>(sm.a[st], arow + mi * 16, lane);
    };
    auto read_b = [&](int st, int ni) {
      return read_frag<kRows, S::TN>(sm.b[st], brow + ni * 16, lane);
    };
    auto read_scale = [&](int st, int ni, int h) {
      return sm.scale[st][h][brow + ni * 16 + (lane & 15)];
    };
    la.issue(at(0), sm.a[0]);
    la.issue(at(1), sm.a[1]);
    lb.fetch(at(0));
    lb.take();
#pragma unroll
    for (int j = 0; j < 4; ++j) lb.put(sm, 0, j);
    lb.fetch(at(1));
    lb.take();
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    Frag bf[FN], af = read_a(0, 0);
    float scale[FN][kParts];
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) {
      bf[ni] = read_b(0, ni);
#pragma unroll
      for (int h = 0; h < kParts; ++h) scale[ni][h] = read_scale(0, ni, h);
    }
    // unit u: a row of fragments over a stage, or over half of one
    v4f part[2][FN];
    for (int s = 0; s < steps; ++s) {
      const int st = s & 1;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int mi = u / kParts, h = u % kParts;
        const bool last = u == kUnits - 1;
        // quarters of the next stage's codes, taken at the last barrier
        auto put = [&]() {
          constexpr int kEach = kUnits >= 4 ? 1 : 4 / kUnits;
#pragma unroll
          for (int j = u * kEach; j < (u + 1) * kEach && j < 4; ++j) lb.put(sm, st ^ 1, j);
        };
        if (u == 0) lb.fetch(at(s + 2));
        if (last) put();
        Frag an;
        if (h == kParts - 1) {
          if (!last) {
            an = read_a(st, mi + 1);
          } else {
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
            la.issue(at(s + 2), sm.a[st]);
            lb.take();
            an = read_a(st ^ 1, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ni = 0; ni < FN; ++ni)
          part[u & 1][ni] = T::mfma(af.h[h], bf[ni].h[h], v4f{0, 0, 0, 0});
        if constexpr (!G32) {
#pragma unroll
          for (int ni = 0; ni < FN; ++ni)
            part[u & 1][ni] = T::mfma(af.h[1], bf[ni].h[1], part[u & 1][ni]);
        }
        // the unit before this one
        if (u > 0) {
          const int m = (u - 1) / kParts, p = (u - 1) % kParts;
#pragma unroll
          for (int ni = 0; ni < FN; ++ni)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][ni][r] =
                  __builtin_fmaf(part[(u - 1) & 1][ni][r], scale[ni][p], acc[m][ni][r]);
        }
        if (!last) put();
        // vector instructions in the shadow of each matrix instruction
#pragma unroll
        for (int i = 0; i < (G32 ? FN : 2 * FN); ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (u < 4) __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
          else __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (h == kParts - 1) af = an;
      }
#pragma unroll
      for (int ni = 0; ni < FN; ++ni) {
        bf[ni] = read_b(st ^ 1, ni);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[FM - 1][ni][r] = __builtin_fmaf(part[(kUnits - 1) & 1][ni][r],
                                              scale[ni][kParts - 1], acc[FM - 1][ni][r]);
#pragma unroll
        for (int h = 0; h < kParts; ++h) scale[ni][h] = read_scale(st ^ 1, ni, h);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // LDS is left with no load into it in flight
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  }
};

template <typename T, typename Tile, bool G32>
__global__ __launch_bounds__(Tile::kThreads) void w4_product_kernel(Operand a, W4<G32> w, Out p) {
  using S = typename Tile::Across;
  __shared__ W4Smem<S> sm;
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
  lb.at(w, a.k, min(n0 + (int64_t)W4Loader<T, S>::tile_row(), p.cols - 1));
  const int s0 = p.first_step(range);
  typename S::Acc acc;
  W4<G32>::template multiply<T, S>(la, lb, s0, p.first_step(range + 1) - s0, sm, acc);
  store_tile<T, S>(p, acc, m0, n0, range, reinterpret_cast<uint8_t *>(&sm));
}

// ---------------------------------------------------------------------------
// One or two rows of x (single decoding sequences): the weights stream past once, a
// wave per few rows of W, 32 codes a lane and row.  Bound: HBM traffic of the
// codes.
//
// Codes become 16-bit floats 16 + q by placing them in the mantissa of 16, two at a
// time; the dot product's instruction takes them by pairs (k, k + 4) against x in
// the same order, and what the 16 and the zero point add is taken off the 32 codes'
// sum, (16 + z) times the sum of their x.  The bias is of the codes' own size, so
// nothing is lost to it in fp32 (128 + q would cost three bits more).
template <typename T>
struct Pairs;
template <>
struct Pairs<Bf16> {
  typedef __bf16 V __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kOne = 0x3f803f80u;
  static __device__ __forceinline__ float dot(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c,
                                           false);
  }
  template <int J>   // codes J and J + 4 of a dword
  static __device__ __forceinline__ uint32_t codes(uint32_t c) {
    uint32_t v = c << 3;
    if constexpr (J > 0) v = c >> (4 * J - 3);
    return (v & 0x00780078u) | 0x41804180u;
  }
};
template <>
struct Pairs<F16> {
  typedef _Float16 V __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kOne = 0x3c003c00u;
  static __device__ __forceinline__ float dot(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, false);
  }
  template <int J>
  static __device__ __forceinline__ uint32_t codes(uint32_t c) {
    const uint32_t v = J == 0 ? c << 6 : J == 1 ? c << 2 : J == 2 ? c >> 2 : c >> 6;
    return (v & 0x03c003c0u) | 0x4c004c00u;
  }
};

// x's 8 values at k as pairs (k, k + 4).
__device__ __forceinline__ v4u pair_order(v4u x) {
  return v4u{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u),
             __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
             __builtin_amdgcn_perm(x[3], x[1], 0x05040100u),
             __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

struct W4Few {
  Weights w;
  const uint16_t *x;
  int64_t ldx, K, I;      // I: outputs (rows of W, or half of them)
  int M, act;
  uint16_t *out;          // [M, I]
};

// Where the sum with the bias is not finite, the output is formed again from codes less
// their zero point, as the tiles do it.  The bias makes NaN of an infinite x (the same
// infinity is added and taken off) and may pass fp32's range where the sum does not.
// A wave together, a row's outputs one after another; a row with a NaN, as the unused
// rows of a padded batch may hold, is NaN without them.
__device__ __forceinline__ bool finite(float v) {
  return __builtin_fabsf(v) < __builtin_inff();
}
template <typename T>
__device__ __forceinline__ float w4_plain(const W4Few &p, int64_t m, int64_t n, int lane) {
  const uint16_t *x = p.x + m * p.ldx;
  const uint8_t *codes = p.w.codes + n * (p.K / 2);
  const int64_t first = n * (p.K >> p.w.shift);
  float acc = 0.0f;
#pragma unroll 1
  for (int64_t k = lane * 8; k < p.K; k += 512) {      // (8 of K are in one group)
    const int64_t at = first + (k >> p.w.shift);
    const v4u v = *reinterpret_cast<const v4u_any *>(x + k);
    float w[8], sum = 0.0f;
    decode8(*reinterpret_cast<const uint32_t *>(codes + k / 2),
            p.w.zeros ? (float)p.w.zeros[at] : 8.0f, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum = __builtin_fmaf(w[2 * j], T::value(v[j] & 0xffff), sum);
      sum = __builtin_fmaf(w[2 * j + 1], T::value(v[j] >> 16), sum);
    }
    acc = __builtin_fmaf(sum, T::value(p.w.scale[at]), acc);
  }
  for (int d = 32; d >= 1; d /= 2) acc += __shfl_xor(acc, d);
  return acc;
}
// Whether row m of x holds a NaN, by a wave.
template <typename T>
__device__ __forceinline__ bool w4_nan_row(const W4Few &p, int64_t m, int lane) {
  const uint16_t *x = p.x + m * p.ldx;
  bool nan = false;
#pragma unroll 2
  for (int64_t k = lane * 8; k < p.K; k += 512) {
    const v4u v = *reinterpret_cast<const v4u_any *>(x + k);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      nan |= __builtin_isunordered(T::value(v[j] & 0xffff), T::value(v[j] >> 16));
  }
  return __ballot(nan) != 0;
}
// v, output n of row m, if it is finite, else that sum (by a whole wave; lanes without an
// output bring a zero).
template <typename T>
__device__ __forceinline__ float w4_finish(const W4Few &p, float v, int m, int64_t n, int lane) {
  for (uint64_t left = __ballot(!finite(v)); left;) {
    const int row = __shfl(m, __builtin_ctzll(left));
    uint64_t same = left & __ballot(m == row);      // the row's
    left &= ~same;
    if (w4_nan_row<T>(p, row, lane)) {
      if (same >> lane & 1) v = __builtin_nanf("");
      continue;
    }
    for (; same; same &= same - 1) {
      const int from = __builtin_ctzll(same);
      const float sum = w4_plain<T>(p, row, __shfl((long long)n, from), lane);
      if (lane == from) v = sum;
    }
  }
  return v;
}

// R outputs a wave, MT rows of x (M of them there), the K range shared by KS waves.
template <typename T, bool PAIR, int R, int MT, int KS>
__global__ __launch_bounds__(256) void w4_few_kernel(W4Few p) {
  using P = Pairs<T>;
  constexpr int kHalves = PAIR ? 2 : 1, kRows = R * kHalves, kOuts = 4 / KS * R;
  __shared__ float red[4][kRows * MT];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kOuts;
  const uint8_t *codes[kRows];
  int64_t at[kRows];        // first scale of the row
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t n = min(n0 + wave / KS * R + i % R, p.I - 1) + (i >= R ? p.I : 0);
    codes[i] = p.w.codes + n * (p.K / 2) + lane * 16;
    at[i] = n * (p.K >> p.w.shift);
  }
  float acc[kRows * MT];
#pragma unroll
  for (int i = 0; i < kRows * MT; ++i) acc[i] = 0.0f;
  for (int64_t k0 = (int64_t)(wave % KS) * 2048; k0 < p.K; k0 += KS * 2048) {
    const int64_t k = k0 + lane * 32;
    const bool in = k < p.K;          // (K is a multiple of 32)
    v4u c[kRows];
    float s[kRows], z[kRows];
    const int64_t g = in ? k >> p.w.shift : 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      c[i] = *reinterpret_cast<const v4u *>(codes[i] + (in ? k0 / 2 : -(int64_t)lane * 16));
    v4u xv[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint16_t *x = p.x + min(m, p.M - 1) * p.ldx + (in ? k : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) xv[m][j] = *reinterpret_cast<const v4u_any *>(x + 8 * j);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      s[i] = T::value(p.w.scale[at[i] + g]);
      z[i] = p.w.zeros ? (float)p.w.zeros[at[i] + g] : 8.0f;
    }
    float sum[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      sum[m] = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xv[m][j] = in ? pair_order(xv[m][j]) : v4u{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[m] = P::dot(xv[m][j][i], P::kOne, sum[m]);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float part[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) part[m] = -(16.0f + z[i]) * sum[m];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t q[4] = {P::template codes<0>(c[i][j]), P::template codes<1>(c[i][j]),
                               P::template codes<2>(c[i][j]), P::template codes<3>(c[i][j])};
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[m] = P::dot(q[e], xv[m][j][e], part[m]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
        acc[i * MT + m] = __builtin_fmaf(part[m], s[i], acc[i * MT + m]);
    }
  }
  wave_sums<kRows * MT>(acc, red[wave], lane);
  __syncthreads();
  // a thread an output
  static_assert(kOuts * MT <= 64, "a wave's");
  if (wave) return;
  const int m = lane % MT, o = lane / MT, r = o % R, w0 = o / R * KS;
  const int64_t n = n0 + o;
  const bool there = lane < kOuts * MT && m < p.M && n < p.I;
  float v[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    v[h] = 0.0f;
    if (there) {
#pragma unroll
      for (int i = 0; i < KS; ++i) v[h] += red[w0 + i][(h * R + r) * MT + m];
    }
    v[h] = w4_finish<T>(p, v[h], m, n + h * p.I, lane);
  }
  if (!there) return;
  float y = v[0];
  if constexpr (PAIR) y = act_any(p.act, v[0]) * v[1];
  p.out[m * p.I + n] = (uint16_t)T::bits(y);
}

// ---------------------------------------------------------------------------
// Up to 48 rows of x (decode batches): matrix instructions on codes that never pass
// through LDS.  A workgroup's eight waves share NR blocks of 16 rows of W and split K
// among them, 128 at a time.  A wave loads its codes and x row by row (16 bytes a lane,
// neighbouring lanes on neighbouring bytes: loaded in the instructions' order, a row
// a lane, 16 rows of 14336 -> 4096 took 22.8 us instead of 13.7) and turns them through
// LDS of its own; a 4 x 4 exchange of dwords among the four lanes of a row of codes
// then gives each instruction 32 neighbouring K, so a group never shares one with
// another.  No wave waits for another until their sums meet at the end.  Codes enter
// as 16 + q (see above), x in the same order of k; the sums of x that the bias asks
// for come from one more instruction on ones, for all blocks together.  Bound: the
// codes' HBM traffic, then x's from L2 (4 MF / NR bytes a byte of codes).
//
// GS: groups in 128 of K; MF: blocks of 16 rows of x.
template <typename T, bool PAIR, int GS, int NR, int MF>
__global__ __launch_bounds__(512, MF == 1 ? 4 : 2) void w4_slab_kernel(W4Few p) {
  using P = Pairs<T>;
  constexpr int kWaves = 8, kOut = PAIR ? NR / 2 : NR;
  // a wave's codes and x on their way to the instructions' order, then its sums
  struct Wave {
    uint8_t w[NR][16 * 64], x[MF][16 * 256];
  };
  union Smem {
    Wave wave[kWaves];
    float red[kWaves][NR * MF * 4][64];
  };
  __shared__ __align__(16) Smem sm;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (kOut * 16);
  const int64_t groups = p.K >> p.w.shift;
  // loads: four lanes on a row's 64 bytes of codes, sixteen on a row's 256 bytes of x
  const uint8_t *codes[NR];
  const uint16_t *scale[NR];
  const uint8_t *zeros[NR];
  const bool has_zeros = p.w.zeros != nullptr;
#pragma unroll
  for (int b = 0; b < NR; ++b) {
    const int64_t from = n0 + b % kOut * 16, half = b >= kOut ? p.I : 0;
    codes[b] = p.w.codes + (min(from + (lane >> 2), p.I - 1) + half) * (p.K / 2);
    const int64_t n = min(from + r16, p.I - 1) + half;
    scale[b] = p.w.scale + n * groups;
    // (without zero points their loads bring bytes of the scales, not used)
    zeros[b] = (has_zeros ? p.w.zeros : reinterpret_cast<const uint8_t *>(p.w.scale)) + n * groups;
  }
  const uint16_t *x[MF][4];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[m][i] = p.x + (int64_t)min(m * 16 + 4 * i + (lane >> 4), p.M - 1) * p.ldx;

  struct Chunk {
    v4u c[NR], x[MF][4];
    uint32_t s[NR], z[NR];     // of the group that lane q stands for
  };
  // K values from chunk * 128 on; past the last one x counts as zero.
  auto load = [&](int64_t chunk, Chunk &t) {
    const int64_t k0 = chunk * 128;
    const int left = (int)min(p.K - k0, (int64_t)128);
    const int64_t kc = k0 / 2 + ((lane & 3) * 32 < left ? (lane & 3) * 16 : 0);
    const int64_t kx = k0 + (8 * r16 < left ? 8 * r16 : 0);
#pragma unroll
    for (int b = 0; b < NR; ++b) t.c[b] = *reinterpret_cast<const v4u *>(codes[b] + kc);
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) t.x[m][i] = *reinterpret_cast<const v4u_any *>(x[m][i] + kx);
    const int64_t g = min(chunk * GS + q * GS / 4, groups - 1);
#pragma unroll
    for (int b = 0; b < NR; ++b) {
      t.s[b] = scale[b][g];
      t.z[b] = zeros[b][g];
    }
  };
  Wave &mine = sm.wave[wave];
  v4f acc[NR][MF];
#pragma unroll
  for (int b = 0; b < NR; ++b)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[b][m] = v4f{0, 0, 0, 0};
  const v4u ones = {P::kOne, P::kOne, P::kOne, P::kOne};
  auto compute = [&](int64_t chunk, const Chunk &t) {
    const int left = (int)min(p.K - chunk * 128, (int64_t)128);
    // through the wave's own LDS, whose accesses stay in order: no barrier.  A row's
    // 16-byte pieces are kept at c ^ (row / 4 % 4) of its codes and c ^ row of its x.
#pragma unroll
    for (int b = 0; b < NR; ++b)
      *reinterpret_cast<v4u *>(mine.w[b] + (lane >> 2) * 64 +
                               (((lane & 3) ^ (lane >> 4)) << 4)) = t.c[b];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + (lane >> 4);
        *reinterpret_cast<v4u *>(mine.x[m] + row * 256 + ((r16 ^ row) << 4)) =
            8 * r16 < left ? pair_order(t.x[m][i]) : v4u{0, 0, 0, 0};
      }
    __builtin_amdgcn_wave_barrier();
    uint32_t c[NR][4];
#pragma unroll
    for (int b = 0; b < NR; ++b) {
      const v4u own = *reinterpret_cast<const v4u *>(mine.w[b] + r16 * 64 + ((q ^ (r16 >> 2)) << 4));
      // lane q's dword j <- lane j's dword q
      const auto e = __builtin_amdgcn_permlane32_swap(own[0], own[2], false, false);
      const auto f = __builtin_amdgcn_permlane32_swap(own[1], own[3], false, false);
      const auto g = __builtin_amdgcn_permlane16_swap(e[0], f[0], false, false);
      const auto h = __builtin_amdgcn_permlane16_swap(e[1], f[1], false, false);
      c[b][0] = g[0];
      c[b][1] = g[1];
      c[b][2] = h[0];
      c[b][3] = h[1];
    }
    // each group's scale and zero point to all four lanes of a row
    uint32_t sz[NR][GS];
#pragma unroll
    for (int b = 0; b < NR; ++b) {
      const uint32_t v = t.s[b] | ((has_zeros ? t.z[b] : 8u) << 16);
      if constexpr (GS == 1) {
        sz[b][0] = v;
      } else {
        const auto e = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        if constexpr (GS == 2) {
          sz[b][0] = e[0];
          sz[b][1] = e[1];
        } else {
          const auto f = __builtin_amdgcn_permlane16_swap(e[0], e[0], false, false);
          const auto g = __builtin_amdgcn_permlane16_swap(e[1], e[1], false, false);
          sz[b][0] = f[0];
          sz[b][1] = f[1];
          sz[b][2] = g[0];
          sz[b][3] = g[1];
        }
      }
    }
    constexpr int kEach = 4 / GS;
#pragma unroll
    for (int g = 0; g < GS; ++g) {
      v4f part[NR][MF], sum[MF];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = g * kEach + i;
        v4u w[NR];
#pragma unroll
        for (int b = 0; b < NR; ++b)
          w[b] = v4u{P::template codes<0>(c[b][j]), P::template codes<1>(c[b][j]),
                     P::template codes<2>(c[b][j]), P::template codes<3>(c[b][j])};
#pragma unroll
        for (int m = 0; m < MF; ++m) {
          const v4u xv = *reinterpret_cast<const v4u *>(mine.x[m] + r16 * 256 +
                                                        (((4 * j + q) ^ r16) << 4));
          const v4f zero = {0, 0, 0, 0};
          sum[m] = T::mfma(xv, ones, i ? sum[m] : zero);
#pragma unroll
          for (int b = 0; b < NR; ++b)
            part[b][m] = T::mfma(xv, w[b], i ? part[b][m] : zero);
        }
      }
#pragma unroll
      for (int b = 0; b < NR; ++b) {
        const float s = T::value(sz[b][g] & 0xffffu), bias = -16.0f - (float)(sz[b][g] >> 16);
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[b][m][r] = __builtin_fmaf(s, __builtin_fmaf(bias, sum[m][r], part[b][m][r]),
                                          acc[b][m][r]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
  // two chunks in turn, the next one's loads ahead of the products; past the last
  // one it is loaded again, and not used
  const int64_t chunks = (p.K + 127) / 128;
  Chunk t[2];
  if (wave < chunks) {
    load(wave, t[0]);
    for (int64_t i = wave; i < chunks; i += 2 * kWaves) {
      load(min(i + kWaves, chunks - 1), t[1]);
      compute(i, t[0]);
      if (i + kWaves >= chunks) break;
      load(min(i + 2 * kWaves, chunks - 1), t[0]);
      compute(i + kWaves, t[1]);
    }
  }
  __syncthreads();      // (the sums take the place of the other waves' codes and x)
#pragma unroll
  for (int b = 0; b < NR; ++b)
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) sm.red[wave][(b * MF + m) * 4 + r][lane] = acc[b][m][r];
  __syncthreads();
  // a lane of each output's place adds the waves' sums, in order
  for (int e = threadIdx.x; e < kOut * MF * 256; e += kWaves * 64) {
    const int l = e & 63, v = e >> 6;       // v = (block * MF + m) * 4 + r
    const int m = v / 4 % MF * 16 + 4 * (l >> 4) + v % 4;
    const int64_t n = n0 + v / (4 * MF) * 16 + (l & 15);
    const bool there = m < p.M && n < p.I;
    float y[PAIR ? 2 : 1];
#pragma unroll
    for (int h = 0; h < (PAIR ? 2 : 1); ++h) {
      y[h] = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) y[h] += sm.red[i][h * kOut * MF * 4 + v][l];
      y[h] = w4_finish<T>(p, there ? y[h] : 0.0f, m, n + h * p.I, lane);
    }
    if (!there) continue;
    float out = y[0];
    if constexpr (PAIR) out = act_any(p.act, y[0]) * y[1];
    p.out[m * p.I + n] = (uint16_t)T::bits(out);
  }
}

__global__ __launch_bounds__(256) void align_x_kernel(const uint16_t *in, int64_t ld, int64_t rows,
                                                      int64_t cols, uint16_t *out) {
  align_rows(in, ld, rows, cols, out, cols);
}

// ---------------------------------------------------------------------------
// Host side.

Weights weights(const W4Call &c) {
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

// Three rows and more go by matrix instructions (4 rows of 4096 -> 28672: 28 us, here 42).
constexpr int64_t kFewRows = 2;

template <typename T, bool PAIR, int MT>
hipError_t few(const W4Few &p, hipStream_t stream) {
  // Four rows of W a wave; whole K a wave where those alone give the chip enough waves,
  // else K shared by four.  One row, weights from HBM, us (whole K, shared): 4096 -> 8192
  // 9.6, 9.8; 4096 -> 14336 12, 14; 4096 -> 28672 18, 25; gated 4096 -> 8192 12.4, 15.6,
  // 4096 -> 14336 18, 25, 7168 -> 18432 39, 44.  Below the border 14336 -> 4096 17, 11.7;
  // gated 8192 -> 3584 13.6, 11.7.  The rule loses where many rows meet a long K (14336 ->
  // 8192 23, 19; 8192 -> 16384 24.5, 23.3, but two rows of it 28, 35).
  constexpr int R = PAIR ? 2 : 4;
  if (p.I / R >= 2048 || p.K <= 2048)
    w4_few_kernel<T, PAIR, R, MT, 1><<<dim3((unsigned)tiles(p.I, 4 * R)), 256, 0, stream>>>(p);
  else
    w4_few_kernel<T, PAIR, R, MT, 4><<<dim3((unsigned)tiles(p.I, R)), 256, 0, stream>>>(p);
  return hipGetLastError();
}
template <typename T, bool PAIR>
hipError_t few(const W4Call &c, int act, void *out, hipStream_t stream) {
  const W4Few p{weights(c), static_cast<const uint16_t *>(c.x), c.ldx, c.K,
                PAIR ? c.rows / 2 : c.rows, (int)c.M, act, static_cast<uint16_t *>(out)};
  return c.M == 1 ? few<T, PAIR, 1>(p, stream) : few<T, PAIR, 2>(p, stream);
}

// With more the kernel's registers run out.  Against the tiles, weights from HBM, us (here,
// tiles): 3 rows of 4096 -> 4096 9.9, 17.3, of 4096 -> 28672 28, 46; 32 rows 9.5, 19 and
// 45, 48; 48 rows 12, 21 and 58, 52, of 7168 -> 18432 63, 52, of 14336 -> 4096 32, 31.5,
// gated of 4096 -> 4096 15, 27, of 4096 -> 14336 58, 52.
constexpr int64_t kSlabRows = 48;

template <typename T, bool PAIR, int GS, int NR, int MF>
hipError_t slab(const W4Few &p, hipStream_t stream) {
  w4_slab_kernel<T, PAIR, GS, NR, MF>
      <<<dim3((unsigned)tiles(p.I, (PAIR ? NR / 2 : NR) * 16)), 512, 0, stream>>>(p);
  return hipGetLastError();
}
template <typename T, bool PAIR, int GS>
hipError_t slab(const W4Few &p, hipStream_t stream) {
  // Two blocks of rows read x half as often, where they still give every compute unit a
  // workgroup.  us (one block, two): 16 rows of 14336 -> 4096 17, 25, of 4096 -> 8192 10.4,
  // 9.7, of 4096 -> 28672 32, 30; 48 rows 32, 40; 21.5, 15; 80, 58.  The gated form takes
  // two at any size, gates and ups.
  constexpr int kNarrow = PAIR ? 2 : 1;
  const bool narrow = p.I < 32 * kCUs;
  if (p.M <= 16)
    return narrow ? slab<T, PAIR, GS, kNarrow, 1>(p, stream) : slab<T, PAIR, GS, 2, 1>(p, stream);
  if (p.M <= 32)
    return narrow ? slab<T, PAIR, GS, kNarrow, 2>(p, stream) : slab<T, PAIR, GS, 2, 2>(p, stream);
  return narrow ? slab<T, PAIR, GS, kNarrow, 3>(p, stream) : slab<T, PAIR, GS, 2, 3>(p, stream);
}
template <typename T, bool PAIR>
hipError_t slab(const W4Call &c, int act, void *out, hipStream_t stream) {
  const W4Few p{weights(c), static_cast<const uint16_t *>(c.x), c.ldx, c.K,
                PAIR ? c.rows / 2 : c.rows, (int)c.M, act, static_cast<uint16_t *>(out)};
  return c.group == 128 ? slab<T, PAIR, 1>(p, stream)
                        : c.group == 64 ? slab<T, PAIR, 2>(p, stream)
                                        : slab<T, PAIR, 4>(p, stream);
}

template <typename T, bool G32>
hipError_t linear(const W4Call &c, void *y, void *work, hipStream_t stream) {
  if (c.M <= kFewRows) return few<T, false>(c, 0, y, stream);
  if (c.M <= kSlabRows) return slab<T, false>(c, 0, y, stream);
  Space s{static_cast<uint8_t *>(work), 0};
  Operand a;
  if (hipError_t e = lay_x(c, a, s, stream)) return e;
  float *parts = reinterpret_cast<float *>(s.base + s.used);
  hipError_t e = hipSuccess;
  each_launch(cut_of(c.M, c.rows, c.K, true), c.rows,
              [&](int64_t first, int64_t n, const Plan &plan) {
    if (e != hipSuccess) return;
    W4<G32> w{weights(c)};
    w.codes += first * (c.K / 2);
    w.scale += first * (c.K / c.group);
    if (w.zeros) w.zeros += first * (c.K / c.group);
    Out p{c.M, n, static_cast<uint16_t *>(y) + first, c.rows, parts};
    with_shape(plan.shape, [&](auto shape) {
      using S = decltype(shape);
      const dim3 grid = p.tile<S>(plan, c.K);
      w4_product_kernel<T, S, G32><<<grid, S::kThreads, 0, stream>>>(a, w, p);
    });
    e = hipGetLastError();
    if (e == hipSuccess && p.ranges > 1) e = join<T>(p, stream);
  });
  return e;
}

template <typename T, bool G32>
hipError_t gated(const W4Call &c, int act, void *h, void *work, hipStream_t stream) {
  if (c.M <= kFewRows) return few<T, true>(c, act, h, stream);
  if (c.M <= kSlabRows) return slab<T, true>(c, act, h, stream);
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
  return launch_glu<T, false>(p, W4<G32>{weights(c)}, stream);
}

template <typename T>
hipError_t quant(const void *w, int64_t chunks, int group, void *codes, void *scale, void *zeros,
                 hipStream_t stream) {
  auto run = [&](auto size) {
    constexpr int G = size.value;
    const uint16_t *in = static_cast<const uint16_t *>(w);
    uint32_t *q = static_cast<uint32_t *>(codes);
    uint16_t *s = static_cast<uint16_t *>(scale);
    uint8_t *z = static_cast<uint8_t *>(zeros);
    const dim3 grid = groups(tiles(chunks, kAhead));
    if (z) w4_quant_kernel<T, G, true><<<grid, 256, 0, stream>>>(in, chunks, q, s, z);
    else w4_quant_kernel<T, G, false><<<grid, 256, 0, stream>>>(in, chunks, q, s, z);
  };
  if (group == 32) run(std::integral_constant<int, 32>{});
  else if (group == 64) run(std::integral_constant<int, 64>{});
  else run(std::integral_constant<int, 128>{});
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
  const dim3 grid = groups(tiles(chunks, kAhead));
  if (c.bf16) w4_dequant_kernel<Bf16><<<grid, 256, 0, stream>>>(weights(c), chunks, out);
  else w4_dequant_kernel<F16><<<grid, 256, 0, stream>>>(weights(c), chunks, out);
  return hipGetLastError();
}

// (the kernels of few rows launch 32 threads a row of W at most: 2^32 in all are too many)
bool w4_fits(int64_t M, int64_t rows) {
  return rows <= (int64_t(1) << 26) && grid_fits(M, rows);
}

size_t w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t ldx) {
  if (M <= kSlabRows) return 0;
  Space s{nullptr, 0};
  x_space(M, K, ldx, s);
  return s.used + part_bytes(M, N, K, true);
}

size_t w4_gated_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t ldx) {
  if (M <= kSlabRows) return 0;
  Space s{nullptr, 0};
  x_space(M, K, ldx, s);
  return s.used + part_bytes(M, 2 * I, K, true);
}

hipError_t launch_w4_linear(const W4Call &c, void *y, void *work, hipStream_t stream) {
  if (c.group == 32)
    return c.bf16 ? linear<Bf16, true>(c, y, work, stream) : linear<F16, true>(c, y, work, stream);
  return c.bf16 ? linear<Bf16, false>(c, y, work, stream) : linear<F16, false>(c, y, work, stream);
}

hipError_t launch_w4_gated(const W4Call &c, int act, void *h, void *work, hipStream_t stream) {
  if (c.group == 32)
    return c.bf16 ? gated<Bf16, true>(c, act, h, work, stream)
                  : gated<F16, true>(c, act, h, work, stream);
  return c.bf16 ? gated<Bf16, false>(c, act, h, work, stream)
                : gated<F16, false>(c, act, h, work, stream);
}

}  // namespace fp8blk
