// Tiled products of 16-bit floats for gfx950, shared by the gated projections
// (gated_kernels.hip) and the 4-bit weights' batches (w4_kernels.hip):
//   D[m, n] = sum_k A[m, k] B[n, k],   fp32 sums.
//
// An operand lies in memory with the summed index contiguous (kRows: a row of
// the operand per row of memory) or with it going down (kCols: a row of the
// operand is a column of memory), so that a layer's forward product, the
// gradient of its input and that of its weights all read their operands where
// they are.  Both kinds pass through LDS by direct-to-LDS loads, 64 of K a
// stage, two stages:
//   kRows  [rows][64 of K], 128 bytes a row, 16-byte chunk c of row r kept at
//          c ^ swz_f(r); a fragment is two ds_read_b128 a lane.
//   kCols  [64 of K][rows], 32-byte pairs p of K row k kept at p ^ col_f(k); a
//          fragment is four ds_read_b64_tr_b16 a lane, which transpose 4 x 16
//          values among 16 lanes.
// A lane (r = lane & 15, q = lane >> 4) of a matrix instruction holds 8 values of
// K of the operand's row r.  A stage is two instructions deep, and since both
// operands agree, instruction h takes K = 16 q + 8 h + 0..7 (or, where an
// instruction has to stay within 32 neighbouring K, 32 h + 8 q + 0..7).
#pragma once

#include "fp8blk_device.h"

namespace fp8blk {

typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

namespace t16 {

constexpr int kCUs = 256;
inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
inline int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// 16 and 8 bytes at any even address (gfx950's global loads and stores take those).
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned v2u_any __attribute__((ext_vector_type(2), aligned(2)));

// The 16-bit types: fp32 -> bits (round to nearest even), bits -> fp32, product.
struct Bf16 {
  static __device__ __forceinline__ uint32_t bits(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
  }
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
struct F16 {
  static __device__ __forceinline__ uint32_t bits(float f) {
    return __builtin_bit_cast(uint16_t, (_Float16)f);
  }
  static __device__ __forceinline__ float value(uint32_t b) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
  }
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return T::bits(lo) | (T::bits(hi) << 16);
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kK = 64;              // of K a stage
constexpr uint32_t kOut = 0xfffffff0u;   // an offset past every resource: reads zeros

// Loads through a buffer resource read zeros past its byte count.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, int64_t bytes) {
  const uint32_t n = bytes <= 0 ? 0u : (uint32_t)min(bytes, (int64_t)kOut);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)n, 0x00020000);
}
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t off, void *lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)lds, 16, (int)off, 0, 0, 0);
}

// As in the fp8 tiles: 16 lanes on one chunk of 16 consecutive rows meet no bank twice.
__device__ __forceinline__ int swz_f(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }
// 32 lanes of a transposing read take 32 bytes of K rows k, k + 1, k + 2, k + 3 and
// of those 16 further: eight different pairs of the 256 bytes that the banks span.
__device__ __forceinline__ int col_f(int k) { return (k & 3) | (((k >> 4) & 1) << 2); }

// A workgroup's tile: WM x WN waves of FM x FN fragments of 16 x 16.
template <int WM, int WN, int FM, int FN>
struct Shape {
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  static constexpr int TM = WM * FM * 16, TN = WN * FN * 16;
  static constexpr int kFM = FM, kFN = FN, kWM = WM, kWN = WN;
  struct Smem {
    uint8_t a[2][TM * kK * 2];
    uint8_t b[2][TN * kK * 2];
  };
};
// 256 x 256 on 8 waves (a wave 128 x 64), and 128 x 128 on 4 (64 x 64) for grids
// that the large tile would leave mostly idle.
using Large = Shape<2, 4, 8, 4>;
using Small = Shape<2, 2, 4, 4>;

// An operand in memory: `rows` of it along the output, `k` along the sum, both
// counted from p; `ld` elements from one row of memory to the next.  Rows of
// memory are 16-byte aligned and whole 16-byte chunks (ld and the contiguous
// extent are multiples of 8).
struct Operand {
  const uint16_t *p;
  int64_t ld;
  int64_t rows, k;
};

// The loads of one operand of ROWS rows into a stage, 1 KB each, shared among the
// waves.
enum Kind { kRows, kCols };
template <Kind KIND, int ROWS, int WAVES>
struct Loader {
  static constexpr int kLoads = ROWS / 8, kDma = (kLoads + WAVES - 1) / WAVES;
  uint32_t off[kDma];
  uint32_t chunk[kDma];   // kRows: the lane's chunk of the stage's K
  int wave;
  Operand o;

  // Whether load i of this wave exists (where the loads do not divide evenly).
  __device__ __forceinline__ bool has(int i) const {
    return kLoads % WAVES == 0 || kDma * wave + i < kLoads;
  }
  __device__ __forceinline__ void init(const Operand &op, int wave_, int lane) {
    o = op;
    wave = wave_;
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      if constexpr (KIND == kRows) {
        const int row = 8 * (kDma * wave + i) + (lane >> 3);
        chunk[i] = (lane & 7) ^ swz_f(row);
        off[i] = row < o.rows ? (uint32_t)(row * o.ld * 2) + chunk[i] * 16 : kOut;
      } else {
        constexpr int kChunks = ROWS / 8;     // 16-byte chunks of a K row
        const int at = (kDma * wave + i) * 64 + lane;
        const int k = at / kChunks, c = (at % kChunks) ^ (col_f(at / kChunks) << 1);
        chunk[i] = k;
        off[i] = c * 8 < o.rows ? (uint32_t)(k * o.ld * 2) + c * 16 : kOut;
      }
    }
  }
  // K values past the last one read as zeros, and so do rows past the last.
  __device__ __forceinline__ void issue(int step, uint8_t *stage) const {
    const int64_t k0 = (int64_t)step * kK;
    const int64_t left = o.k - k0;     // > 0
    if constexpr (KIND == kRows) {
      const __amdgpu_buffer_rsrc_t r = rsrc(o.p + k0, ((o.rows - 1) * o.ld + left) * 2);
      const uint32_t chunks = (uint32_t)min(left, (int64_t)kK) >> 3;
#pragma unroll
      for (int i = 0; i < kDma; ++i)
        if (has(i))
          dma16(r, chunk[i] < chunks ? off[i] : kOut, stage + (kDma * wave + i) * 1024);
    } else {
      const __amdgpu_buffer_rsrc_t r =
          rsrc(o.p + k0 * o.ld, ((min(left, (int64_t)kK) - 1) * o.ld + o.rows) * 2);
#pragma unroll
      for (int i = 0; i < kDma; ++i)
        if (has(i)) dma16(r, off[i], stage + (kDma * wave + i) * 1024);
    }
  }
};

struct Frag {
  v4u h[2];
};

// The fragment of 16 rows from `row0` of a stage of ROWS rows.
template <Kind KIND, int ROWS, bool HALVES = false>
__device__ __forceinline__ Frag read_frag(const uint8_t *stage, int row0, int lane) {
  Frag f;
  const int r = lane & 15, q = lane >> 4;
  if constexpr (KIND == kRows) {
    const int row = row0 + r, s = swz_f(row);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      f.h[h] = *reinterpret_cast<const v4u *>(
          stage + row * 128 + (((HALVES ? 4 * h + q : 2 * q + h) ^ s) << 4));
  } else {
    static_assert(!HALVES, "K rows are placed for the other order");
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 16 * q + 8 * h + 4 * j + (r >> 2);
        const uint8_t *at = stage + k * (ROWS * 2) + (((row0 >> 4) ^ col_f(k)) << 5) + (r & 3) * 8;
        const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)at);
        const v2u u = __builtin_bit_cast(v2u, v);
        f.h[h][2 * j] = u[0];
        f.h[h][2 * j + 1] = u[1];
      }
  }
  return f;
}

// The wave's sums acc[mi][ni][r] = D[16 mi + (lane & 15)][16 ni + 4 (lane >> 4) + r]
// of its FM x FN fragments, over `steps` stages from `step0`.
template <typename T, typename S, Kind KA, Kind KB, typename LoadA, typename LoadB>
__device__ __forceinline__ void multiply(const LoadA &la, const LoadB &lb, int step0, int steps,
                                         typename S::Smem &sm, v4f (&acc)[S::kFM][S::kFN]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int FM = S::kFM, FN = S::kFN;
  const int arow = wave / S::kWN * (FM * 16), brow = wave % S::kWN * (FN * 16);
#pragma unroll
  for (int mi = 0; mi < FM; ++mi)
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = v4f{0, 0, 0, 0};
  auto issue = [&](int s) {
    la.issue(step0 + s, sm.a[s & 1]);
    lb.issue(step0 + s, sm.b[s & 1]);
  };
  if (steps > 0) issue(0);
  for (int s = 0; s < steps; ++s) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (s + 1 < steps) issue(s + 1);
    const uint8_t *a = sm.a[s & 1], *b = sm.b[s & 1];
    Frag bf[FN];
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) bf[ni] = read_frag<KB, S::TN>(b, brow + ni * 16, lane);
#pragma unroll
    for (int mi = 0; mi < FM; ++mi) {
      const Frag af = read_frag<KA, S::TM>(a, arow + mi * 16, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = T::mfma(bf[ni].h[h], af.h[h], acc[mi][ni]);
    }
  }
}

// Tile (tm, tn) of workgroup `bid` of tiles_m x tiles_n: workgroups go round-robin
// over the 8 XCDs, so each XCD gets a consecutive run of tiles, in groups of 8
// tile rows whose neighbours share operands in its L2.
__device__ __forceinline__ void tile_of(int bid, int tiles_m, int tiles_n, int &tm, int &tn) {
  const int total = tiles_m * tiles_n, per = total >> 3, more = total & 7, x = bid & 7;
  const int at = x * per + min(x, more) + (bid >> 3);
  const int group = at / (8 * tiles_n), first = group * 8, in = at - group * 8 * tiles_n;
  const int height = min(tiles_m - first, 8);
  tm = first + in % height;
  tn = in / height;
}

// ---------------------------------------------------------------------------
// Stores and loads of four neighbouring columns, of which `left` > 0 exist.

template <typename T>
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4], int64_t left) {
  if (left >= 4) {
    const v2u u = {pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
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
// The same of fp32 sums, at any 4-byte address.
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void store4(float *p, v4f v, int64_t left) {
  if (left >= 4) {
    *reinterpret_cast<v4f_any *>(p) = v;
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < left) p[r] = v[r];
  }
}
__device__ __forceinline__ v4f load4(const float *p, int64_t left) {
  if (left >= 4) return *reinterpret_cast<const v4f_any *>(p);
  v4f v = {0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 3; ++r)
    if (r < left) v[r] = p[r];
  return v;
}
// Four fp32 values in 24 bits each (the top ones, to nearest even), 12 bytes.
typedef unsigned v3u __attribute__((ext_vector_type(3), aligned(4)));
__device__ __forceinline__ void store_24(uint8_t *p, const float (&v)[4]) {
  uint32_t b[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t u = __float_as_uint(v[r]);
    b[r] = (u + 0x7fu + ((u >> 8) & 1u)) >> 8;
  }
  *reinterpret_cast<v3u *>(p) =
      v3u{b[0] | (b[1] << 24), (b[1] >> 8) | (b[2] << 16), (b[2] >> 16) | (b[3] << 8)};
}
__device__ __forceinline__ void store_24_one(uint8_t *p, float v) {
  const uint32_t u = __float_as_uint(v), b = u + 0x7fu + ((u >> 8) & 1u);
  p[0] = (uint8_t)(b >> 8);
  p[1] = (uint8_t)(b >> 16);
  p[2] = (uint8_t)(b >> 24);
}
__device__ __forceinline__ void load_24(const uint8_t *p, float (&v)[4]) {
  const v3u d = *reinterpret_cast<const v3u *>(p);
  v[0] = __uint_as_float(d[0] << 8);
  v[1] = __uint_as_float(((d[0] >> 24) << 8) | (d[1] << 16));
  v[2] = __uint_as_float(((d[1] >> 16) << 8) | (d[2] << 24));
  v[3] = __uint_as_float(d[2] & 0xffffff00u);
}

// The sum of four columns' `ranges` parts, `step` apart, in order.
__device__ __forceinline__ v4f join4(const float *p, int ranges, int64_t step, int64_t left) {
  v4f v = load4(p, left);
  for (int s = 1; s < ranges; ++s) v += load4(p + s * step, left);
  return v;
}

// Element-wise kernels: as many workgroups as the work has, up to a grid that HIP
// runs whole, whose threads then take several items each.
constexpr int64_t kMostGroups = 1 << 20;
inline dim3 groups(int64_t items) {
  return dim3((unsigned)(tiles(items, 256) < kMostGroups ? tiles(items, 256) : kMostGroups));
}
__device__ __forceinline__ int64_t first_item() { return (int64_t)blockIdx.x * 256 + threadIdx.x; }
__device__ __forceinline__ int64_t all_threads() { return (int64_t)gridDim.x * 256; }

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

template <typename S>
int64_t grid_of(int64_t rows, int64_t cols) {
  return tiles(rows, S::TM) * tiles(cols, S::TN);
}

// How a product of rows x cols outputs over k is tiled.
struct Plan {
  bool large;
  int ranges;     // of K, a workgroup each
};
inline Plan plan_of(int64_t rows, int64_t cols, int64_t k) {
  // 256 x 256 tiles where they fill most of the chip
  if (grid_of<Large>(rows, cols) >= 192) return {true, 1};
  // ranges of K: enough workgroups for two a compute unit, at least 8 stages each
  const int64_t grid = grid_of<Small>(rows, cols), steps = tiles(k, kK);
  int64_t r = 2 * kCUs / grid;
  r = r < steps / 8 ? r : steps / 8;
  return {false, (int)(r > 1 ? r : 1)};
}

// A product's outputs, or its parts.
struct Out {
  int64_t rows, cols;
  uint16_t *out;          // [rows, cols]
  float *parts;           // [ranges][rows][cols], ranges > 1
  int steps, ranges;
  int tiles_m, tiles_n;

  __device__ __forceinline__ int first_step(int range) const {
    return (int)((int64_t)steps * range / ranges);
  }
};

template <typename T, typename S>
__device__ __forceinline__ void store_tile(const Out &p, const v4f (&acc)[S::kFM][S::kFN],
                                           int64_t m0, int64_t n0, int range) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  m0 += wave / S::kWN * (S::kFM * 16);
  n0 += wave % S::kWN * (S::kFN * 16);
#pragma unroll
  for (int mi = 0; mi < S::kFM; ++mi) {
    const int64_t m = m0 + mi * 16 + r16;
    if (m >= p.rows) continue;
#pragma unroll
    for (int ni = 0; ni < S::kFN; ++ni) {
      const int64_t n = n0 + ni * 16 + 4 * q;
      const int64_t left = p.cols - n;
      if (left <= 0) continue;
      if (p.ranges == 1) {
        const float v[4] = {acc[mi][ni][0], acc[mi][ni][1], acc[mi][ni][2], acc[mi][ni][3]};
        store4<T>(p.out + m * p.cols + n, v, left);
      } else {
        store4(p.parts + ((int64_t)range * p.rows + m) * p.cols + n, acc[mi][ni], left);
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void join_kernel(Out p) {
  const int64_t n = p.rows * p.cols;
  for (int64_t i = first_item() * 4; i < n; i += all_threads() * 4) {
    const v4f s = join4(p.parts + i, p.ranges, n, n - i);
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store4<T>(p.out + i, v, n - i);
  }
}

// The sums over a wave of N values (a power of two up to 64) of each lane, to out[N]:
// halves of the values are traded between halves of the lanes until a lane has one.
template <int N>
__device__ __forceinline__ void wave_sums(float (&v)[N], float *out, int lane) {
  static_assert(N <= 64 && (N & (N - 1)) == 0, "a power of two");
  int d = 32;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, d /= 2) {
    const bool upper = lane & d;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? v[i + n] : v[i], send = upper ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor(send, d);
    }
  }
  const int same = 2 * d;      // lanes that hold parts of one value
  for (; d >= 1; d /= 2) v[0] += __shfl_xor(v[0], d);
  if (lane % same == 0) out[lane / same] = v[0];
}

// Rows brought to a 16-byte pitch (whole chunks, zeros past a row's end).
__device__ __forceinline__ void align_rows(const uint16_t *in, int64_t ld, int64_t rows,
                                           int64_t cols, uint16_t *out, int64_t ldo) {
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

}  // namespace t16
}  // namespace fp8blk
