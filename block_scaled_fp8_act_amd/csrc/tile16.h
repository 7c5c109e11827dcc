// Tiled products of 16-bit floats for gfx950, shared by the gated projections
// (gated_kernels.hip) and the 4-bit weights' batches (w4_kernels.hip):
//   D[m, n] = sum_k A[m, k] B[n, k],   fp32 sums.
//
// An operand lies in memory with the summed index contiguous (kRows: a row of
// the operand per row of memory) or with it going down (kCols: a row of the
// operand is a column of memory), so that a layer's forward product, the
// gradient of its input and that of its weights all read their operands where
// they are.  Both kinds pass through LDS by direct-to-LDS loads, 64 of K a
// stage, two stages or four:
//   kRows  [rows][64 of K], 128 bytes a row, 16-byte chunk c of row r kept at
//          c ^ swz_f(r); a fragment is two ds_read_b128 a lane.
//   kCols  [64 of K][rows], 32-byte pairs p of K row k kept at p ^ col_f(k); a
//          fragment is four ds_read_b64_tr_b16 a lane, which transpose 4 x 16
//          values among 16 lanes.
// Lane l of a matrix instruction (16 x 16 outputs, 32 of K) holds 8 values of K of
// the operand's row l % 16, from K = 8 (l / 16) of the instruction's.  (On the 32 x 32
// form the same tiles measured 10-15 % slower.)
#pragma once

#include <type_traits>

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
constexpr int64_t tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// 16 and 8 bytes at any even address (gfx950's global loads and stores take those).
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned v2u_any __attribute__((ext_vector_type(2), aligned(2)));

// The 16-bit types: fp32 -> bits (round to nearest even), bits -> fp32, product.
struct Bf16 {
  typedef __bf16 Pair __attribute__((ext_vector_type(2)));
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
  typedef _Float16 Pair __attribute__((ext_vector_type(2)));
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
  typedef float v2f __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t,
                            __builtin_convertvector(v2f{lo, hi}, typename T::Pair));
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kK = 64;              // of K a stage
constexpr uint32_t kOut = 0xfffffff0u;   // an offset past every resource: reads zeros

__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return uniform((uint32_t)v) | ((uint64_t)uniform((uint32_t)(v >> 32)) << 32);
}

// A buffer resource of `bytes` bytes from `base` (both uniform); loads past them
// read zeros.
__device__ __forceinline__ v4u rsrc(uint64_t base, uint32_t bytes) {
  return v4u{(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, bytes, 0x00020000u};
}
// 16 bytes a lane from r at byte `off` to LDS at `lds` + 16 lane.  In assembly,
// because the compiler takes every later transposing read of LDS for one of what the
// load writes and waits for it there; the one wait that is needed stands before the
// barrier that opens the stage.  (It has no output register.)  The first of a stage's
// loads keeps the five wait states that a resource register written by a vector
// instruction (readfirstlane) needs before a load reads it.
template <bool FIRST>
__device__ __forceinline__ void dma16(v4u r, uint32_t off, const void *lds) {
  const uint32_t to = (uint32_t)(uintptr_t)(const lds_void *)lds;
  if constexpr (FIRST)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(off), "s"(r)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(off), "s"(r)
                 : "memory", "m0");
}

// Fragment reads of both sizes run at the LDS's full rate so: 247-251 bytes a clock
// and compute unit measured, half that with row & 7, or with the fp8 tiles' order,
// whose lanes take other chunks.
__device__ __forceinline__ int swz_f(int row) { return (row >> 1) & 7; }
// 32 lanes of a transposing read take 32 bytes of each of K rows k .. k + 3 and of
// those 8 further: eight different pairs of the 256 bytes that the banks span (of all
// there are, in operands of fewer than 128 rows).
template <int ROWS>
__device__ __forceinline__ int col_f(int k) {
  return (((k & 3) << 1) | ((k >> 3) & 1)) & (ROWS / 16 - 1);
}

// A workgroup's tile: WM x WN waves of FM x FN fragments of 16 x 16.  A lane holds
// four outputs of each fragment (i, j): of one row, neighbouring columns, or (ACROSS,
// where the products with the operands exchanged are formed) of one column,
// neighbouring rows; row(i, r, lane) and col(j, r, lane) are the r-th's place.
// STAGES (a power of two) are in LDS at a time.
template <int WM, int WN, int FM, int FN, int STAGES = 2, bool ACROSS = false>
struct Shape {
  static constexpr int kFM = FM, kFN = FN, kWM = WM, kWN = WN;
  static constexpr bool kAcross = ACROSS;
  static constexpr int kStages = STAGES;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  static constexpr int kWaveM = FM * 16, kWaveN = FN * 16;
  static constexpr int TM = WM * kWaveM, TN = WN * kWaveN;
  using Across = Shape<WM, WN, FM, FN, 2, true>;
  using Acc = v4f[FM][FN];
  static __device__ __forceinline__ int row(int i, int r, int lane) {
    return 16 * i + (ACROSS ? 4 * (lane >> 4) + r : lane & 15);
  }
  static __device__ __forceinline__ int col(int j, int r, int lane) {
    return 16 * j + (ACROSS ? lane & 15 : 4 * (lane >> 4) + r);
  }
  struct Smem {
    uint8_t a[STAGES][TM * kK * 2];
    uint8_t b[STAGES][TN * kK * 2];
  };
  static_assert(sizeof(Smem) >= TM * TN * 2, "room for the outputs on their way out");
};
// 256 x 256 on 8 waves (a wave 128 x 64); 128 x 128, 64 x 128 and 32 x 128 on 4 for
// grids that the larger tiles would leave mostly idle, and for few rows.  The flat ones
// keep four stages: their time is the loads' latency (64 rows of 4096 -> 14336: 69 ->
// 56 us; four stages of 128 x 128, one workgroup a compute unit, gained nothing).
using Large = Shape<2, 4, 8, 4>;
using Small = Shape<2, 2, 4, 4>;
using Low = Shape<2, 2, 2, 4, 4>;
using Flat = Shape<2, 2, 1, 4, 4>;

// An operand in memory: `rows` of it along the output, `k` along the sum, both
// counted from p; `ld` elements from one row of memory to the next.  Rows of
// memory are 16-byte aligned and whole 16-byte chunks (ld and the contiguous
// extent are multiples of 8, and at most 2^22).
struct Operand {
  const uint16_t *p;
  int64_t ld;
  int64_t rows, k;
};

// The loads of one operand's ROWS rows into a stage, 1 KB each, shared among the
// waves.  K values past the last one read as zeros, and so do rows past the last.
// Offsets and byte counts of a stage stay below 2^32: 256 rows of 2^22 elements.
enum Kind { kRows, kCols };
template <Kind KIND, int ROWS, int WAVES>
struct Loader {
  static constexpr int kDma = ROWS / 8 / WAVES;
  static_assert(kDma * 8 * WAVES == ROWS, "as many loads for each wave");
  uint32_t off[kDma];
  uint32_t chunk[kDma];   // kRows: the lane's chunk of the stage's K
  int wave;
  // uniform
  uint64_t base;
  uint32_t step_bytes;    // from one stage to the next
  uint32_t bytes;         // kRows: of the first stage's resource; kCols: of a row of memory
  uint32_t row_bytes;     // kCols: valid bytes of a row
  int k;                  // left at the first stage

  __device__ __forceinline__ void place(const Operand &o, int wave_) {
    wave = wave_;
    base = uniform((uint64_t)(uintptr_t)o.p);
    k = (int)uniform((uint32_t)o.k);
    const uint32_t ld = uniform((uint32_t)o.ld) * 2, rows = uniform((uint32_t)o.rows);
    step_bytes = KIND == kRows ? kK * 2 : ld * kK;
    bytes = KIND == kRows ? (rows - 1) * ld + k * 2 : ld;
    row_bytes = rows * 2;
  }
  __device__ __forceinline__ void init(const Operand &o, int wave_, int lane) {
    place(o, wave_);
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      if constexpr (KIND == kRows) {
        const int row = 8 * (kDma * wave + i) + (lane >> 3);
        chunk[i] = (lane & 7) ^ swz_f(row);
        off[i] = row < o.rows ? row * (uint32_t)o.ld * 2 + chunk[i] * 16 : kOut;
      } else {
        constexpr int kChunks = ROWS / 8;     // 16-byte chunks of a K row
        const int at = (kDma * wave + i) * 64 + lane;
        const int kr = at / kChunks, c = (at % kChunks) ^ (col_f<ROWS>(at / kChunks) << 1);
        off[i] = c * 8 < o.rows ? kr * (uint32_t)o.ld * 2 + c * 16 : kOut;
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    f(std::true_type{}, 0);
#pragma unroll
    for (int i = 1; i < kDma; ++i) f(std::false_type{}, i);
  }
  __device__ __forceinline__ void issue(int step, const uint8_t *stage) const {
    const uint64_t from = base + (uint64_t)(uint32_t)step * step_bytes;
    const int left = k - step * kK;     // > 0
    if constexpr (KIND == kRows) {
      const v4u r = rsrc(from, bytes - step * (kK * 2));
      const uint32_t chunks = min(left, kK) >> 3;
      each([&](auto first, int i) {
        dma16<first.value>(r, chunk[i] < chunks ? off[i] : kOut, stage + (kDma * wave + i) * 1024);
      });
    } else {
      const v4u r = rsrc(from, (min(left, kK) - 1) * bytes + row_bytes);
      each([&](auto first, int i) {
        dma16<first.value>(r, off[i], stage + (kDma * wave + i) * 1024);
      });
    }
  }
};

// A fragment of 16 rows over a stage: two instructions' operands.
struct Frag {
  v4u h[2];
};

// The fragment of the 16 rows from `row0` of a stage of ROWS rows.
template <Kind KIND, int ROWS>
__device__ __forceinline__ Frag read_frag(const uint8_t *stage, int row0, int lane) {
  Frag f;
  const int r = lane & 15, q = lane >> 4;
  if constexpr (KIND == kRows) {
    const int row = row0 + r, s = swz_f(row);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      f.h[h] = *reinterpret_cast<const v4u *>(stage + row * 128 + (((4 * h + q) ^ s) << 4));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 32 * h + 8 * q + 4 * j + (r >> 2);
        const uint8_t *at =
            stage + k * (ROWS * 2) + (((row0 >> 4) ^ col_f<ROWS>(k)) << 5) + (r & 3) * 8;
        const v2u u = __builtin_bit_cast(
            v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)at));
        f.h[h][2 * j] = u[0];
        f.h[h][2 * j + 1] = u[1];
      }
  }
  return f;
}

// The wave's sums over `steps` >= 1 stages from `step0`, as Shape places them.
//
// Step s reads stage s % N of the N in LDS.  Its barrier sits before the last row of
// fragments' matrix instructions: every wave has then read the stage, and the next one
// has landed in its own.  That stage's first fragments are read under the last row's
// instructions, and the loads of stage s + N go out into the one just read, N - 1 whole
// steps ahead, so the matrix cores do not wait at a step's start.  Past the last step
// the loads bring the last stage again, which nobody uses: a branch inside the
// unrolled instructions would cost more.
//
// Barrier for stages: at most LEFT of the wave's loads are still in flight, and its LDS
// reads are done.
template <int LEFT>
__device__ __forceinline__ void stage_barrier() {
  static_assert(LEFT <= 63, "the counter's range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(LEFT) : "memory");
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <typename T, typename S, Kind KA, Kind KB, typename LoadA, typename LoadB>
__device__ __forceinline__ void multiply(const LoadA &la, const LoadB &lb, int step0, int steps,
                                         typename S::Smem &sm, typename S::Acc &acc) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int FM = S::kFM, FN = S::kFN, N = S::kStages, kEach = LoadA::kDma + LoadB::kDma;
  const int arow = wave / S::kWN * S::kWaveM, brow = wave % S::kWN * S::kWaveN;
#pragma unroll
  for (int mi = 0; mi < FM; ++mi)
#pragma unroll
    for (int ni = 0; ni < FN; ++ni) acc[mi][ni] = v4f{0, 0, 0, 0};
  auto issue = [&](int s) {
    const int at = step0 + min(s, steps - 1);
    la.issue(at, sm.a[s % N]);
    lb.issue(at, sm.b[s % N]);
  };
  auto read_a = [&](int st, int mi) {
    return read_frag<KA, S::TM>(sm.a[st], arow + mi * 16, lane);
  };
  auto read_b = [&](int st, int ni) {
    return read_frag<KB, S::TN>(sm.b[st], brow + ni * 16, lane);
  };
#pragma unroll
  for (int s = 0; s < N; ++s) issue(s);
  stage_barrier<(N - 1) * kEach>();
  Frag bf[FN], af = read_a(0, 0);
#pragma unroll
  for (int ni = 0; ni < FN; ++ni) bf[ni] = read_b(0, ni);
  for (int s = 0; s < steps; ++s) {
    const int st = s % N, next = (s + 1) % N;
#pragma unroll
    for (int mi = 0; mi < FM; ++mi) {
      Frag an;
      if (mi < FM - 1) {
        an = read_a(st, mi + 1);
      } else {
        stage_barrier<(N - 2) * kEach>();
        issue(s + N);
        an = read_a(next, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int ni = 0; ni < FN; ++ni) {
          acc[mi][ni] = T::mfma(bf[ni].h[h], af.h[h], acc[mi][ni]);
          if (mi == FM - 1 && h == 1) {
            __builtin_amdgcn_sched_barrier(0);
            bf[ni] = read_b(next, ni);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      af = an;
    }
  }
  // LDS is left with no load into it in flight
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
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

// Whether a product's launches stay below 2^32 threads, whatever its plan: the
// smaller tiles (half the threads or less) are launched for grids of a few thousand,
// and for few rows, where they are at most twice the large ones.
inline bool grid_fits(int64_t rows, int64_t cols) {
  return tiles(rows, Large::TM) * tiles(cols, Large::TN) <
         (int64_t(1) << 32) / Large::kThreads;
}

// How a product of rows x cols outputs over k is tiled: the shape, and ranges of K
// on workgroups of their own (fp32 parts, added in order by a second kernel) where
// the tiles alone leave the chip idle.  The plan with the least time by a model
// whose constants are measurements: a workgroup alone on its compute unit takes
// `alone` us a stage, several take `shared` each (with 16-bit operands both follow the
// bytes that pass into LDS, 50 to 58 GB/s a compute unit; with 4-bit weights the
// decoding), `start` covers launch, first stage and epilogue, and the parts travel
// twice at 5 TB/s.
enum ShapeId { kLarge, kSmall, kLow, kFlat };
struct Plan {
  ShapeId shape;
  int ranges;
  double us;      // by the model
};
inline Plan plan_of(int64_t rows, int64_t cols, int64_t k, bool w4 = false) {
  struct Cost {
    int tm, tn;
    double alone, shared, start;
  };
  static constexpr Cost kCosts[2][4] = {{{Large::TM, Large::TN, 1.25, 1.45, 9.0},
                                         {Small::TM, Small::TN, 0.64, 0.55, 4.5},
                                         {Low::TM, Low::TN, 0.50, 0.42, 4.5},
                                         {Flat::TM, Flat::TN, 0.45, 0.36, 4.5}},
                                        {{Large::TM, Large::TN, 1.72, 2.00, 9.0},
                                         {Small::TM, Small::TN, 1.08, 0.78, 4.5},
                                         {Low::TM, Low::TN, 0.88, 0.56, 4.5},
                                         {Flat::TM, Flat::TN, 0.85, 0.52, 4.5}}};
  const int64_t steps = tiles(k, kK);
  Plan best{kSmall, 1, 1e30};
  for (int s = 0; s < 4; ++s) {
    const Cost &c = kCosts[w4][s];
    // a flatter tile only reads the columns' operand more often
    if ((s == kLow && rows > 2 * Low::TM) || (s == kFlat && rows > 2 * Flat::TM)) continue;
    const int64_t grid = tiles(rows, c.tm) * tiles(cols, c.tn);
    for (int r = 1; r <= 16 && (r == 1 || (steps / r >= 4 && grid * r <= 4 * kCUs)); ++r) {
      const int64_t n = tiles(grid * r, kCUs);
      const double per = n == 1 && (s != kLarge || grid * r <= kCUs / 2) ? c.alone : n * c.shared;
      double t = c.start + per * tiles(steps, r);
      if (r > 1) t += 4.0 + 8e-6 / 5 * r * (double)rows * (double)cols;
      if (t < best.us) best = {(ShapeId)s, r, t};
    }
  }
  return best;
}
// A product's columns in one or two launches: where large tiles leave the last round
// of compute units mostly idle, the columns of the whole rounds first, then the others
// by a plan of their own (2048 x 7168 -> 18432 with 4-bit weights, 2.25 rounds: 649 ->
// 565 us).
struct Cut {
  int64_t first;      // columns of the first launch (all of them: no second)
  Plan plan, rest;
};
inline Cut cut_of(int64_t rows, int64_t cols, int64_t k, bool w4 = false) {
  Cut cut{cols, plan_of(rows, cols, k, w4), {}};
  const int64_t tm = tiles(rows, Large::TM), tn = tiles(cols, Large::TN);
  const int64_t rounds = tm * tn / kCUs;
  if (rounds < 1 || tm * tn % kCUs == 0) return cut;
  const int64_t first = rounds * kCUs / tm * Large::TN;
  if (first < Large::TN || first >= cols) return cut;
  const Plan whole = plan_of(rows, first, k, w4), rest = plan_of(rows, cols - first, k, w4);
  // (by a clear margin: the model is no better than that)
  if (whole.shape != kLarge || whole.ranges > 1 || whole.us + rest.us > 0.95 * cut.plan.us)
    return cut;
  return {first, whole, rest};
}
inline size_t part_bytes(int64_t rows, int64_t cols, int64_t k, bool w4 = false) {
  const Cut c = cut_of(rows, cols, k, w4);
  const Plan &p = c.first < cols ? c.rest : c.plan;      // (the first of two has none)
  return p.ranges == 1 ? 0
                       : (size_t)p.ranges * rows * (c.first < cols ? cols - c.first : cols) *
                             sizeof(float);
}
// f(first column, columns, plan) for each launch.
template <typename F>
void each_launch(const Cut &c, int64_t cols, F f) {
  f((int64_t)0, c.first, c.plan);
  if (c.first < cols) f(c.first, cols - c.first, c.rest);
}
// f of the plan's shape (a value of its type).
template <typename F>
void with_shape(ShapeId s, F f) {
  switch (s) {
    case kLarge: f(Large{}); break;
    case kSmall: f(Small{}); break;
    case kLow: f(Low{}); break;
    case kFlat: f(Flat{}); break;
  }
}

// A product's outputs, or its parts.
struct Out {
  int64_t rows, cols;
  uint16_t *out;          // rows ld apart
  int64_t ld;
  float *parts;           // [ranges][rows][cols], ranges > 1
  int steps, ranges;
  int tiles_m, tiles_n;

  // Sets the plan's tiling over k; the grid.
  template <typename S>
  dim3 tile(const Plan &plan, int64_t k) {
    steps = (int)tiles(k, kK);
    ranges = plan.ranges;
    tiles_m = (int)tiles(rows, S::TM);
    tiles_n = (int)tiles(cols, S::TN);
    return dim3((unsigned)tiles_m * tiles_n * ranges);
  }
  __device__ __forceinline__ int first_step(int range) const {
    return (int)((int64_t)steps * range / ranges);
  }
};

// ---------------------------------------------------------------------------
// A tile's outputs of COLS columns pass through the stages' LDS, so that they leave
// in 16-byte pieces of whole rows: 16-byte chunk c of row r is kept at
// c ^ (r % (COLS / 8)), which spreads the writes of 16 rows over the banks.

template <int COLS>
__device__ __forceinline__ uint8_t *staged(uint8_t *lds, int row, int col) {
  return lds + row * (COLS * 2) + (((col >> 3) ^ (row & (COLS / 8 - 1))) << 4) + (col & 7) * 2;
}
// The four values of fragment (i, j) of the wave whose outputs begin at (row0, col0).
template <typename T, typename S, int COLS>
__device__ __forceinline__ void stage4(uint8_t *lds, int row0, int col0, int i, int j,
                                       const float (&v)[4], int lane) {
  if constexpr (S::kAcross) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<uint16_t *>(
          staged<COLS>(lds, row0 + S::row(i, r, lane), col0 + S::col(j, r, lane))) =
          (uint16_t)T::bits(v[r]);
  } else {
    *reinterpret_cast<v2u *>(
        staged<COLS>(lds, row0 + S::row(i, 0, lane), col0 + S::col(j, 0, lane))) =
        v2u{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
  }
}
// The staged tile's first `rows` x `cols` outputs to out, ld apart.
template <int THREADS, int ROWS, int COLS>
__device__ __forceinline__ void store_staged(uint8_t *lds, uint16_t *out, int64_t ld, int64_t rows,
                                             int64_t cols) {
  constexpr int kChunks = COLS / 8;
#pragma unroll 4
  for (int at = threadIdx.x; at < ROWS * kChunks; at += THREADS) {
    const int row = at / kChunks, col = at % kChunks * 8;
    if (row >= rows || col >= cols) continue;
    const v4u v = *reinterpret_cast<const v4u *>(staged<COLS>(lds, row, col));
    uint16_t *p = out + row * ld + col;
    if (col + 8 <= cols) {
      // read by another kernel, if at all: not kept beside the operands in L2
      __builtin_nontemporal_store(v, reinterpret_cast<v4u_any *>(p));
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (col + e < cols) p[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    }
  }
}
// A fragment's fp32 sums as parts, at p in rows ld apart; rows and cols are what is
// there from the fragment's first output on.
template <typename S>
__device__ __forceinline__ void store_part(float *p, int64_t ld, int64_t rows, int64_t cols, v4f v,
                                           int lane) {
  if constexpr (S::kAcross) {
    const int c = S::col(0, 0, lane);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (S::row(0, r, lane) < rows && c < cols) p[S::row(0, r, lane) * ld + c] = v[r];
  } else {
    const int m = S::row(0, 0, lane), c = S::col(0, 0, lane);
    if (m < rows && c < cols) store4(p + m * ld + c, v, cols - c);
  }
}

// A wave's place among its workgroup's.
template <typename S>
__device__ __forceinline__ int wave_row() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / S::kWN * S::kWaveM;
}
template <typename S>
__device__ __forceinline__ int wave_col() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % S::kWN * S::kWaveN;
}

template <typename T, typename S>
__device__ __forceinline__ void store_tile(const Out &p, const typename S::Acc &acc, int64_t m0,
                                           int64_t n0, int range, uint8_t *lds) {
  const int lane = threadIdx.x & 63, row = wave_row<S>(), col = wave_col<S>();
  if (p.ranges > 1) {
    float *parts = p.parts + ((int64_t)range * p.rows + m0 + row) * p.cols + n0 + col;
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
      for (int j = 0; j < S::kFN; ++j)
        store_part<S>(parts + i * 16 * p.cols + j * 16, p.cols, p.rows - m0 - row - i * 16,
                      p.cols - n0 - col - j * 16, acc[i][j], lane);
    return;
  }
  __syncthreads();      // every wave is past its last stage
#pragma unroll
  for (int i = 0; i < S::kFM; ++i)
#pragma unroll
    for (int j = 0; j < S::kFN; ++j) {
      const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      stage4<T, S, S::TN>(lds, row, col, i, j, v, lane);
    }
  __syncthreads();
  store_staged<S::kThreads, S::TM, S::TN>(lds, p.out + m0 * p.ld + n0, p.ld, p.rows - m0,
                                          p.cols - n0);
}

template <typename T>
__global__ __launch_bounds__(256) void join_kernel(Out p) {
  const int64_t quads = (p.cols + 3) / 4, step = p.rows * p.cols;
  for (int64_t at = first_item(); at < p.rows * quads; at += all_threads()) {
    const int64_t m = at / quads, n = (at - m * quads) * 4, left = p.cols - n;
    const v4f s = join4(p.parts + m * p.cols + n, p.ranges, step, left);
    const float v[4] = {s[0], s[1], s[2], s[3]};
    store4<T>(p.out + m * p.ld + n, v, left);
  }
}
template <typename T>
hipError_t join(const Out &p, hipStream_t stream) {
  join_kernel<T><<<groups(p.rows * tiles(p.cols, 4)), 256, 0, stream>>>(p);
  return hipGetLastError();
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
