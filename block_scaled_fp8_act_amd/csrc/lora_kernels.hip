// Low-rank adapters of many requests beside a shared projection, for gfx950:
//   out[t] = base[t] + scale[g] * (x[t] A[g]^T) B[g]^T,   g = the row's adapter,
// with x [T, K], A [L, r, K], B [L, N, r], base and out [T, N] in bf16.
//
// Two launches: lora_shrink_kernel forms h = x A^T (fp32, in the workspace,
// K split over workgroups where there are few rows) and lora_expand_kernel
// adds the parts of h, multiplies by scale and B^T and adds the base in its
// epilogue.  Rows of one adapter are taken 16 at a time, the width of a
// matrix instruction, so every adapter in the batch is read once per 16 of
// its rows and rows of different adapters never share a product.
//
// Bound: HBM traffic (x once, base and out once, the adapters in use once);
// at ranks up to 256 the products are far below the matrix cores' rate.
#include "fp8blk_device.h"
#include "fp8blk_launch.h"

namespace fp8blk {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));

namespace {

constexpr int kTileRows = 16;
constexpr int kLoraThreads = 256;
constexpr int kLoraWaves = kLoraThreads / 64;
// Batches up to a wave's width find their rows from the adapter numbers
// directly; larger ones through a listing by adapter (order, offsets).
constexpr int kDirectRows = 64;
constexpr int kWideRows = 64;
// Batches from here on take the kernels with 64-row tiles (measured at 515
// rows of 32 adapters, 7168 -> 1536, r = 64: 26 us against 36 us).
constexpr int64_t kWideBatch = 512;
constexpr int kMaxSplit = 16;

struct LoraArgs {
  const uint16_t *x, *a, *b, *base;
  int64_t ldx, ldb, ldo;
  const int32_t *ids;             // [T], T <= kDirectRows
  const int32_t *order, *offsets; // [T], [L + 1], T > kDirectRows
  const float *scale;             // [L] or NULL (1)
  float *h;                       // [S][T][r]
  uint16_t *hs;                   // [T][r / 8][16]: h split, for large batches
  uint16_t *out;
  int64_t T, K, N;
  int L, r, S, copy_bare;         // copy_bare: rows without adapter: out = base
};

// The rows of one tile: all of adapter g (g == L: rows without adapter).
struct Tile {
  int g;
  int row;   // of slot lane & 15, or -1
};

// Tile `index` of a batch of at most 64 rows: every lane holds a row's
// adapter, equal ones find each other by ballots over the number's bits, and
// adapters come in the order of their first rows.
__device__ __forceinline__ bool find_tile_direct(const LoraArgs &p, int index, Tile *t) {
  const int lane = threadIdx.x & 63;
  const int id = lane < p.T ? p.ids[lane] : -1;
  const bool worn = (unsigned)id < (unsigned)p.L;
  const int key = worn ? id : p.L;
  const bool in = lane < p.T && (worn || p.copy_bare);
  uint64_t same = __builtin_amdgcn_ballot_w64(in);
  const int bits = 32 - __builtin_clz(p.L);
  for (int b = 0; b < bits; ++b) {
    const bool set = (key >> b) & 1;
    const uint64_t m = __builtin_amdgcn_ballot_w64(set);
    same &= set ? m : ~m;
  }
  const uint64_t below = (1ull << lane) - 1;
  const int leader = in ? __builtin_ctzll(same) : 0;
  const int rank = __popcll(same & below);
  const int more = (__popcll(same) - 1) / kTileRows;   // tiles past the first: 0..3
  const bool leads = in && lane == leader;
  const uint64_t first = (1ull << leader) - 1;
  const int before = __popcll(__builtin_amdgcn_ballot_w64(leads) & first) +
                     __popcll(__builtin_amdgcn_ballot_w64(leads && (more & 1)) & first) +
                     2 * __popcll(__builtin_amdgcn_ballot_w64(leads && (more & 2)) & first);
  const bool mine = in && before + rank / kTileRows == index;
  const uint64_t members = __builtin_amdgcn_ballot_w64(mine);
  if (members == 0) return false;
  t->g = __builtin_amdgcn_readlane(key, (int)__builtin_ctzll(members));
  // each member sends its row to lane (slot); the others to a lane not read
  const int sent = __builtin_amdgcn_ds_permute((mine ? rank % kTileRows : 63) * 4,
                                               mine ? lane + 1 : 0);
  t->row = __builtin_amdgcn_ds_bpermute((lane & 15) * 4, sent) - 1;
  return true;
}

// Tile `index` (ROWS rows) of a batch listed by adapter: a wave adds up the
// adapters' tile counts, 64 adapters at a time, until it reaches the tile.
struct ListedTile {
  int g, start, rows;   // order[start .. start + rows)
};

template <int ROWS>
__device__ __forceinline__ bool find_listed(const LoraArgs &p, int index, ListedTile *t) {
  const int lane = threadIdx.x & 63;
  const int T = (int)p.T;
  int done = 0;
  for (int g0 = 0; g0 <= p.L; g0 += 64) {
    const int g = g0 + lane;
    int lo = g <= p.L ? p.offsets[g] : T;
    int hi = g < p.L ? p.offsets[g + 1] : T;
    lo = min(max(lo, 0), T);
    hi = min(max(hi, lo), T);
    int n = (hi - lo + ROWS - 1) / ROWS;
    if (g > p.L || (g == p.L && !p.copy_bare)) n = 0;
    int scan = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(scan, d);
      scan += lane >= d ? o : 0;
    }
    const uint64_t past = __builtin_amdgcn_ballot_w64(done + scan > index);
    if (past) {
      const int l = (int)__builtin_ctzll(past);
      t->g = g0 + l;
      t->start = __builtin_amdgcn_readlane(lo, l) +
                 (index - done - __builtin_amdgcn_readlane(scan - n, l)) * ROWS;
      t->rows = min(ROWS, __builtin_amdgcn_readlane(hi, l) - t->start);
      return true;
    }
    done += __builtin_amdgcn_readlane(scan, 63);
  }
  return false;
}

__device__ __forceinline__ bool find_tile_listed(const LoraArgs &p, int index, Tile *t) {
  ListedTile lt;
  if (!find_listed<kTileRows>(p, index, &lt)) return false;
  t->g = lt.g;
  const int slot = threadIdx.x & 15;
  const int row = slot < lt.rows ? p.order[lt.start + slot] : -1;
  t->row = row < p.T ? row : -1;
  return true;
}

template <bool DIRECT>
__device__ __forceinline__ bool find_tile(const LoraArgs &p, int index, Tile *t) {
  if constexpr (DIRECT) return find_tile_direct(p, index, t);
  else return find_tile_listed(p, index, t);
}

__device__ __forceinline__ v8bf as_bf(const uint4 &v) { return __builtin_bit_cast(v8bf, v); }

struct __attribute__((packed, aligned(2))) U128 {
  uint32_t v[4];
};

__device__ __forceinline__ uint4 load16(const uint16_t *p) {
  const U128 w = *reinterpret_cast<const U128 *>(p);
  return make_uint4(w.v[0], w.v[1], w.v[2], w.v[3]);
}

__device__ __forceinline__ v4u load16v(const uint16_t *p) {
  typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));
  return *reinterpret_cast<const v4u_any *>(p);
}

__device__ __forceinline__ uint16_t bf_bits(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

}  // namespace

// h[s][row][:] = the part of x[row] A[g]^T over K range s.  The instruction's
// rows are ranks (A) and its columns the tile's rows (x): both operands are
// 16-byte loads along K, and a lane ends with four consecutive ranks of one
// row.  The four waves take every fourth 32 of K and add up through LDS.
template <bool DIRECT, int NT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink_kernel(LoraArgs p) {
  __shared__ float part[kLoraWaves][NT * 256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = blockIdx.x % p.S;
  Tile t;
  if (!find_tile<DIRECT>(p, blockIdx.x / p.S, &t) || t.g >= p.L) return;
  const int KB = (int)(p.K / kBlock);
  const int kb0 = (int)((int64_t)KB * s / p.S), kb1 = (int)((int64_t)KB * (s + 1) / p.S);
  const int koff = wave * 32 + (lane >> 4) * 8;
  // slots past the tile's rows repeat slot 0's row (a tile has one at least)
  const int row0 = __builtin_amdgcn_readlane(t.row, 0);
  const int row = max(t.row >= 0 ? t.row : row0, 0);
  const uint16_t *xr = p.x + (int64_t)row * p.ldx + koff;
  const uint16_t *ar[NT];
#pragma unroll
  for (int f = 0; f < NT; ++f)
    ar[f] = p.a + ((int64_t)t.g * p.r + min(f * 16 + (lane & 15), p.r - 1)) * p.K + koff;
  v4f acc[NT];
#pragma unroll
  for (int f = 0; f < NT; ++f) acc[f] = v4f{0, 0, 0, 0};
#pragma unroll 4
  for (int kb = kb0; kb < kb1; ++kb) {
    const int64_t k = (int64_t)kb * kBlock;
    const v8bf xv = as_bf(load16(xr + k));
#pragma unroll
    for (int f = 0; f < NT; ++f) {
      if (f * 16 < p.r)
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            as_bf(*reinterpret_cast<const uint4 *>(ar[f] + k)), xv, acc[f], 0, 0, 0);
    }
  }
#pragma unroll
  for (int f = 0; f < NT; ++f)
    *reinterpret_cast<v4f *>(&part[wave][f * 256 + lane * 4]) = acc[f];
  __syncthreads();
  // wave w stores fragments w, w + 4, ...
  for (int f = wave; f * 16 < p.r; f += kLoraWaves) {
    v4f v = v4f{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kLoraWaves; ++w)
      v += *reinterpret_cast<const v4f *>(&part[w][f * 256 + lane * 4]);
    const int rank = f * 16 + (lane >> 4) * 4;
    if (t.row >= 0 && rank < p.r)
      *reinterpret_cast<v4f *>(p.h + ((int64_t)s * p.T + t.row) * p.r + rank) = v;
  }
}

// out = base + (scale * sum of h's parts) B^T for 16 rows and 64 columns a
// wave.  h enters the product as the sum of two bf16 values, its upper half
// and the rest, which keeps 16 significant bits of it (2^-17, far below the
// output's rounding): the instruction's 32 values of K hold 16 ranks' upper
// halves and rests, against B's ranks twice.  The instruction's rows are
// columns of the output, mapped so that a lane ends with two runs of 8
// consecutive columns of one row, the four lanes of a row side by side: base
// and out move 16 bytes a lane, 64 together.
template <bool DIRECT, int NS>
__global__ __launch_bounds__(kLoraThreads) void lora_expand_kernel(LoraArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blocks_n = (int)((p.N + 255) / 256);
  Tile t;
  if (!find_tile<DIRECT>(p, blockIdx.x / blocks_n, &t)) return;
  const int64_t n0 = (int64_t)(blockIdx.x % blocks_n) * 256 + wave * 64;
  if (n0 >= p.N) return;
  v4f acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f] = v4f{0, 0, 0, 0};
  if (t.g < p.L) {
    const float scale = p.scale ? p.scale[t.g] : 1.0f;
    const bool rest = (lane >> 4) & 1;
    const int m = lane & 15;
    const uint16_t *br[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int64_t n = n0 + (f >> 1) * 32 + (m >> 2) * 8 + (f & 1) * 4 + (m & 3);
      br[f] = p.b + ((int64_t)t.g * p.N + (n < p.N ? n : p.N - 1)) * p.r;
    }
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      if (st * 16 >= p.r) break;
      const int rank = st * 16 + (lane >> 5) * 8;
      const bool in = rank < p.r;
      float h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = 0.0f;
      if (in && t.row >= 0) {
        const float *hp = p.h + (int64_t)t.row * p.r + rank;
        for (int s = 0; s < p.S; ++s) {
          const float4 u = *reinterpret_cast<const float4 *>(hp + (int64_t)s * p.T * p.r);
          const float4 v = *reinterpret_cast<const float4 *>(hp + (int64_t)s * p.T * p.r + 4);
          h[0] += u.x; h[1] += u.y; h[2] += u.z; h[3] += u.w;
          h[4] += v.x; h[5] += v.y; h[6] += v.z; h[7] += v.w;
        }
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t q[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float v = h[2 * i + j] * scale;
          const float hi = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
          // an infinite or NaN value has no rest
          const float lo = __builtin_isfinite(v) ? v - hi : 0.0f;
          q[j] = rest ? bf_bits(lo) : __float_as_uint(hi) >> 16;
        }
        w[i] = q[0] | (q[1] << 16);
      }
      const v8bf hv = as_bf(make_uint4(w[0], w[1], w[2], w[3]));
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const uint4 bv = in ? *reinterpret_cast<const uint4 *>(br[f] + rank) : make_uint4(0, 0, 0, 0);
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(bv), hv, acc[f], 0, 0, 0);
      }
    }
  }
  if (t.row < 0) return;
  uint16_t *o = p.out + (int64_t)t.row * p.ldo;
  const uint16_t *bs = p.base ? p.base + (int64_t)t.row * p.ldb : nullptr;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t c = n0 + q * 32 + (lane >> 4) * 8;
    if (c + 8 <= p.N) {
      float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (bs) unpack8(load16(bs + c), f);
      U128 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4f v = acc[q * 2 + i / 2];
        w.v[i] = (uint32_t)bf_bits(f[2 * i] + v[(2 * i) & 3]) |
                 ((uint32_t)bf_bits(f[2 * i + 1] + v[(2 * i + 1) & 3]) << 16);
      }
      *reinterpret_cast<U128 *>(o + c) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < p.N) {
          const float f = bs ? bf16_lo(bs[c + i]) : 0.0f;
          o[c + i] = bf_bits(f + acc[q * 2 + i / 4][i & 3]);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Large batches: tiles of 64 rows.
//
// A and B come from L2 once per 64 rows instead of 16 and x, base and out stay
// the only HBM traffic of weight.  h is kept as the second product takes it:
// per row and 8 ranks, the 8 upper halves and then the 8 rests in bf16.


// v as upper half and rest (an infinite or NaN value has no rest).
__device__ __forceinline__ void split_bf16(float v, uint16_t *hi, uint16_t *lo) {
  const uint32_t u = __float_as_uint(v) & 0xffff0000u;
  *hi = (uint16_t)(u >> 16);
  *lo = bf_bits(__builtin_isfinite(v) ? v - __uint_as_float(u) : 0.0f);
}

// Chunk swizzle of 128-byte LDS rows: 16-byte chunk c of row r is kept at
// c ^ f(r), so that 16 lanes reading one chunk of 16 consecutive rows meet no
// bank twice.
__device__ __forceinline__ int swz_f(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }

// Barrier for data passed through LDS alone: unlike __syncthreads() it leaves
// global loads and stores in flight (waiting for them cost 5 us a stage).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A lane of a matrix instruction holds 16 bytes of one row, and neighbouring
// lanes hold different rows: loaded that way every lane's 16 bytes are a
// request of their own (measured: 60 us at 8192 x 7168, r = 32, and no
// faster with more loads in flight).  So both operands pass through LDS: 64
// of K a stage, loaded with eight neighbouring lanes on a row's 128 bytes, two
// stages ahead in registers.  WR x WN waves take MR row fragments and NR rank
// fragments each.  h goes out in fp32 parts, one per K range.
template <int WR, int WN, int MR, int NR>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink_wide_kernel(LoraArgs p) {
  static_assert(WR * WN == kLoraWaves && WR * MR * 16 == kWideRows, "tile shape");
  constexpr int RA = WN * NR * 16;                      // rows of A in a stage
  constexpr int NX = kWideRows * 8 / kLoraThreads;      // 16-byte chunks a thread loads
  constexpr int NA = (RA * 8 + kLoraThreads - 1) / kLoraThreads;
  constexpr int kStage = (kWideRows + RA) * 128;
  __shared__ __align__(16) uint8_t lds[2][kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int s = blockIdx.x % p.S;
  ListedTile t;
  if (!find_listed<kWideRows>(p, blockIdx.x / p.S, &t) || t.g >= p.L) return;
  const int KB = (int)(p.K / 64);
  const int kb0 = (int)((int64_t)KB * s / p.S), n = (int)((int64_t)KB * (s + 1) / p.S) - kb0;
  auto row_of = [&](int slot) {   // slots past the tile's rows repeat its last row
    const int row = p.order[t.start + min(slot, t.rows - 1)];
    return min(max(row, 0), (int)p.T - 1);
  };
  const uint16_t *xp[NX], *ap[NA];
  int xo[NX], ao[NA];
#pragma unroll
  for (int j = 0; j < NX; ++j) {
    const int c = tid + j * kLoraThreads, r = c >> 3;
    xp[j] = p.x + (int64_t)row_of(r) * p.ldx + (int64_t)kb0 * 64 + (c & 7) * 8;
    xo[j] = r * 128 + (((c & 7) ^ swz_f(r)) << 4);
  }
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    const int c = min(tid + j * kLoraThreads, RA * 8 - 1), r = c >> 3;
    ap[j] = p.a + ((int64_t)t.g * p.r + min(r, p.r - 1)) * p.K + (int64_t)kb0 * 64 + (c & 7) * 8;
    ao[j] = (kWideRows + r) * 128 + (((c & 7) ^ swz_f(r)) << 4);
  }
  v4f acc[MR][NR];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int f = 0; f < NR; ++f) acc[i][f] = v4f{0, 0, 0, 0};
  const int first = (wave / WN) * MR * 16;   // the wave's first row in the tile
  const int rank0 = (wave % WN) * NR * 16;
  const bool idle = first >= t.rows || rank0 >= p.r;

  // loads past the last stage repeat it (and are not used)
  auto load = [&](v4u (&x)[NX], v4u (&w)[NA], int i) {
    const int64_t k = (int64_t)min(i, n - 1) * 64;
#pragma unroll
    for (int j = 0; j < NX; ++j) x[j] = load16v(xp[j] + k);
#pragma unroll
    for (int j = 0; j < NA; ++j) w[j] = *reinterpret_cast<const v4u *>(ap[j] + k);
  };
  auto stage = [&](v4u (&x)[NX], v4u (&w)[NA], int b, int i) {
#pragma unroll
    for (int j = 0; j < NX; ++j) *reinterpret_cast<v4u *>(&lds[b][xo[j]]) = x[j];
#pragma unroll
    for (int j = 0; j < NA; ++j)
      if (RA * 8 % kLoraThreads == 0 || tid + j * kLoraThreads < RA * 8)
        *reinterpret_cast<v4u *>(&lds[b][ao[j]]) = w[j];
    load(x, w, i + 2);
    lds_barrier();
    if (idle) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int chunk = h * 4 + (lane >> 4);
      v8bf xv[MR], av[NR];
#pragma unroll
      for (int q = 0; q < MR; ++q) {
        const int r = first + q * 16 + (lane & 15);
        xv[q] = as_bf(*reinterpret_cast<const uint4 *>(&lds[b][r * 128 + ((chunk ^ swz_f(r)) << 4)]));
      }
#pragma unroll
      for (int f = 0; f < NR; ++f) {
        const int r = rank0 + f * 16 + (lane & 15);
        av[f] = as_bf(*reinterpret_cast<const uint4 *>(
            &lds[b][(kWideRows + r) * 128 + ((chunk ^ swz_f(r)) << 4)]));
      }
#pragma unroll
      for (int q = 0; q < MR; ++q)
#pragma unroll
        for (int f = 0; f < NR; ++f)
          acc[q][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[f], xv[q], acc[q][f], 0, 0, 0);
    }
  };
  v4u x0[NX], x1[NX], a0[NA], a1[NA];
  load(x0, a0, 0);
  load(x1, a1, 1);
  int i = 0;
  for (; i + 1 < n; i += 2) {
    stage(x0, a0, 0, i);
    stage(x1, a1, 1, i + 1);
  }
  if (i < n) stage(x0, a0, 0, i);
  if (idle) return;
#pragma unroll
  for (int q = 0; q < MR; ++q) {
    const int slot = first + q * 16 + (lane & 15);
    if (slot >= t.rows) continue;
    float *hp = p.h + ((int64_t)s * p.T + row_of(slot)) * p.r;
#pragma unroll
    for (int f = 0; f < NR; ++f) {
      const int rank = rank0 + f * 16 + (lane >> 4) * 4;
      if (rank < p.r) *reinterpret_cast<v4f *>(hp + rank) = acc[q][f];
    }
  }
}

// Adds the parts of h, scales and splits them: a thread takes 8 ranks of a row.
__global__ __launch_bounds__(kLoraThreads) void lora_join_kernel(LoraArgs p) {
  const int chunks = p.r / 8;
  const int64_t i = (int64_t)blockIdx.x * kLoraThreads + threadIdx.x;
  if (i >= p.T * chunks) return;
  const int64_t row = i / chunks;
  const int g = p.ids[row];
  if ((unsigned)g >= (unsigned)p.L) return;
  const float *hp = p.h + row * p.r + (i - row * chunks) * 8;
  float h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int s = 0; s < p.S; ++s) {
    const float4 u = *reinterpret_cast<const float4 *>(hp + (int64_t)s * p.T * p.r);
    const float4 v = *reinterpret_cast<const float4 *>(hp + (int64_t)s * p.T * p.r + 4);
    h[0] += u.x; h[1] += u.y; h[2] += u.z; h[3] += u.w;
    h[4] += v.x; h[5] += v.y; h[6] += v.z; h[7] += v.w;
  }
  const float scale = p.scale ? p.scale[g] : 1.0f;
  uint16_t q[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) split_bf16(h[j] * scale, &q[j], &q[8 + j]);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = q[2 * j] | ((uint32_t)q[2 * j + 1] << 16);
  uint4 *o = reinterpret_cast<uint4 *>(p.hs + i * 16);
  o[0] = make_uint4(w[0], w[1], w[2], w[3]);
  o[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// out for a tile's 64 rows and CT runs of 128 columns, 16 rows a wave.  Rows
// of the instruction are rows of the batch, its columns columns of out, and a
// lane's eight fragments are eight consecutive columns: base and out move as
// 256 contiguous bytes of a row per 16 lanes.  h stays in registers for all CT
// runs; B's run goes through LDS (it is contiguous in memory, but a fragment
// takes a row per lane), loaded one run ahead in registers, with an odd number
// of 16-byte chunks between rows so that 16 rows' chunks meet no bank twice.
constexpr int kExpandCols = 128;

template <int NS>
__global__ __launch_bounds__(kLoraThreads) void lora_expand_wide_kernel(LoraArgs p, int ct) {
  extern __shared__ __align__(16) uint8_t lds[];   // B's run: [fragment][16] rows
  __shared__ int rows[kWideRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int runs = (int)((p.N + kExpandCols - 1) / kExpandCols);
  const int groups = (runs + ct - 1) / ct;
  ListedTile t;
  if (!find_listed<kWideRows>(p, blockIdx.x / groups, &t)) return;
  const int run0 = (int)(blockIdx.x % groups) * ct;
  const int run1 = min(run0 + ct, runs);
  if (tid < kWideRows)
    rows[tid] = min(max(p.order[t.start + min(tid, t.rows - 1)], 0), (int)p.T - 1);
  lds_barrier();
  const bool worn = t.g < p.L;
  const int i16 = lane & 15, g16 = lane >> 4;
  const int chunks = p.r / 8;                 // 16-byte chunks of a row of B
  const int pitch = (chunks | 1) * 16;
  constexpr int NB = NS;                      // chunks a thread loads: 128 * r / 8 / 256 = r / 16
  v4u hv[NS], br[NB];
  const uint16_t *hr = p.hs + (int64_t)rows[wave * 16 + i16] * p.r * 2 + g16 * 8;
  if (worn) {
#pragma unroll
    for (int st = 0; st < NS; ++st)
      hv[st] = st * 16 + (g16 >> 1) * 8 < p.r ? *reinterpret_cast<const v4u *>(hr + st * 32)
                                              : v4u{0, 0, 0, 0};
  }
  // chunk c of a run is row (column of out) c / chunks of it; column n = 8 i + f
  // is row i of fragment f.  Columns past N repeat the last one.
  int bn[NB], bc[NB], bo[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int c = min(tid + j * kLoraThreads, kExpandCols * chunks - 1);
    bn[j] = c / chunks;
    bc[j] = c - bn[j] * chunks;
    bo[j] = ((bn[j] & 7) * 16 + (bn[j] >> 3)) * pitch + bc[j] * 16;
  }
  const uint16_t *bg = p.b + (worn ? (int64_t)t.g * p.N * p.r : 0);
  auto load_b = [&](int run) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t col = min((int64_t)run * kExpandCols + bn[j], p.N - 1);
      br[j] = *reinterpret_cast<const v4u *>(bg + col * p.r + bc[j] * 8);
    }
  };
  if (worn) load_b(run0);
  for (int run = run0; run < run1; ++run) {
    const int64_t c0 = (int64_t)run * kExpandCols + i16 * 8;
    uint4 bs[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      bs[q] = p.base && c0 + 8 <= p.N
                  ? load16(p.base + (int64_t)rows[wave * 16 + g16 * 4 + q] * p.ldb + c0)
                  : make_uint4(0, 0, 0, 0);
    v4f acc[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[f] = v4f{0, 0, 0, 0};
    if (worn) {
      lds_barrier();   // the run before has been read
#pragma unroll
      for (int j = 0; j < NB; ++j) *reinterpret_cast<v4u *>(&lds[bo[j]]) = br[j];
      lds_barrier();
      load_b(min(run + 1, run1 - 1));
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        // past the rank h is zero, and B's last chunk stands in
        const int chunk = min(st * 2 + (g16 >> 1), chunks - 1);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          const v8bf bv = *reinterpret_cast<const v8bf *>(&lds[(f * 16 + i16) * pitch + chunk * 16]);
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, hv[st]), bv,
                                                           acc[f], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int slot = wave * 16 + g16 * 4 + q;
      if (slot >= t.rows) continue;
      uint16_t *o = p.out + (int64_t)rows[slot] * p.ldo;
      if (c0 + 8 <= p.N) {
        float f[8];
        unpack8(bs[q], f);
        U128 w;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w.v[j] = (uint32_t)bf_bits(f[2 * j] + acc[2 * j][q]) |
                   ((uint32_t)bf_bits(f[2 * j + 1] + acc[2 * j + 1][q]) << 16);
        *reinterpret_cast<U128 *>(o + c0) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c0 + j < p.N) {
            const float f = p.base ? bf16_lo(p.base[(int64_t)rows[slot] * p.ldb + c0 + j]) : 0.0f;
            o[c0 + j] = bf_bits(f + acc[j][q]);
          }
      }
    }
  }
}

namespace {
bool is_wide(int64_t T) { return T >= kWideBatch; }

// Tiles a batch can have at most: full ones, and one more per adapter (and
// for the rows without one).
int64_t max_tiles(int64_t T, int L) {
  if (T <= kDirectRows) return T;
  const int64_t groups = (int64_t)L + 1 < T ? (int64_t)L + 1 : T;
  return T / (is_wide(T) ? kWideRows : kTileRows) + groups;
}

// K ranges: enough workgroups to fill the chip, at least 256 of K each.
int split_of(int64_t T, int64_t K, int L) {
  const int64_t tiles = max_tiles(T, L);
  int64_t s = 512 / tiles;
  if (s > K / 256) s = K / 256;
  if (s > kMaxSplit) s = kMaxSplit;
  return s < 1 ? 1 : (int)s;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t K, int32_t r, int32_t L, bool listed) {
  size_t n = align256(sizeof(float) * (size_t)split_of(T, K, L) * T * r);
  if (is_wide(T)) n += align256(sizeof(float) * (size_t)T * r);
  if (T > kDirectRows && !listed)
    n += align256(sizeof(int32_t) * (size_t)T) * 2 + align256(sizeof(int32_t) * ((size_t)L + 1)) +
         group_workspace_bytes(T, L);
  return n;
}

hipError_t launch_lora_add(const void *base, int64_t ldb, const void *x, int64_t ldx,
                           const void *a, const void *b, const int32_t *ids, const float *scale,
                           const int32_t *order, const int32_t *offsets, int64_t T, int64_t K,
                           int64_t N, int32_t r, int32_t L, void *out, int64_t ldo, void *work,
                           hipStream_t stream) {
  LoraArgs p{};
  p.x = static_cast<const uint16_t *>(x);
  p.a = static_cast<const uint16_t *>(a);
  p.b = static_cast<const uint16_t *>(b);
  p.base = static_cast<const uint16_t *>(base);
  p.out = static_cast<uint16_t *>(out);
  p.ldx = ldx;
  p.ldb = ldb;
  p.ldo = ldo;
  p.ids = ids;
  p.order = order;
  p.offsets = offsets;
  p.scale = scale;
  p.T = T;
  p.K = K;
  p.N = N;
  p.L = L;
  p.r = r;
  p.S = split_of(T, K, L);
  p.copy_bare = base != out;
  char *w = static_cast<char *>(work);
  p.h = reinterpret_cast<float *>(w);
  w += align256(sizeof(float) * (size_t)p.S * T * r);
  const bool direct = T <= kDirectRows;
  const bool wide = is_wide(T);
  if (wide) {
    p.hs = reinterpret_cast<uint16_t *>(w);
    w += align256(sizeof(float) * (size_t)T * r);
  }
  if (!direct && !order) {
    int32_t *ord = reinterpret_cast<int32_t *>(w);
    w += align256(sizeof(int32_t) * (size_t)T);
    int32_t *pos = reinterpret_cast<int32_t *>(w);
    w += align256(sizeof(int32_t) * (size_t)T);
    int32_t *off = reinterpret_cast<int32_t *>(w);
    w += align256(sizeof(int32_t) * ((size_t)L + 1));
    if (hipError_t e = launch_group_rows(ids, T, L, ord, pos, off, w, stream)) return e;
    p.order = ord;
    p.offsets = off;
  }
  const int64_t tiles = max_tiles(T, L);
  const unsigned gs = (unsigned)(tiles * p.S);
  const unsigned ge = (unsigned)(tiles * ((N + 255) / 256));
  if (wide) {
    if (r <= 16) lora_shrink_wide_kernel<4, 1, 1, 1><<<gs, kLoraThreads, 0, stream>>>(p);
    else if (r <= 32) lora_shrink_wide_kernel<4, 1, 1, 2><<<gs, kLoraThreads, 0, stream>>>(p);
    else if (r <= 64) lora_shrink_wide_kernel<2, 2, 2, 2><<<gs, kLoraThreads, 0, stream>>>(p);
    else if (r <= 128) lora_shrink_wide_kernel<2, 2, 2, 4><<<gs, kLoraThreads, 0, stream>>>(p);
    else lora_shrink_wide_kernel<2, 2, 2, 8><<<gs, kLoraThreads, 0, stream>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
    const int64_t pieces = T * (r / 8);
    lora_join_kernel<<<(unsigned)((pieces + kLoraThreads - 1) / kLoraThreads), kLoraThreads, 0,
                       stream>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
    // several runs of columns a workgroup where that leaves enough of them
    const int64_t runs = (N + kExpandCols - 1) / kExpandCols;
    int64_t ct = tiles * runs / 1024;
    ct = ct < 1 ? 1 : ct > 4 ? 4 : ct;
    const unsigned gw = (unsigned)(tiles * ((runs + ct - 1) / ct));
    const size_t lds = (size_t)kExpandCols * ((r / 8) | 1) * 16;
    if (r <= 16) lora_expand_wide_kernel<1><<<gw, kLoraThreads, lds, stream>>>(p, (int)ct);
    else if (r <= 32) lora_expand_wide_kernel<2><<<gw, kLoraThreads, lds, stream>>>(p, (int)ct);
    else if (r <= 64) lora_expand_wide_kernel<4><<<gw, kLoraThreads, lds, stream>>>(p, (int)ct);
    else if (r <= 128) lora_expand_wide_kernel<8><<<gw, kLoraThreads, lds, stream>>>(p, (int)ct);
    else lora_expand_wide_kernel<16><<<gw, kLoraThreads, lds, stream>>>(p, (int)ct);
    return hipGetLastError();
  }
#define FP8BLK_LORA(D, NT)                                                  \
  do {                                                                      \
    lora_shrink_kernel<D, NT><<<gs, kLoraThreads, 0, stream>>>(p);          \
    if (hipError_t e = hipGetLastError()) return e;                         \
    lora_expand_kernel<D, NT><<<ge, kLoraThreads, 0, stream>>>(p);          \
    return hipGetLastError();                                               \
  } while (0)
#define FP8BLK_LORA_RANK(D)                                                 \
  do {                                                                      \
    if (r <= 16) FP8BLK_LORA(D, 1);                                         \
    if (r <= 32) FP8BLK_LORA(D, 2);                                         \
    if (r <= 64) FP8BLK_LORA(D, 4);                                         \
    if (r <= 128) FP8BLK_LORA(D, 8);                                        \
    FP8BLK_LORA(D, 16);                                                     \
  } while (0)
  if (direct) FP8BLK_LORA_RANK(true);
  FP8BLK_LORA_RANK(false);
#undef FP8BLK_LORA_RANK
#undef FP8BLK_LORA
}

}  // namespace fp8blk
