// Low-rank adapters of many requests beside a shared projection, for gfx950:
//   out[t] = base[t] + scale[g] * (x[t] A[g]^T) B[g]^T,   g = the row's adapter,
// with x [T, K], A [L, r, K], B [L, N, r], base and out [T, N] in bf16.
//
// The shrink kernels form h = x A^T in fp32 parts (K split over workgroups so
// that they fill the chip), the expand kernels multiply it by B^T and add the
// base in their epilogue.  Rows of one adapter are taken in tiles, so every
// adapter in the batch is read from HBM once and rows of different adapters
// never share a product.  Up to 64 rows the tiles are 16 rows and two launches
// do all; beyond, the rows are listed by adapter (group_rows, unless the caller
// did) in tiles of 64, and a small launch between the two adds h's parts up and
// lays them out for the matrix instruction.
//
// Bound: HBM traffic (x once, base and out once, the adapters in use once); at
// ranks up to 256 the products are far below the matrix cores' rate.  Measured,
// bf16 from HBM, all launches: 16 rows of 16 adapters, 4096 x 4096, r = 16: 10 us
// (latency; 4.6 MB); 515 rows of 32, 7168 -> 1536, r = 64: 23 us; 8192 rows of
// 8, 7168 -> 18432, r = 32: 152 us (723 MB, 4.8 TB/s); 4099 rows of 5, 14336 ->
// 4096, r = 128: 75 us (208 MB, 2.8 TB/s: the shrink kernel's passes through LDS
// and its products, which grow with the rank, take longer there than x's way
// from HBM).
//
// Grids and K ranges are sized for a tile of every adapter of the pool, used or
// not: the host does not know which are.  A pool far larger than the batch's use
// of it so leaves compute units without work in the shrink kernel (one adapter in
// use of 256, 515 rows: 9 workgroups).
#include "fp8blk_device.h"
#include "fp8blk_launch.h"

namespace fp8blk {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));

namespace {

constexpr int kTileRows = 16;   // rows of a matrix instruction, and of a small batch's tile
constexpr int kLoraThreads = 256;
constexpr int kLoraWaves = kLoraThreads / 64;
// Batches up to a wave's width find their rows from the adapter numbers
// directly and take tiles of 16 rows; larger ones go by a listing by adapter
// (order, offsets) in tiles of 64.  16-row tiles past 64 rows measured 16-20 %
// faster with an adapter per row (128 rows, 4096 x 4096, r = 16: 22 against
// 27 us) and up to three times slower with shared ones (400 rows of 20
// adapters, r = 128: 90 against 31 us).
constexpr int kDirectRows = 64;
constexpr int kWideRows = 64;
constexpr int kMaxSplit = 8;
// h in the second product: the parts of a value's split, the ranks of an
// instruction, and the bytes of 16 rows of both.
constexpr int kParts = 3;
constexpr int kStepRanks = 32;
constexpr int kStepBytes = kParts * 64 * 16;
__host__ __device__ constexpr int rank_steps(int r) { return (r + kStepRanks - 1) / kStepRanks; }
// Bytes between B's rows in LDS: whole steps, of which the chunks past the rank
// hold zeros (h is zero there, and another rank's infinity must not meet it),
// and an odd number of 16-byte chunks, so that 16 rows' chunks spread over the
// banks.
__host__ __device__ constexpr int rank_pitch(int r) { return rank_steps(r) * kStepRanks * 2 + 16; }

struct LoraArgs {
  const uint16_t *x, *a, *b, *base;
  int64_t ldx, ldb, ldo;
  const int32_t *ids;             // [T], T <= kDirectRows
  const int32_t *order, *offsets; // [T], [L + 1], T > kDirectRows
  const float *scale;             // [L] or NULL (1)
  float *h;                       // [S][T][r]
  // larger batches: per tile of 64 rows its adapter, its rows and its h, split
  int32_t *tile_adapter, *tile_rows;
  uint16_t *hs;
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

// 16 bytes at any even address (gfx950's global loads and stores take those);
// the _once forms for what is read or written once: non-temporal, so that it
// does not displace the adapters in L2.
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ v4u load16v(const uint16_t *p) {
  return *reinterpret_cast<const v4u_any *>(p);
}
__device__ __forceinline__ v4u load16_once(const uint16_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const v4u_any *>(p));
}
__device__ __forceinline__ void store16_once(uint16_t *p, v4u v) {
  __builtin_nontemporal_store(v, reinterpret_cast<v4u_any *>(p));
}

__device__ __forceinline__ uint16_t bf_bits(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

}  // namespace

// ---------------------------------------------------------------------------
// Batches of up to 64 rows: a tile of up to 16 rows of one adapter.
//
// Latency counts here: the adapters in use are read once each from HBM (A and B
// of 16 requests at 4096 x 4096, r = 16: 4 MB, 1 us) by as many workgroups as
// the chip holds, in two launches.
//
// Chunk swizzle of 128-byte LDS rows: 16-byte chunk c of row r is kept at
// c ^ f(r), so that 16 lanes reading one chunk of 16 consecutive rows meet no
// bank twice.
__device__ __forceinline__ int swz_f(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }

// Barrier for data passed through LDS alone: unlike __syncthreads() it leaves
// global loads and stores in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// h[s][row][16 ranks] = the part of x[row] A[g]^T over K range s, a workgroup
// per tile, 16 ranks and range.  A lane of a matrix instruction holds 16 bytes
// of one row and its neighbours other rows; loaded that way every lane's 16
// bytes are a request of their own.  So 256 of K at a time pass through LDS,
// loaded with 32 neighbouring lanes on a row's 512 bytes, one stage ahead in
// registers; each wave takes 64 of them, and the waves' sums add up through
// LDS.  The instruction's rows are ranks, its columns the tile's rows.
constexpr int kSmallK = 256;

__global__ __launch_bounds__(kLoraThreads) void lora_shrink_kernel(LoraArgs p) {
  __shared__ __align__(16) uint8_t lds[kLoraWaves][32 * 128];   // 64 of K: 16 rows of x, 16 of A
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pieces = (p.r + 15) / 16;
  const int s = blockIdx.x % p.S, piece = blockIdx.x / p.S % pieces;
  Tile t;
  if (!find_tile_direct(p, blockIdx.x / p.S / pieces, &t) || t.g >= p.L) return;
  const int KB = (int)((p.K + kSmallK - 1) / kSmallK);
  const int kb0 = (int)((int64_t)KB * s / p.S), kb1 = (int)((int64_t)KB * (s + 1) / p.S);
  // thread: rows tid / 32 and + 8 of x (slots past the tile's rows repeat the
  // first) and of A, 16 bytes at column tid % 32 * 8 of the stage
  const int r8 = tid >> 5, c32 = tid & 31;
  const int row0 = __builtin_amdgcn_readlane(t.row, 0);
  const uint16_t *src[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int slot = r8 + 8 * j;
    const int row = __shfl(t.row, slot);
    src[j] = p.x + (int64_t)(row >= 0 ? row : row0) * p.ldx + c32 * 8;
    src[2 + j] = p.a + ((int64_t)t.g * p.r + min(piece * 16 + slot, p.r - 1)) * p.K + c32 * 8;
  }
  const int dst = r8 * 128 + (((c32 & 7) ^ swz_f(r8)) << 4);   // (row + 8: the same swizzle)
  v4u v[4];
  auto load = [&](int kb) {
    const int64_t k = (int64_t)min(kb, kb1 - 1) * kSmallK;
    const bool in = k + c32 * 8 < p.K;    // (K is a multiple of 128)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = in ? load16v(src[j] + k) : v4u{0, 0, 0, 0};
  };
  v4f acc = v4f{0, 0, 0, 0};
  load(kb0);
  for (int kb = kb0; kb < kb1; ++kb) {
    lds_barrier();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<v4u *>(&lds[c32 >> 3][dst + j * 8 * 128]) = v[j];
    load(kb + 1);
    lds_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane & 15;
      const int at = r * 128 + ((((lane >> 4) * 2 + h) ^ swz_f(r)) << 4);
      const v8bf xv = *reinterpret_cast<const v8bf *>(&lds[wave][at]);
      const v8bf av = *reinterpret_cast<const v8bf *>(&lds[wave][16 * 128 + at]);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, xv, acc, 0, 0, 0);
    }
  }
  lds_barrier();
  v4f *part = reinterpret_cast<v4f *>(&lds[0][0]);
  part[wave * 64 + lane] = acc;
  lds_barrier();
  if (wave) return;
#pragma unroll
  for (int w = 1; w < kLoraWaves; ++w) acc += part[w * 64 + lane];
  const int rank = piece * 16 + (lane >> 4) * 4;
  if (t.row >= 0 && rank < p.r)
    *reinterpret_cast<v4f *>(p.h + ((int64_t)s * p.T + t.row) * p.r + rank) = acc;
}

// v as the sum of three bf16 values, its 24 bits eight at a time: each is cut, not
// rounded, so each rest is exact, has at most 16, then 8 bits, and v's sign.  A
// part that would be zero takes half of the one before (exact too), so that
// every part of a v other than zero times an infinite entry of B is the
// infinity that v times it is, and no 0 times infinity makes a NaN.  An
// infinite or NaN v is in every part.
__device__ __forceinline__ float cut_bf16(float v) {
  return __uint_as_float(__float_as_uint(v) & 0xffff0000u);
}
__device__ __forceinline__ void split_bf16(float v, uint32_t *part) {
  static_assert(kParts == 3, "the parts below");
  float a = cut_bf16(v);
  float b = cut_bf16(v - a);
  float c = v - a - b;
  if (v == a || !__builtin_isfinite(v)) a = b = v * 0.5f;
  if (c == 0.0f || !__builtin_isfinite(v)) b = c = b * 0.5f;
  part[0] = __float_as_uint(a) >> 16;
  part[1] = __float_as_uint(b) >> 16;
  part[2] = __float_as_uint(c) >> 16;
}

// scale times the sum of h's parts at hp (8 ranks), split.
__device__ __forceinline__ void join_parts(const LoraArgs &p, const float *hp, float scale,
                                           v4u (&out)[kParts]) {
  const int64_t step = p.T * p.r;
  v4f h[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
  for (int s0 = 0; s0 < p.S; s0 += 8) {   // 8 parts' loads in flight
    v4f u[8][2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float *q = hp + min(s0 + j, p.S - 1) * step;
      u[j][0] = *reinterpret_cast<const v4f *>(q);
      u[j][1] = *reinterpret_cast<const v4f *>(q + 4);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s0 + j < p.S) {
        h[0] += u[j][0];
        h[1] += u[j][1];
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t a[kParts], b[kParts];
    split_bf16(h[j >> 1][2 * j & 3] * scale, a);
    split_bf16(h[j >> 1][(2 * j & 3) + 1] * scale, b);
#pragma unroll
    for (int i = 0; i < kParts; ++i) out[i][j] = a[i] | (b[i] << 16);
  }
}

// Zeros in the chunks past the rank of B's ROWS rows in LDS.
template <int ROWS>
__device__ __forceinline__ void clear_past_rank(uint8_t *lb, int r, int tid) {
  const int chunks = r / 8, pad = rank_steps(r) * (kStepRanks / 8) - chunks;   // 0..3
  for (int c = tid / ROWS; c < pad; c += kLoraThreads / ROWS)
    *reinterpret_cast<v4u *>(&lb[tid % ROWS * rank_pitch(r) + (chunks + c) * 16]) =
        v4u{0, 0, 0, 0};
}

// out = base + (scale * sum of h's parts) B^T for a tile and 128 columns, 32 a
// wave.  h enters the product as the sum of three bf16 values, which holds every
// bit of its fp32 value: three instructions of 32 ranks on one fragment of B.
// B's 128 rows are contiguous in memory and pass through LDS for the reason
// above.
constexpr int kSmallCols = 128;

__global__ __launch_bounds__(kLoraThreads) void lora_expand_kernel(LoraArgs p) {
  extern __shared__ __align__(16) uint8_t lds[];   // h's fragments, then B's rows [2][64]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int runs = (int)((p.N + kSmallCols - 1) / kSmallCols);
  Tile t;
  if (!find_tile_direct(p, blockIdx.x / runs, &t)) return;
  const int64_t n0 = (int64_t)(blockIdx.x % runs) * kSmallCols;
  const int i16 = lane & 15, g16 = lane >> 4;
  const int chunks = p.r / 8, steps = rank_steps(p.r);
  const int pitch = rank_pitch(p.r);
  uint8_t *lb = lds + steps * kStepBytes;
  const bool worn = t.g < p.L;
  // base of rows g16 * 4 + q, columns c0 and c0 + 1
  const int64_t c0 = n0 + wave * 32 + i16 * 2;
  int row[4];
  uint32_t bs[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    row[q] = __shfl(t.row, g16 * 4 + q);
    bs[q] = 0;
    if (p.base && row[q] >= 0) {
      const uint16_t *b = p.base + (int64_t)row[q] * p.ldb + c0;
      if (c0 < p.N) bs[q] = b[0];
      if (c0 + 1 < p.N) bs[q] |= (uint32_t)b[1] << 16;
    }
  }
  v4f acc[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
  if (worn) {
    // B's chunks: the first kHeld of a thread are loaded here and written below,
    // so that their latency and that of h's parts pass together
    constexpr int kHeld = 4;
    const uint16_t *bg = p.b + (int64_t)t.g * p.N * p.r;
    v4u held[kHeld];
    int at[kHeld];
    auto fetch = [&](int c, v4u *v, int *dst) {
      const int n = c / chunks, ch = c - n * chunks;
      // column n = 2 i + f is row i of half f; columns past N repeat the last one
      *dst = ((n & 1) * 64 + (n >> 1)) * pitch + ch * 16;
      *v = *reinterpret_cast<const v4u *>(bg + min(n0 + n, p.N - 1) * p.r + ch * 8);
    };
    const int total = kSmallCols * chunks;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) fetch(min(tid + j * kLoraThreads, total - 1), &held[j], &at[j]);
    clear_past_rank<kSmallCols>(lb, p.r, tid);
    const float scale = p.scale ? p.scale[t.g] : 1.0f;
    for (int c = tid; c < 64 * steps; c += kLoraThreads) {
      const int slot = c & 15, ch = c >> 4;
      const int r = __shfl(t.row, slot);            // (lane & 15 == slot)
      v4u h[kParts] = {};
      if (r >= 0 && ch < chunks) join_parts(p, p.h + (int64_t)r * p.r + ch * 8, scale, h);
      v4u *f = reinterpret_cast<v4u *>(lds + (ch >> 2) * kStepBytes) + (ch & 3) * 16 + slot;
#pragma unroll
      for (int i = 0; i < kParts; ++i) f[i * 64] = h[i];
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) *reinterpret_cast<v4u *>(&lb[at[j]]) = held[j];
    for (int c = tid + kHeld * kLoraThreads; c < total; c += kHeld * kLoraThreads) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        fetch(min(c + j * kLoraThreads, total - 1), &held[j], &at[j]);
#pragma unroll
      for (int j = 0; j < kHeld; ++j) *reinterpret_cast<v4u *>(&lb[at[j]]) = held[j];
    }
    lds_barrier();
#pragma unroll 2
    for (int st = 0; st < steps; ++st) {
      const int chunk = st * 4 + g16;
      const v8bf *hv = reinterpret_cast<const v8bf *>(lds + st * kStepBytes) + lane;
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const v8bf bv = *reinterpret_cast<const v8bf *>(
            &lb[(f * 64 + wave * 16 + i16) * pitch + chunk * 16]);
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hv[i * 64], bv, acc[f], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (row[q] < 0) continue;
    uint16_t *o = p.out + (int64_t)row[q] * p.ldo + c0;
    if (c0 < p.N) o[0] = bf_bits(bf16_lo(bs[q]) + acc[0][q]);
    if (c0 + 1 < p.N) o[1] = bf_bits(bf16_hi(bs[q]) + acc[1][q]);
  }
}

// ---------------------------------------------------------------------------
// Larger batches: tiles of 64 rows.
//
// A and B come from L2 once per 64 or 128 rows, and x, base and out stay the
// only HBM traffic of weight.
//
// A lane of a matrix instruction holds 16 bytes of one row, and neighbouring
// lanes hold different rows: loaded that way every lane's 16 bytes are a
// request of their own (measured: 60 us at 8192 x 7168, r = 32, and no
// faster with more loads in flight).  So both operands pass through LDS: 64
// of K a stage, loaded with eight neighbouring lanes on a row's 128 bytes, two
// stages ahead in registers.  WR x WN waves take MR row fragments and NR rank
// fragments each.  h goes out in fp32 parts, one per K range.  Now 25 us there
// (4.7 TB/s of x), and 35 us at 4099 x 14336, r = 128 (3.3 TB/s), where the time
// grows with the rank and not with what is in flight: four stages ahead, more
// workgroups, or a K range per XCD measured no faster.  No unit is full there (LDS
// 32 %, matrix cores 25 % of the busy cycles, no bank conflicts): a workgroup's
// writes, barrier, reads and products follow one another.
template <int WR, int WN, int MR, int NR>
__global__ __launch_bounds__(WR * WN * 64) void lora_shrink_wide_kernel(LoraArgs p) {
  constexpr int ROWS = WR * MR * 16, THREADS = WR * WN * 64;
  constexpr int RA = WN * NR * 16;                      // rows of A in a stage
  constexpr int NX = ROWS * 8 / THREADS;      // 16-byte chunks a thread loads
  constexpr int NA = (RA * 8 + THREADS - 1) / THREADS;
  constexpr int kStage = (ROWS + RA) * 128;
  __shared__ __align__(16) uint8_t lds[2][kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int s = blockIdx.x % p.S;
  ListedTile t;
  if (!find_listed<ROWS>(p, blockIdx.x / p.S, &t) || t.g >= p.L) return;
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
    const int c = tid + j * THREADS, r = c >> 3;
    xp[j] = p.x + (int64_t)row_of(r) * p.ldx + (int64_t)kb0 * 64 + (c & 7) * 8;
    xo[j] = r * 128 + (((c & 7) ^ swz_f(r)) << 4);
  }
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    const int c = min(tid + j * THREADS, RA * 8 - 1), r = c >> 3;
    ap[j] = p.a + ((int64_t)t.g * p.r + min(r, p.r - 1)) * p.K + (int64_t)kb0 * 64 + (c & 7) * 8;
    ao[j] = (ROWS + r) * 128 + (((c & 7) ^ swz_f(r)) << 4);
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
      if (RA * 8 % THREADS == 0 || tid + j * THREADS < RA * 8)
        *reinterpret_cast<v4u *>(&lds[b][ao[j]]) = w[j];
    load(x, w, i + 2);
    lds_barrier();
    if (idle) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int chunk = (lane >> 4) * 2 + h;
      v8bf xv[MR], av[NR];
#pragma unroll
      for (int q = 0; q < MR; ++q) {
        const int r = first + q * 16 + (lane & 15);
        xv[q] = *reinterpret_cast<const v8bf *>(&lds[b][r * 128 + ((chunk ^ swz_f(r)) << 4)]);
      }
#pragma unroll
      for (int f = 0; f < NR; ++f) {
        const int r = rank0 + f * 16 + (lane & 15);
        av[f] = *reinterpret_cast<const v8bf *>(
            &lds[b][(ROWS + r) * 128 + ((chunk ^ swz_f(r)) << 4)]);
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

// A tile's rows and adapter for the expand kernel, and its h: the parts added,
// scaled, split, in the order in which the matrix instruction takes them (per
// 16 rows, 32 ranks and part of the split 64 lanes' 16 bytes), so that the many
// workgroups of the expand kernel find all of it by the tile's number alone.  A
// workgroup takes 4 runs of 8 ranks of a tile.
constexpr int kJoinChunks = kLoraThreads / kWideRows;
static_assert(kJoinChunks * 8 == kStepRanks, "a workgroup per tile and step");

__global__ __launch_bounds__(kLoraThreads) void lora_join_kernel(LoraArgs p) {
  const int chunks = p.r / 8, steps = rank_steps(p.r);
  const int tile = blockIdx.x / steps, part = blockIdx.x % steps;
  ListedTile t;
  const bool found = find_listed<kWideRows>(p, tile, &t);
  if (part == 0 && threadIdx.x == 0) p.tile_adapter[tile] = found ? t.g : -1;
  if (!found) return;
  // neighbouring threads take neighbouring runs of a row
  const int slot = threadIdx.x / kJoinChunks;
  int row = slot < t.rows ? p.order[t.start + slot] : -1;
  row = row < p.T ? row : -1;
  if (part == 0 && threadIdx.x % kJoinChunks == 0) p.tile_rows[(int64_t)tile * kWideRows + slot] = row;
  if (t.g >= p.L || row < 0) return;
  const float scale = p.scale ? p.scale[t.g] : 1.0f;
  const int ch = part * kJoinChunks + threadIdx.x % kJoinChunks;
  v4u h[kParts] = {};   // (zeros past a rank that is not a multiple of 32)
  if (ch < chunks) join_parts(p, p.h + (int64_t)row * p.r + ch * 8, scale, h);
  v4u *o = reinterpret_cast<v4u *>(p.hs) +
           (((int64_t)tile * 4 + (slot >> 4)) * steps + part) * (kParts * 64) + (ch & 3) * 16 +
           (slot & 15);
#pragma unroll
  for (int i = 0; i < kParts; ++i) o[i * 64] = h[i];
}

// out for a tile's 64 rows and ct runs of 16 F columns, 16 rows a wave.  Rows
// of the instruction are rows of the batch, its columns columns of out, and a
// lane's F fragments are F consecutive columns: base and out move as 32 F
// contiguous bytes of a row per 16 lanes.  h stays in registers for all ct
// runs; B's run goes through LDS (it is contiguous in memory, but a fragment
// takes a row per lane).  B and base are loaded one run ahead in registers (base
// in the run it is used in: 117 against 109 us below).
// F = 8 up to rank 32, where base and out are all that counts, and 4 above,
// where its fewer registers let more workgroups overlap (8192 rows, N = 18432,
// r = 32: 117 us with 8, 127 with 4; 4099 rows, N = 4096, r = 128: 29 and 27).
// Now 110 us (5.5 TB/s of base and out) and 24 us (2.8 TB/s; vector ALU 46 %, matrix
// cores 29 %, LDS 24 % of the busy cycles).
template <int NS, int F>   // up to NS steps of 32 ranks (NS = 0: up to 16 ranks)
__global__ __launch_bounds__(kLoraThreads) void lora_expand_wide_kernel(LoraArgs p, int ct) {
  extern __shared__ __align__(16) uint8_t lds[];   // B's run: [fragment][16] rows
  constexpr int COLS = 16 * F;
  constexpr int NH = NS ? NS : 1;
  constexpr int NB = NS ? F * NS / 4 : F / 8;   // 16-byte chunks a thread loads of a run
  typedef unsigned piece __attribute__((ext_vector_type(F / 2), aligned(2)));   // F columns
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int runs = (int)((p.N + COLS - 1) / COLS);
  const int groups = (runs + ct - 1) / ct;
  const int tile = blockIdx.x / groups;
  const int run0 = (int)(blockIdx.x % groups) * ct;
  const int run1 = min(run0 + ct, runs);
  const int i16 = lane & 15, g16 = lane >> 4;
  const int g = p.tile_adapter[tile];
  // rows g16 * 4 + q of the wave's 16, -1 past the tile's
  const int4 row4 = reinterpret_cast<const int4 *>(p.tile_rows)[(int64_t)tile * 16 + wave * 4 + g16];
  const int row[4] = {row4.x, row4.y, row4.z, row4.w};
  const int chunks = p.r / 8;                 // 16-byte chunks of a row of B
  const int steps = rank_steps(p.r);
  const int pitch = rank_pitch(p.r);
  v4u hv[NH][kParts], br[NB];
  const v4u *hr = reinterpret_cast<const v4u *>(p.hs) +
                  ((int64_t)tile * 4 + wave) * steps * (kParts * 64) + lane;
#pragma unroll
  for (int st = 0; st < NH; ++st)
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      hv[st][i] = st < steps ? hr[(st * kParts + i) * 64] : v4u{0, 0, 0, 0};
  if (g < 0) return;
  const bool worn = g < p.L;
  // chunk c of a run is row (column of out) n = c / chunks of it, and n = F i + f
  // is row i of fragment f.  Columns past N read as zeros.
  int off[NB], dst[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int c = min(tid + j * kLoraThreads, COLS * chunks - 1);
    const int n = c / chunks, ch = c - n * chunks;
    off[j] = n * p.r + ch * 8;
    dst[j] = ((n % F) * 16 + n / F) * pitch + ch * 16;
  }
  const uint16_t *bg = p.b + (worn ? (int64_t)g * p.N * p.r : 0);
  auto load_b = [&](int run) {
    const int64_t left = (p.N - (int64_t)run * COLS) * p.r;
#pragma unroll
    for (int j = 0; j < NB; ++j)
      br[j] = off[j] < left ? *reinterpret_cast<const v4u *>(bg + (int64_t)run * COLS * p.r + off[j])
                            : v4u{0, 0, 0, 0};
  };
  piece next[4];   // base of the run to come
  auto load_base = [&](int run) {
    const int64_t c = (int64_t)run * COLS + i16 * F;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      next[q] = p.base && row[q] >= 0 && c + F <= p.N
                    ? __builtin_nontemporal_load(reinterpret_cast<const piece *>(
                          p.base + (int64_t)row[q] * p.ldb + c))
                    : piece(0);
  };
  if (worn) {
    load_b(run0);
    clear_past_rank<COLS>(lds, p.r, tid);
  }
  load_base(run0);
  for (int run = run0; run < run1; ++run) {
    const int64_t c0 = (int64_t)run * COLS + i16 * F;
    piece bs[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) bs[q] = next[q];
    if (run + 1 < run1) load_base(run + 1);
    v4f acc[F];
#pragma unroll
    for (int f = 0; f < F; ++f) acc[f] = v4f{0, 0, 0, 0};
    if (worn) {
      lds_barrier();   // the run before has been read
#pragma unroll
      for (int j = 0; j < NB; ++j) *reinterpret_cast<v4u *>(&lds[dst[j]]) = br[j];
      lds_barrier();
      load_b(min(run + 1, run1 - 1));
#pragma unroll
      for (int st = 0; st < NH; ++st) {
        if (st >= steps) break;
        const int chunk = st * 4 + g16;
        v8bf bv[F];
#pragma unroll
        for (int f = 0; f < F; ++f)
          bv[f] = *reinterpret_cast<const v8bf *>(&lds[(f * 16 + i16) * pitch + chunk * 16]);
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
          for (int f = 0; f < F; ++f)
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, hv[st][i]),
                                                             bv[f], acc[f], 0, 0, 0);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (row[q] < 0) continue;
      uint16_t *o = p.out + (int64_t)row[q] * p.ldo;
      if (c0 + F <= p.N) {
        piece w;
#pragma unroll
        for (int j = 0; j < F / 2; ++j)
          w[j] = (uint32_t)bf_bits(bf16_lo(bs[q][j]) + acc[2 * j][q]) |
                 ((uint32_t)bf_bits(bf16_hi(bs[q][j]) + acc[2 * j + 1][q]) << 16);
        __builtin_nontemporal_store(w, reinterpret_cast<piece *>(o + c0));
      } else {
#pragma unroll
        for (int j = 0; j < F; ++j)
          if (c0 + j < p.N) {
            const float f = p.base ? bf16_lo(p.base[(int64_t)row[q] * p.ldb + c0 + j]) : 0.0f;
            o[c0 + j] = bf_bits(f + acc[j][q]);
          }
      }
    }
  }
}

namespace {
// Rows of a shrink tile of a larger batch.  From kBigBatch rows on 128, with
// eight waves: A is read from L2 once per 128 rows, which is what bounds the
// kernel there (4099 rows, K = 14336, r = 128: 45 -> 36 us; 4096 rows, K = 4096,
// r = 64: 14.5 -> 12.0).  With fewer rows the larger tiles leave compute units
// idle (2048 rows, K = 14336, r = 128: 20.6 us in tiles of 64, 25.3 in 128).  With
// many adapters of few rows each they cost more than they save (K = 4096, r = 16:
// 4096 rows of 512 adapters 30.3 us against 22.4 in 64, of 64 adapters 11.6 against
// 9.4, 8192 rows of 200 19.2 against 17.8), but the pool's size, all that is known
// here, does not tell how many are in use.
constexpr int64_t kBigBatch = 4096;
int shrink_rows(int64_t T) { return T >= kBigBatch ? 128 : kWideRows; }

// Tiles a batch can have at most: full ones, and one more per adapter (and
// for the rows without one).
int64_t max_tiles(int64_t T, int L, int rows) {
  const int64_t groups = (int64_t)L + 1 < T ? (int64_t)L + 1 : T;
  const int64_t tiles = T / rows + groups;
  return tiles < T ? tiles : T;
}

// K ranges, each at least 256 of K, that give two workgroups of four waves or
// one of eight per compute unit (more of either measured slower: 36 -> 43 us
// at the sizes above).
int split_of(int64_t T, int64_t K, int32_t r, int L) {
  int64_t units = T <= kDirectRows ? max_tiles(T, L, kTileRows) * ((r + 15) / 16)
                                   : max_tiles(T, L, shrink_rows(T));
  int64_t s = (T >= kBigBatch ? 256 : 512) / units;
  if (s > K / 256) s = K / 256;
  if (s > kMaxSplit) s = kMaxSplit;
  return s < 1 ? 1 : (int)s;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// h of the tiles, split: 64 lanes' 16 bytes per 16 rows, 32 ranks and part.
size_t split_bytes(int64_t tiles, int32_t r) { return (size_t)tiles * 4 * rank_steps(r) * kStepBytes; }

// Columns of a run of the larger batches' expand kernel: 16 times its F.
int run_cols(int32_t r) { return r <= 32 ? 128 : 64; }

// Workgroups of a batch's launches and the columns' runs of one of the last.
struct LoraGrid {
  int64_t shrink, join, expand, ct;
};
LoraGrid lora_grid(int64_t T, int64_t K, int64_t N, int32_t r, int L) {
  LoraGrid g{};
  if (T <= kDirectRows) {
    const int64_t tiles = max_tiles(T, L, kTileRows);
    g.shrink = tiles * ((r + 15) / 16) * split_of(T, K, r, L);
    g.expand = tiles * ((N + kSmallCols - 1) / kSmallCols);
    return g;
  }
  const int64_t tiles = max_tiles(T, L, kWideRows);
  const int64_t runs = (N + run_cols(r) - 1) / run_cols(r);
  g.shrink = max_tiles(T, L, shrink_rows(T)) * split_of(T, K, r, L);
  g.join = tiles * rank_steps(r);
  // several runs of columns a workgroup where that leaves five per compute unit
  g.ct = tiles * runs / 1280;
  g.ct = g.ct < 1 ? 1 : g.ct > 4 ? 4 : g.ct;
  g.expand = tiles * ((runs + g.ct - 1) / g.ct);
  return g;
}

}  // namespace

// Whether every launch stays below 2^32 threads (a larger grid wraps).
bool lora_fits(int64_t T, int64_t K, int64_t N, int32_t r, int32_t L) {
  if (T == 0) return true;
  const LoraGrid g = lora_grid(T, K, N, r, L);
  constexpr int64_t most = ((int64_t(1) << 32) - 1) / (2 * kLoraThreads);   // (shrink: 512)
  return g.shrink <= most && g.join <= 2 * most && g.expand <= 2 * most;
}

size_t lora_workspace_bytes(int64_t T, int64_t K, int32_t r, int32_t L, bool listed) {
  size_t n = align256(sizeof(float) * (size_t)split_of(T, K, r, L) * T * r);
  const int64_t tiles = max_tiles(T, L, kWideRows);
  if (T > kDirectRows)
    n += split_bytes(tiles, r) + sizeof(int32_t) * (size_t)tiles * kWideRows +
         align256(sizeof(int32_t) * (size_t)tiles);
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
  p.S = split_of(T, K, r, L);
  p.copy_bare = base != out;
  char *w = static_cast<char *>(work);
  p.h = reinterpret_cast<float *>(w);
  w += align256(sizeof(float) * (size_t)p.S * T * r);
  const LoraGrid grid = lora_grid(T, K, N, r, L);
  if (T <= kDirectRows) {
    lora_shrink_kernel<<<(unsigned)grid.shrink, kLoraThreads, 0, stream>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
    const size_t lds = (size_t)rank_steps(r) * kStepBytes + (size_t)kSmallCols * rank_pitch(r);
    lora_expand_kernel<<<(unsigned)grid.expand, kLoraThreads, lds, stream>>>(p);
    return hipGetLastError();
  }
  const int64_t tiles = max_tiles(T, L, kWideRows);
  p.hs = reinterpret_cast<uint16_t *>(w);
  w += split_bytes(tiles, r);
  p.tile_rows = reinterpret_cast<int32_t *>(w);
  w += sizeof(int32_t) * (size_t)tiles * kWideRows;
  p.tile_adapter = reinterpret_cast<int32_t *>(w);
  w += align256(sizeof(int32_t) * (size_t)tiles);
  if (!order) {
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
  const unsigned gs = (unsigned)grid.shrink;
#define FP8BLK_SHRINK(W, NR)                                                                 \
  (shrink_rows(T) == kWideRows                                                               \
       ? (lora_shrink_wide_kernel<4 / W, W, W, NR><<<gs, 256, 0, stream>>>(p), hipSuccess)   \
       : (lora_shrink_wide_kernel<8 / W, W, W, NR><<<gs, 512, 0, stream>>>(p), hipSuccess))
  if (r <= 16) FP8BLK_SHRINK(1, 1);
  else if (r <= 32) FP8BLK_SHRINK(1, 2);
  else if (r <= 64) FP8BLK_SHRINK(2, 2);
  else if (r <= 128) FP8BLK_SHRINK(2, 4);
  else FP8BLK_SHRINK(2, 8);
#undef FP8BLK_SHRINK
  if (hipError_t e = hipGetLastError()) return e;
  lora_join_kernel<<<(unsigned)grid.join, kLoraThreads, 0, stream>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
#define FP8BLK_EXPAND(NS, F)                                                              \
  (lora_expand_wide_kernel<NS, F><<<(unsigned)grid.expand, kLoraThreads, lds, stream>>>(   \
      p, (int)grid.ct))
  const size_t lds = (size_t)run_cols(r) * rank_pitch(r);
  if (r <= 16) FP8BLK_EXPAND(0, 8);
  else if (r <= 32) FP8BLK_EXPAND(1, 8);
  else if (r <= 64) FP8BLK_EXPAND(2, 4);
  else if (r <= 128) FP8BLK_EXPAND(4, 4);
  else FP8BLK_EXPAND(8, 4);
#undef FP8BLK_EXPAND
  return hipGetLastError();
}

}  // namespace fp8blk
