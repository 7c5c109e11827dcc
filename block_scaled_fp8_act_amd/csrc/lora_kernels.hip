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

namespace {

constexpr int kTileRows = 16;
constexpr int kLoraThreads = 256;
constexpr int kLoraWaves = kLoraThreads / 64;
// Batches up to a wave's width find their rows from the adapter numbers
// directly; larger ones through a listing by adapter (order, offsets).
constexpr int kDirectRows = 64;
constexpr int kMaxRank = 256;
constexpr int kMaxSplit = 16;

struct LoraArgs {
  const uint16_t *x, *a, *b, *base;
  int64_t ldx, ldb, ldo;
  const int32_t *ids;             // [T], T <= kDirectRows
  const int32_t *order, *offsets; // [T], [L + 1], T > kDirectRows
  const float *scale;             // [L] or NULL (1)
  float *h;                       // [S][T][r]
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

// Tile `index` of a batch listed by adapter: a wave adds up the adapters'
// tile counts, 64 adapters at a time, until it reaches the tile.
__device__ __forceinline__ bool find_tile_listed(const LoraArgs &p, int index, Tile *t) {
  const int lane = threadIdx.x & 63;
  const int T = (int)p.T;
  int done = 0;
  for (int g0 = 0; g0 <= p.L; g0 += 64) {
    const int g = g0 + lane;
    int lo = g <= p.L ? p.offsets[g] : T;
    int hi = g < p.L ? p.offsets[g + 1] : T;
    lo = min(max(lo, 0), T);
    hi = min(max(hi, lo), T);
    int n = (hi - lo + kTileRows - 1) / kTileRows;
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
      const int start = __builtin_amdgcn_readlane(lo, l) +
                        (index - done - __builtin_amdgcn_readlane(scan - n, l)) * kTileRows;
      const int end = __builtin_amdgcn_readlane(hi, l);
      const int at = start + (lane & 15);
      const int row = at < end ? p.order[at] : -1;
      t->row = row < T ? row : -1;
      return true;
    }
    done += __builtin_amdgcn_readlane(scan, 63);
  }
  return false;
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
// columns of the output, mapped so that a lane ends with 16 consecutive
// columns of one row, and base and out move 16 bytes at a time.
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
      const int64_t n = n0 + (m >> 2) * 16 + f * 4 + (m & 3);
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
  const int64_t c0 = n0 + (lane >> 4) * 16;
  uint16_t *o = p.out + (int64_t)t.row * p.ldo;
  const uint16_t *bs = p.base ? p.base + (int64_t)t.row * p.ldb : nullptr;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t c = c0 + q * 8;
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

namespace {

// Tiles a batch can have at most: full ones, and one more per adapter (and
// for the rows without one).
int64_t max_tiles(int64_t T, int L) {
  if (T <= kDirectRows) return T;
  const int64_t groups = (int64_t)L + 1 < T ? (int64_t)L + 1 : T;
  return T / kTileRows + groups;
}

// K ranges: enough workgroups to fill the chip twice, at least 256 of K each.
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
  const bool direct = T <= kDirectRows;
  if (!direct && !order) {
    w += align256(sizeof(float) * (size_t)p.S * T * r);
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
