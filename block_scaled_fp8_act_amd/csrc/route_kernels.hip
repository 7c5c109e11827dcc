// Mixture-of-experts routing for gfx950: the top-k experts of each token with
// their softmax weights, the rows per expert and the balance loss, and the
// gradient of the logits; rows listed by group (a stable counting sort); and
// the weighted sum that brings the experts' rows back to their tokens, with
// its gradient.
//
// All of it is memory work with little arithmetic, except the selection of the
// top k, which is bound by the vector ALU (see route_kernel); at the sizes of a
// decode step launches and latency are all there is.
#include "fp8blk_device.h"
#include "fp8blk_launch.h"

#include <float.h>
#include <math.h>

namespace fp8blk {

namespace {

constexpr float kNegInf = -INFINITY;

// Reductions over the LPR lanes that share a row (16: one DPP row; 64: the
// wave).  Each step adds the mirror lane's value, so every lane of the row
// holds the same bits afterwards.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<0xB1>(v);    // quad_perm [1,0,3,2]
  v += dpp_f<0x4E>(v);    // quad_perm [2,3,0,1]
  v += dpp_f<0x141>(v);   // row_half_mirror
  v += dpp_f<0x140>(v);   // row_mirror
  if constexpr (LPR == 64) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
  }
  return v;
}

template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  v = row16_max(v);
  if constexpr (LPR == 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
}

template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}

template <int LPR>
__device__ __forceinline__ int row_min(int v) {
  v = min(v, dpp_i<0xB1>(v));
  v = min(v, dpp_i<0x4E>(v));
  v = min(v, dpp_i<0x141>(v));
  v = min(v, dpp_i<0x140>(v));
  if constexpr (LPR == 64) {
    v = min(v, __shfl_xor(v, 16));
    v = min(v, __shfl_xor(v, 32));
  }
  return v;
}

// How many of the other 15 lanes of a DPP row come before this one: a larger
// value, or an equal one with a lower index (LANES 15 .. 1, by rotation); and
// how many have a larger value.
template <int N = 15>
__device__ __forceinline__ int row_rank(float v, int e) {
  const float ov = dpp_f<0x120 + N>(v);   // row_ror:N
  const int oe = dpp_i<0x120 + N>(e);
  const int before = ov > v || (ov == v && oe < e) ? 1 : 0;
  if constexpr (N > 1) return before + row_rank<N - 1>(v, e);
  else return before;
}
template <int N = 15>
__device__ __forceinline__ int row_larger(float v) {
  const int before = dpp_f<0x120 + N>(v) > v ? 1 : 0;
  if constexpr (N > 1) return before + row_larger<N - 1>(v);
  else return before;
}

// e^(v - peak) for v <= peak: the difference first, so that logits of any size
// (a row of the type's lowest value among them) leave it small.  The hardware's
// 2^y takes the rounded y = d log2 e; what e^d has beyond it, d - y ln 2, is tiny and
// added to first order.  That leaves 3 units of 2^-24 and the constant's 0.05 |d|,
// not |d| for y's rounding.  Where 2^y is 0 the correction can be of any size, an
// infinity or (v = -inf) NaN: the bounds make a number of it.  NaN stays NaN.
__device__ __forceinline__ float exp_from(float v, float peak) {
  const float d = v - peak;
  const float y = d * 0x1.715476p+0f;                                    // log2 e
  const float e = __builtin_amdgcn_exp2f(y);
  const float rest = __builtin_amdgcn_fmed3f(fmaf(y, -0x1.62e43p-1f, d), -1.0f, 1.0f);   // ln 2
  return fmaf(e, rest, e);
}

// Element c of lane `sub` of a row: VEC consecutive experts per load.
template <int LPR, int VEC>
__device__ __forceinline__ int expert_of(int c, int sub) {
  return ((c / VEC) * LPR + sub) * VEC + c % VEC;
}

// A lane's logits of a row.  Slots past E load the row's start, so that no load
// waits for a condition, and become -inf, like all of a row that is not live.
// (Loading the next rows ahead of the present ones' work measured no faster:
// the vector ALU is the bound.)
template <typename T, int LPR, int V, int VEC>
struct RowLoad {
  static_assert(VEC == 1 || VEC == 4, "one element or four per load");
  static constexpr int W = VEC * sizeof(T) <= 4 ? 1 : VEC * sizeof(T) / 4;   // dwords a load
  uint32_t w[V / VEC][W];

  __device__ __forceinline__ void load(const T *row, int E, int sub) {
#pragma unroll
    for (int i = 0; i < V / VEC; ++i) {
      const int e = expert_of<LPR, VEC>(i * VEC, sub);
      const T *p = row + (e < E ? e : 0);
      if constexpr (W == 4) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        w[i][0] = q.x; w[i][1] = q.y; w[i][2] = q.z; w[i][3] = q.w;
      } else if constexpr (W == 2) {
        const uint2 q = *reinterpret_cast<const uint2 *>(p);
        w[i][0] = q.x; w[i][1] = q.y;
      } else {
        w[i][0] = *p;
      }
    }
  }
  __device__ __forceinline__ void unpack(int E, int sub, bool live, float *v) const {
#pragma unroll
    for (int i = 0; i < V / VEC; ++i) {
      const bool in = live && expert_of<LPR, VEC>(i * VEC, sub) < E;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float f;
        if constexpr (sizeof(T) == 4) f = __uint_as_float(w[i][j]);
        else f = j & 1 ? bf16_hi(w[i][j / 2]) : bf16_lo(w[i][j / 2]);
        v[i * VEC + j] = in ? f : kNegInf;
      }
    }
  }
};

// fp32 -> bf16 bits with the hardware's rounding (nearest even, NaN kept).
__device__ __forceinline__ uint16_t to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)to_bf16(a) | ((uint32_t)to_bf16(b) << 16);
}

template <typename T, int LPR, int V, int VEC>
__device__ __forceinline__ void store_row(T *row, int E, int sub, const float *v) {
#pragma unroll
  for (int c = 0; c < V; c += VEC) {
    const int e = expert_of<LPR, VEC>(c, sub);
    if (e >= E) continue;
    if constexpr (sizeof(T) == 4 && VEC == 4) {
      *reinterpret_cast<uint4 *>(row + e) =
          make_uint4(__float_as_uint(v[c]), __float_as_uint(v[c + 1]), __float_as_uint(v[c + 2]),
                     __float_as_uint(v[c + 3]));
    } else if constexpr (sizeof(T) == 2 && VEC == 4) {
      *reinterpret_cast<uint2 *>(row + e) =
          make_uint2(pack_bf16(v[c], v[c + 1]), pack_bf16(v[c + 2], v[c + 3]));
    } else {
      if constexpr (sizeof(T) == 4) row[e] = __float_as_uint(v[c]);
      else row[e] = to_bf16(v[c]);
    }
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Routing, forward.
//
// For a live row (mask set, some logit above -inf): S = its k largest logits,
// ties to the lowest expert; m their largest; p_e = e^(l_e - m) / sum over all
// experts; weights = the same over S alone (renormalize) or p on S.  c_e = the
// number of rows that chose e, n = the number of live rows, and the balance
// loss = coef * sum_e (c_e E / (k n)) * (sum_t p_te / n).
//
// LPR lanes hold a row, V logits each, so a wave holds 64 / LPR rows and the
// row reductions are DPP steps (16 lanes) with no LDS.  The k largest come from
// the few logits that reach the k-th of the lanes' bests (below); where those
// are more than 16, and in rows over the whole wave, k rounds take the row's
// best of the lanes' bests, and the lane that had it drops it and looks for its
// next.  The probabilities' sums over rows stay in registers (one per logit
// slot) over all rows of a wave and are added over waves and workgroups in a
// fixed order, so results do not vary between runs; counts are integer LDS
// atomics.  The workgroup's sums go to `part` and route_finish_kernel adds them,
// except when one workgroup does all rows.
// Measured: 131072 x 256 fp32, k = 8, with the loss: 49-51 us (2.7 TB/s of logits;
// the vector ALU bounds it: 600 instructions for four rows keep it active 79 % of
// the compute units' busy cycles; 78 us with the rounds alone, 47 with exponentials
// of one uncorrected product), finish 6 us; 4096 x 32: 4.8 and 4 us; 16 x 256, one
// workgroup: 3.6 us.  The more experts a row chooses, the more often it has over 16
// candidates, and one such row takes its wave through both ways.
constexpr int kRouteMaxThreads = 1024;
constexpr int kRouteMaxWaves = kRouteMaxThreads / 64;
constexpr int kRouteMaxBlocks = 256;
constexpr int kRouteMaxK = 32;

struct RouteArgs {
  const void *logits;
  const uint8_t *mask;
  int64_t T;
  int E, k, renorm, loss;   // loss: sums of probabilities wanted
  float coef;
  int32_t *ids;
  float *weights;
  int32_t *counts, *rows;
  float *loss_out;
  // per workgroup: E counts, then one for the live rows, then E fp32 sums
  int32_t *part;
  int32_t *ticket;
};

__device__ __forceinline__ size_t part_stride(int E) { return 2 * (size_t)E + 1; }

__device__ __forceinline__ float balance(double sum, float coef, int E, int k, int64_t n) {
  const double m = n > 0 ? (double)n : 1.0;
  return (float)((double)coef * E / ((double)k * m * m) * sum);
}

template <typename T, int LPR, int V, int VEC>
__global__ __launch_bounds__(kRouteMaxThreads) void route_kernel(RouteArgs a) {
  extern __shared__ float lds[];          // [E] counts, [waves][E] sums
  __shared__ int live_rows[kRouteMaxWaves];
  __shared__ float2 found[LPR == 16 ? kRouteMaxWaves : 1][4][16];
  const int threads = blockDim.x, waves = threads / 64;
  constexpr int RPW = 64 / LPR;
  constexpr int SLOTS = (kRouteMaxK + LPR - 1) / LPR;
  int *hist = reinterpret_cast<int *>(lds);
  float *sums = lds + a.E;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane % LPR;
  for (int e = tid; e < a.E; e += threads) hist[e] = 0;
  __syncthreads();

  float acc[V];
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.0f;
  int live_count = 0;
  const bool all = a.loss || !a.renorm;   // probabilities over every expert
  const int64_t step = (int64_t)gridDim.x * waves * RPW;
  const int64_t first = ((int64_t)blockIdx.x * waves + wave) * RPW;
  for (int64_t r0 = first; r0 < a.T; r0 += step) {
    const int64_t row = r0 + lane / LPR;
    const int64_t r = row < a.T ? row : a.T - 1;
    float v[V];
    RowLoad<T, LPR, V, VEC> in;
    in.load(static_cast<const T *>(a.logits) + r * a.E, a.E, sub);
    in.unpack(a.E, sub, row < a.T && (!a.mask || a.mask[r]), v);
    float bestv = kNegInf;
    int bestc = 0;
#pragma unroll
    for (int c = 0; c < V; ++c) bestv = fmaxf(bestv, v[c]);
#pragma unroll
    for (int c = V - 1; c >= 0; --c) bestc = v[c] == bestv ? c : bestc;
    const float peak = row_max<LPR>(bestv);
    const bool live = peak > kNegInf;
    const float top = live ? peak : 0.0f;
    float inv = 0.0f;
    if (all) {
      float ex[V], total = 0.0f;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        ex[c] = exp_from(v[c], top);
        total += ex[c];
      }
      total = row_sum<LPR>(total);
      inv = live ? 1.0f / total : 0.0f;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] += ex[c] * inv;
    }
    bool done = false;
    if constexpr (LPR == 16) {
      // The k-th largest of the 16 lanes' bests bounds the k-th largest logit
      // from below, and few logits reach it (11 of 256 on average at k = 8).
      // Up to 16 of them are laid out one a lane, where a row's order is 15
      // rotations; with more (ties, or few experts open) the rounds below.
      if (a.k <= 16) {
        const float bound = fmaxf(
            -row_max<LPR>(row_larger(bestv) < a.k ? -bestv : kNegInf), -FLT_MAX);
        int n = 0;
#pragma unroll
        for (int c = 0; c < V; ++c) n += v[c] >= bound ? 1 : 0;
        int at = n;   // inclusive sum over the row's lanes
        at += dpp_i<0x111>(at);   // row_shr:1, 2, 4, 8
        at += dpp_i<0x112>(at);
        at += dpp_i<0x114>(at);
        at += dpp_i<0x118>(at);
        done = __builtin_amdgcn_ballot_w64(at > 16) == 0;
        if (done) {
          float2 *mine = found[wave][lane / LPR];
          mine[sub] = make_float2(kNegInf, 0.0f);
          at -= n;
#pragma unroll
          for (int c = 0; c < V; ++c)
            if (v[c] >= bound)
              mine[at++] = make_float2(v[c], __int_as_float(expert_of<LPR, VEC>(c, sub)));
          // the wave's own LDS: in order, but the compiler has to keep it so
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_wave_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
          const float2 f = mine[sub];
          const int e = __float_as_int(f.y);
          const int rank = row_rank(f.x, e);
          const bool chosen = f.x > kNegInf && rank < a.k;
          const float w = chosen ? exp_from(f.x, top) : 0.0f;
          if (a.renorm) {
            const float total = row_sum<LPR>(w);
            inv = live ? 1.0f / total : 0.0f;
          }
          // lanes past the candidates fill the slots left over
          const int j = chosen ? rank : f.x > kNegInf ? a.k : sub;
          if (j < a.k && row < a.T) {
            a.ids[row * a.k + j] = chosen ? e : -1;
            a.weights[row * a.k + j] = w * inv;
            if (chosen) atomicAdd(&hist[e], 1);
          }
        }
      }
    }
    if (!done) {
      float sel_v[SLOTS];
      int sel_e[SLOTS];
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        sel_v[s] = kNegInf;
        sel_e[s] = -1;
      }
      for (int j = 0; j < a.k; ++j) {
        const float m = j ? row_max<LPR>(bestv) : peak;
        const int mine = expert_of<LPR, VEC>(bestc, sub);
        const int e = row_min<LPR>(m > kNegInf && bestv == m ? mine : INT32_MAX);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          if (j == s * LPR + sub && e != INT32_MAX) {
            sel_v[s] = m;
            sel_e[s] = e;
          }
        }
        if (j + 1 == a.k) break;
        const int drop = mine == e ? bestc : -1;
        bestv = kNegInf;
#pragma unroll
        for (int c = 0; c < V; ++c) {
          v[c] = c == drop ? kNegInf : v[c];
          bestv = fmaxf(bestv, v[c]);
        }
#pragma unroll
        for (int c = V - 1; c >= 0; --c) bestc = v[c] == bestv ? c : bestc;
      }
      float w[SLOTS], total = 0.0f;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        w[s] = sel_e[s] >= 0 ? exp_from(sel_v[s], top) : 0.0f;
        total += w[s];
      }
      if (a.renorm) {
        total = row_sum<LPR>(total);
        inv = live ? 1.0f / total : 0.0f;
      }
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int j = s * LPR + sub;
        if (j < a.k && row < a.T) {
          a.ids[row * a.k + j] = sel_e[s];
          a.weights[row * a.k + j] = w[s] * inv;
          if (sel_e[s] >= 0) atomicAdd(&hist[sel_e[s]], 1);
        }
      }
    }
    live_count += __popcll(__builtin_amdgcn_ballot_w64(live && sub == 0));
  }

  if (lane == 0) live_rows[wave] = live_count;
  if (a.loss) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if constexpr (LPR == 16) {
        acc[c] += __shfl_xor(acc[c], 16);
        acc[c] += __shfl_xor(acc[c], 32);
      }
      const int e = expert_of<LPR, VEC>(c, sub);
      if (lane < LPR && e < a.E) sums[wave * a.E + e] = acc[c];
    }
  }
  __syncthreads();
  int live_total = 0;
  for (int w = 0; w < waves; ++w) live_total += live_rows[w];
  const bool only = gridDim.x == 1;
  int32_t *part = a.part + blockIdx.x * part_stride(a.E);
  float mine = 0.0f;   // this thread's experts: sum of c_e * sum p_e
  for (int e = tid; e < a.E; e += threads) {
    float s = 0.0f;
    if (a.loss)
      for (int w = 0; w < waves; ++w) s += sums[w * a.E + e];
    if (only) {
      a.counts[e] = hist[e];
      mine += (float)hist[e] * s;
    } else {
      part[e] = hist[e];
      if (a.loss) part[a.E + 1 + e] = __float_as_int(s);
    }
  }
  if (!only) {
    if (tid == 0) {
      part[a.E] = live_total;
      if (blockIdx.x == 0) *a.ticket = 0;
    }
    return;
  }
  if (tid == 0 && a.rows) *a.rows = live_total;
  if (!a.loss) return;
  __syncthreads();
  mine = row_sum<64>(mine);
  if (lane == 0) sums[wave] = mine;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < waves; ++w) s += (double)sums[w];
    *a.loss_out = balance(s, a.coef, a.E, a.k, live_total);
  }
}

// Adds the workgroups' counts and sums: COLS experts per workgroup, the other
// threads share the workgroups' entries.  Up to 64 experts one workgroup does
// all of them; beyond, the last one to finish (an integer ticket; nothing
// waits for it) adds the experts' terms of the loss in order.
constexpr int kFinishThreads = 1024;

template <int COLS>
__global__ __launch_bounds__(kFinishThreads) void route_finish_kernel(RouteArgs a, int blocks,
                                                                      float *terms) {
  constexpr int SL = kFinishThreads / COLS;      // slices of the workgroups
  constexpr int WAVES = kFinishThreads / 64;
  __shared__ int cnt[SL][COLS + 1];
  __shared__ float sum[SL][COLS + 1];
  __shared__ int live[WAVES];
  __shared__ double part_sum[WAVES];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = tid % COLS, sl = tid / COLS;
  const int e = blockIdx.x * COLS + col;
  const size_t stride = part_stride(a.E);
  int c = 0, n = tid < blocks ? a.part[tid * stride + a.E] : 0;   // (at most 256 workgroups)
  float s = 0.0f;
  if (e < a.E) {
#pragma unroll 8
    for (int b = sl; b < blocks; b += SL) {
      c += a.part[b * stride + e];
      if (a.loss) s += __int_as_float(a.part[b * stride + a.E + 1 + e]);
    }
  }
  cnt[sl][col] = c;
  sum[sl][col] = s;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) n += __shfl_xor(n, d);
  if (lane == 0) live[wave] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) n += live[w];
  double t = 0.0;
  if (sl == 0 && e < a.E) {
    c = 0;
    s = 0.0f;
#pragma unroll 16
    for (int i = 0; i < SL; ++i) {
      c += cnt[i][col];
      s += sum[i][col];
    }
    a.counts[e] = c;
    t = (double)((float)c * s);
    if (a.loss && gridDim.x > 1)
      __hip_atomic_store(&terms[e], (float)c * s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (blockIdx.x == 0 && tid == 0 && a.rows) *a.rows = n;
  if (!a.loss) return;
  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0)
      last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             (int)gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    t = tid < a.E
            ? (double)__hip_atomic_load(&terms[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
            : 0.0;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) t += __shfl_xor(t, d);
  if (lane == 0) part_sum[wave] = t;
  __syncthreads();
  if (tid == 0) {
    t = 0.0;
    for (int w = 0; w < WAVES; ++w) t += part_sum[w];
    *a.loss_out = balance(t, a.coef, a.E, a.k, n);
  }
}
static_assert(kRouteMaxBlocks <= kFinishThreads, "one entry of live rows a thread");

// ---------------------------------------------------------------------------
// Routing, backward: for a live row, with g_e = dL * coef * E * c_e / (k n^2),
//   renormalize:  dl = p (g - <p, g>) + [on S] w (dw - <w, dw>)
//   otherwise:    the same softmax gradient with g_e + [e in S] dw_e, whose
//                 inner product over S is <w, dw>.
// The counts carry no gradient.  g enters as c_e minus the mean count: p sums
// to one, so the constant cancels exactly in dl and not in the rounding.
// The k values on S reach their lanes through LDS, each wave its own rows.
// Bound by HBM: 131072 x 256 fp32 57-59 us (4.6 TB/s of logits in and gradients
// out); 4096 x 32: 4 us.
struct RouteBackArgs {
  const void *logits;
  int64_t T;
  int E, k, renorm;
  float coef;
  const int32_t *ids;
  const float *weights;
  const int32_t *counts, *rows;
  const float *dw;       // [T, k] or NULL
  const float *dloss;    // one value or NULL
  void *dlogits;
};

constexpr int kBackThreads = 512;
constexpr int kBackWaves = kBackThreads / 64;
constexpr int kBackMaxBlocks = 1024;

template <typename T, int LPR, int V, int VEC>
__global__ __launch_bounds__(kBackThreads) void route_backward_kernel(RouteBackArgs a) {
  extern __shared__ float lds[];     // [waves][RPW][E]
  __shared__ int total_count[kBackWaves];
  constexpr int RPW = 64 / LPR;
  constexpr int SLOTS = (kRouteMaxK + LPR - 1) / LPR;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sub = lane % LPR;
  float *mine = lds + (size_t)(wave * RPW + lane / LPR) * a.E;
  for (int e = sub; e < a.E; e += LPR) mine[e] = 0.0f;
  const float dl = a.dloss ? *a.dloss : 0.0f;

  float g[V];
  if (a.dloss) {
    int part = 0;
    for (int e = tid; e < a.E; e += kBackThreads) part += a.counts[e];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) part += __shfl_xor(part, d);
    if (lane == 0) total_count[wave] = part;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kBackWaves; ++w) total += total_count[w];
    const float mean = (float)total / (float)a.E;
    const float n = (float)max(*a.rows, 1);
    const float f = dl * (a.coef * (float)a.E / ((float)a.k * n)) / n;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = expert_of<LPR, VEC>(c, sub);
      g[c] = e < a.E ? ((float)a.counts[e] - mean) * f : 0.0f;
    }
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) g[c] = 0.0f;
  }

  const int64_t step = (int64_t)gridDim.x * kBackWaves * RPW;
  for (int64_t r0 = ((int64_t)blockIdx.x * kBackWaves + wave) * RPW; r0 < a.T; r0 += step) {
    const int64_t row = r0 + lane / LPR;
    const int64_t at = row < a.T ? row : a.T - 1;
    const bool live = row < a.T && a.ids[at * a.k] >= 0;
    float v[V], d[V];
    RowLoad<T, LPR, V, VEC> in;
    in.load(static_cast<const T *>(a.logits) + at * a.E, a.E, sub);
    in.unpack(a.E, sub, live, v);
    int id[SLOTS];
    float w[SLOTS], dw[SLOTS], dot = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = s * LPR + sub;
      id[s] = -1;
      w[s] = dw[s] = 0.0f;
      if (j < a.k && live && a.dw) {
        const int i = a.ids[at * a.k + j];
        if (i >= 0 && i < a.E) {
          id[s] = i;
          w[s] = a.weights[at * a.k + j];
          dw[s] = a.dw[at * a.k + j];
          dot += w[s] * dw[s];
        }
      }
    }
    dot = row_sum<LPR>(dot);
    const float back = a.renorm ? dot : 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (id[s] >= 0) mine[id[s]] = w[s] * (dw[s] - back);
    // the wave's own LDS: in order, but the compiler has to keep it so
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    float peak = kNegInf;
#pragma unroll
    for (int c = 0; c < V; ++c) peak = fmaxf(peak, v[c]);
    peak = live ? row_max<LPR>(peak) : 0.0f;
    float total = 0.0f, inner = 0.0f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      v[c] = exp_from(v[c], peak);
      total += v[c];
      inner += v[c] * g[c];
    }
    total = row_sum<LPR>(total);
    const float inv = live ? 1.0f / total : 0.0f;
    inner = row_sum<LPR>(inner) * inv + (a.renorm ? 0.0f : dot);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = expert_of<LPR, VEC>(c, sub);
      // (not a product with 0: g and inner can be infinite or NaN)
      d[c] = live ? v[c] * inv * (g[c] - inner) + (e < a.E ? mine[e] : 0.0f) : 0.0f;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (id[s] >= 0) mine[id[s]] = 0.0f;
    if (row < a.T)
      store_row<T, LPR, V, VEC>(static_cast<T *>(a.dlogits) + row * a.E, a.E, sub, d);
  }
}

namespace {

// Kernel of a row width: the fewest logits per lane that cover E, in DPP rows
// of 16 lanes up to 256 experts and in whole waves above; four logits per
// load where the rows' alignment (E % 4 == 0) allows it, except that up to 64
// experts are spread over all lanes (a lane's best then says more).
template <typename T, template <typename, int, int, int> class L, typename... A>
hipError_t by_width(int E, A... args) {
  if (E <= 32) return L<T, 16, 2, 1>::go(args...);
  if (E <= 64) return L<T, 16, 4, 1>::go(args...);
  if (E % 4 == 0) {
    if (E <= 128) return L<T, 16, 8, 4>::go(args...);
    if (E <= 256) return L<T, 16, 16, 4>::go(args...);
    if (E <= 512) return L<T, 64, 8, 4>::go(args...);
    return L<T, 64, 16, 4>::go(args...);
  }
  if (E <= 128) return L<T, 16, 8, 1>::go(args...);
  if (E <= 256) return L<T, 16, 16, 1>::go(args...);
  if (E <= 512) return L<T, 64, 8, 1>::go(args...);
  return L<T, 64, 16, 1>::go(args...);
}

template <typename T, int LPR, int V, int VEC>
struct RouteLaunch {
  static hipError_t go(const RouteArgs *a, int blocks, int threads, hipStream_t st) {
    const size_t lds = sizeof(float) * a->E * (1 + (a->loss ? threads / 64 : 0));
    route_kernel<T, LPR, V, VEC><<<blocks, threads, lds + 64, st>>>(*a);
    return hipGetLastError();
  }
};

template <typename T, int LPR, int V, int VEC>
struct RouteBackLaunch {
  static hipError_t go(const RouteBackArgs *a, int blocks, hipStream_t st) {
    const size_t lds = sizeof(float) * a->E * kBackWaves * (64 / LPR);
    route_backward_kernel<T, LPR, V, VEC><<<blocks, kBackThreads, lds, st>>>(*a);
    return hipGetLastError();
  }
};

int route_rows_per_wave(int E) { return E <= 256 ? 4 : 1; }

// One workgroup for as many rows as cost less than the second launch, spread
// over its waves; else up to 256, of 8 waves while that leaves a wave one
// group of rows and of 16 beyond (fewer sums to add up).
struct RoutePlan {
  int blocks, threads;
};
RoutePlan route_plan(int64_t T, int E) {
  const int64_t waves = (T + route_rows_per_wave(E) - 1) / route_rows_per_wave(E);
  if (waves <= kRouteMaxWaves) return {1, waves <= 4 ? 256 : kRouteMaxThreads};
  const int per = waves <= 8 * kRouteMaxBlocks ? 8 : kRouteMaxWaves;
  const int64_t need = (waves + per - 1) / per;
  return {(int)(need < kRouteMaxBlocks ? need : kRouteMaxBlocks), per * 64};
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int32_t E) {
  const int blocks = route_plan(T, E).blocks;
  if (blocks <= 1) return 0;
  return sizeof(int32_t) * (blocks * (2 * (size_t)E + 1) + E + 1);
}

hipError_t launch_route(const void *logits, bool bf16, const uint8_t *mask, int64_t T, int32_t E,
                        int32_t k, bool renorm, float coef, int32_t *ids, float *weights,
                        int32_t *counts, int32_t *rows, float *loss, void *work,
                        hipStream_t stream) {
  RouteArgs a{};
  a.logits = logits;
  a.mask = mask;
  a.T = T;
  a.E = E;
  a.k = k;
  a.renorm = renorm;
  a.loss = loss != nullptr;
  a.coef = coef;
  a.ids = ids;
  a.weights = weights;
  a.counts = counts;
  a.rows = rows;
  a.loss_out = loss;
  const RoutePlan plan = route_plan(T, E);
  const int blocks = plan.blocks;
  a.part = static_cast<int32_t *>(work);
  float *terms = nullptr;
  if (blocks > 1) {
    terms = reinterpret_cast<float *>(a.part + blocks * (2 * (size_t)E + 1));
    a.ticket = reinterpret_cast<int32_t *>(terms + E);
  }
  hipError_t e = bf16 ? by_width<uint16_t, RouteLaunch>(E, &a, blocks, plan.threads, stream)
                      : by_width<uint32_t, RouteLaunch>(E, &a, blocks, plan.threads, stream);
  if (e != hipSuccess || blocks == 1) return e;
  if (E <= 32) route_finish_kernel<32><<<1, kFinishThreads, 0, stream>>>(a, blocks, terms);
  else if (E <= 64) route_finish_kernel<64><<<1, kFinishThreads, 0, stream>>>(a, blocks, terms);
  else route_finish_kernel<16><<<(E + 15) / 16, kFinishThreads, 0, stream>>>(a, blocks, terms);
  return hipGetLastError();
}

hipError_t launch_route_backward(const void *logits, bool bf16, int64_t T, int32_t E, int32_t k,
                                 bool renorm, float coef, const int32_t *ids, const float *weights,
                                 const int32_t *counts, const int32_t *rows, const float *dw,
                                 const float *dloss, void *dlogits, hipStream_t stream) {
  RouteBackArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.renorm = renorm;
  a.coef = coef;
  a.ids = ids;
  a.weights = weights;
  a.counts = counts;
  a.rows = rows;
  a.dw = dw;
  a.dloss = dloss;
  a.dlogits = dlogits;
  const int64_t per = route_rows_per_wave(E) * kBackWaves;
  const int64_t need = (T + per - 1) / per;
  const int blocks = (int)(need < kBackMaxBlocks ? need : kBackMaxBlocks);
  return bf16 ? by_width<uint16_t, RouteBackLaunch>(E, &a, blocks, stream)
              : by_width<uint32_t, RouteBackLaunch>(E, &a, blocks, stream);
}

// ---------------------------------------------------------------------------
// Rows by group: a stable counting sort of R group numbers.
//
// A wave holds a run of up to 16 x 64 consecutive rows, a register per 64.
// Lanes with equal keys find each other with one ballot per key bit; the first
// of them takes as many places from the wave's counter of that group (in LDS)
// as there are lanes, which gives every row its place in its group within the
// run, and leaves the run's counts.  Added up over waves, workgroups and
// groups they give each run's first place.  Rows with a number outside [0, G)
// count as group G: they are listed last and have position -1.  All sums are
// integers, so the order never varies.
//
// Up to 2048 rows one workgroup does all of it.  Beyond, the workgroups' counts
// come first (group_count_kernel), past 16 workgroups their sums over workgroups,
// a wave per group (group_scan_kernel), then the places: two or three launches,
// each of them bound by latency at these sizes.  Measured: 128 rows of 256 groups
// 3.7 us; 8192 of 9 4.0 + 4.4 us; 1M of 256 4.0 + 2.8 + 10.4 us (17 MB; the places:
// ballots, scans and writes one after another in one workgroup per compute unit).
constexpr int kGroupThreads = 1024;
constexpr int kGroupWaves = kGroupThreads / 64;
constexpr int64_t kGroupOneBlock = 2048;

__device__ __forceinline__ int group_key(int id, int G) { return (unsigned)id < (unsigned)G ? id : G; }

// part[g][b] = rows of group g in workgroup b's rows.
__global__ __launch_bounds__(kGroupThreads) void group_count_kernel(
    const int32_t *__restrict__ ids, int64_t R, int G, int64_t per_block,
    int32_t *__restrict__ part) {
  extern __shared__ int hist[];
  for (int g = threadIdx.x; g <= G; g += kGroupThreads) hist[g] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * per_block;
  const int64_t hi = lo + per_block < R ? lo + per_block : R;
#pragma unroll 4
  for (int64_t i = lo + threadIdx.x; i < hi; i += kGroupThreads)
    atomicAdd(&hist[group_key(ids[i], G)], 1);
  __syncthreads();
  for (int g = threadIdx.x; g <= G; g += kGroupThreads) part[(int64_t)g * gridDim.x + blockIdx.x] = hist[g];
}

__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    v += lane >= d ? o : 0;
  }
  return v;
}

// part[g][b] becomes the rows of group g before workgroup b, total[g] all of
// them; a wave per group, 256 workgroups a step.
constexpr int kScanThreads = 256;

__global__ __launch_bounds__(kScanThreads) void group_scan_kernel(int32_t *__restrict__ part,
                                                                  int blocks, int G1,
                                                                  int32_t *__restrict__ total) {
  const int lane = threadIdx.x & 63;
  const int g = blockIdx.x * (kScanThreads / 64) + (threadIdx.x >> 6);
  if (g >= G1) return;
  int32_t *row = part + (int64_t)g * blocks;
  int before = 0;
  for (int b0 = 0; b0 < blocks; b0 += 256) {
    int c[4], sum = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int b = b0 + lane * 4 + q;
      c[q] = b < blocks ? row[b] : 0;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sum += c[q];
    const int scan = wave_scan(sum, lane);
    int at = before + scan - sum;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int b = b0 + lane * 4 + q;
      if (b < blocks) row[b] = at;
      at += c[q];
    }
    before += __builtin_amdgcn_readlane(scan, 63);
  }
  if (lane == 0) total[g] = before;
}

// Several workgroups: `part` holds their counts by group, summed over workgroups
// by group_scan_kernel (SCANNED), or, up to kDirectBlocks of them, added up here.
constexpr int kDirectBlocks = 16;

template <int STEPS, bool SCANNED>
__global__ __launch_bounds__(kGroupThreads) void group_place_kernel(
    const int32_t *__restrict__ ids, int64_t R, int G, const int32_t *__restrict__ part,
    const int32_t *__restrict__ total, int32_t *__restrict__ order,
    int32_t *__restrict__ positions, int32_t *__restrict__ offsets) {
  extern __shared__ int sort_lds[];
  __shared__ int wave_total[2][kGroupWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int G1 = G + 1;
  int *hist = sort_lds;                         // [waves][G + 1]
  int *shift = sort_lds + kGroupWaves * G1;          // [G + 1]: place in order less place in the workgroup
  uint32_t *sorted = reinterpret_cast<uint32_t *>(shift + G1);   // [rows]: key, row
  const bool one = gridDim.x == 1;
  const int64_t base = (int64_t)blockIdx.x * (kGroupThreads * STEPS);
  const int64_t lo = base + wave * (STEPS * 64);
  int key[STEPS], place[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t i = lo + s * 64 + lane;
    key[s] = i < R ? group_key(ids[i], G) : -1;
  }
  // groups 2 tid and 2 tid + 1: rows in all workgroups, and in earlier ones
  int all[2] = {0, 0}, before[2] = {0, 0};
  if (!one) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int g = 2 * tid + q;
      if (g >= G1) continue;
      const int32_t *row = part + (int64_t)g * gridDim.x;
      if constexpr (SCANNED) {
        all[q] = total[g];
        before[q] = row[blockIdx.x];
      } else {
#pragma unroll
        for (int b = 0; b < kDirectBlocks; ++b) {
          const int c = b < (int)gridDim.x ? row[b] : 0;
          all[q] += c;
          before[q] += b < (int)blockIdx.x ? c : 0;
        }
      }
    }
  }
  for (int i = tid; i < kGroupWaves * G1; i += kGroupThreads) hist[i] = 0;
  __syncthreads();
  int *mine = hist + wave * G1;
  const int bits = 32 - __clz(G);   // keys 0 .. G
  const uint64_t lower = (1ull << lane) - 1;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const bool in = key[s] >= 0;
    uint64_t same = __builtin_amdgcn_ballot_w64(in);
    for (int b = 0; b < bits; ++b) {
      const bool set = (key[s] >> b) & 1;
      const uint64_t m = __builtin_amdgcn_ballot_w64(set);
      same &= set ? m : ~m;
    }
    const int leader = in ? __builtin_ctzll(same) : lane;
    int at = 0;
    if (in && lane == leader) at = atomicAdd(&mine[key[s]], (int)__popcll(same));
    place[s] = __shfl(at, leader) + (int)__popcll(same & lower);
  }
  __syncthreads();
  // the groups' first places: in the workgroup's rows (here) and in all rows
  int here[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int g = 2 * tid + q;
    if (g >= G1) continue;
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) here[q] += hist[w * G1 + g];
    if (one) all[q] = here[q];
  }
  const int scan = wave_scan(all[0] + all[1], lane);
  const int scan_here = one ? scan : wave_scan(here[0] + here[1], lane);
  if (lane == 63) {
    wave_total[0][wave] = scan;
    wave_total[1][wave] = scan_here;
  }
  __syncthreads();
  int first = scan - all[0] - all[1], first_here = scan_here - here[0] - here[1];
  for (int w = 0; w < wave; ++w) {
    first += wave_total[0][w];
    first_here += wave_total[1][w];
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int g = 2 * tid + q;
    if (g >= G1) continue;
    if (blockIdx.x == 0) offsets[g] = first;
    shift[g] = first + before[q] - first_here;
    int at = first_here;
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) {
      const int c = hist[w * G1 + g];
      hist[w * G1 + g] = at;
      at += c;
    }
    first += all[q];
    first_here += here[q];
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    if (key[s] < 0) continue;
    const int64_t i = lo + s * 64 + lane;
    const int at = mine[key[s]] + place[s];
    positions[i] = key[s] < G ? at + shift[key[s]] : -1;
    if (one) order[at] = (int)i;
    else sorted[at] = ((uint32_t)key[s] << 16) | (uint32_t)(i - base);
  }
  if (one) return;
  // the workgroup's rows in order, so that a group's run is written as a run
  __syncthreads();
  const int rows = (int)(base + kGroupThreads * STEPS < R ? kGroupThreads * STEPS : R - base);
  for (int i = tid; i < rows; i += kGroupThreads) {
    const uint32_t v = sorted[i];
    order[i + shift[v >> 16]] = (int)(base + (v & 0xffff));
  }
}

namespace {

// Steps of 64 rows a wave.  Up to 2048 rows one workgroup does all; up to 16
// workgroups of 1024 rows their counts are a launch of their own and each adds
// them up.  Both sides, a call among others in a graph, one workgroup and so:
// 3000 rows 6.0 and 6.3 us of 9 groups, 8.0 and 7.4 of 256; 8192 rows 9.4 and 7.0,
// 13.2 and 8.6; 15000 rows 14.8 and 7.1, 21.4 and 8.5.  Beyond, three launches: 4
// steps (256 workgroups at 1M rows, one per compute unit), 16 past that.
int group_steps(int64_t R) {
  if (R <= kGroupOneBlock) return R <= kGroupThreads ? 1 : 2;
  if (R <= (int64_t)kDirectBlocks * kGroupThreads) return 1;
  return R <= (int64_t)256 * 4 * kGroupThreads ? 4 : 16;
}

int64_t group_blocks(int64_t R) {
  const int64_t per = (int64_t)group_steps(R) * kGroupThreads;
  return R > 0 ? (R + per - 1) / per : 1;
}

}  // namespace

size_t group_workspace_bytes(int64_t R, int32_t G) {
  if (R <= kGroupOneBlock) return 0;
  return sizeof(int32_t) * (size_t)(group_blocks(R) + 1) * (G + 1);
}

hipError_t launch_group_rows(const int32_t *ids, int64_t R, int32_t G, int32_t *order,
                             int32_t *positions, int32_t *offsets, void *work,
                             hipStream_t stream) {
  const int steps = group_steps(R);
  const int blocks = (int)group_blocks(R);
  int32_t *total = static_cast<int32_t *>(work);
  int32_t *part = blocks > 1 ? total + G + 1 : nullptr;
  if (blocks > 1) {
    group_count_kernel<<<blocks, kGroupThreads, sizeof(int) * (G + 1), stream>>>(
        ids, R, G, (int64_t)steps * kGroupThreads, part);
    if (hipError_t e = hipGetLastError()) return e;
    if (steps >= 4) {
      constexpr int per = kScanThreads / 64;
      group_scan_kernel<<<(G + per) / per, kScanThreads, 0, stream>>>(part, blocks, G + 1, total);
      if (hipError_t e = hipGetLastError()) return e;
    }
  }
  const size_t lds = sizeof(int) * ((size_t)(kGroupWaves + 1) * (G + 1) +
                                    (blocks > 1 ? (size_t)steps * kGroupThreads : 0));
#define FP8BLK_PLACE(S, SCANNED)                                                        \
  group_place_kernel<S, SCANNED><<<blocks, kGroupThreads, lds, stream>>>(               \
      ids, R, G, part, total, order, positions, offsets)
  if (steps == 1) FP8BLK_PLACE(1, false);
  else if (steps == 2) FP8BLK_PLACE(2, false);
  else if (steps == 4) FP8BLK_PLACE(4, true);
  else FP8BLK_PLACE(16, true);
#undef FP8BLK_PLACE
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Combine: out[t] = base[t] + sum_j w[t,j] * y[pos[t,j]], fp32 sums in the
// order of j, one rounding to bf16.  Slots whose position is outside [0, R)
// add nothing, and their rows of y are not read.
//
// HBM-bound (k + 1 rows of N read or written per token).  A wave takes 512
// columns of one token, 8 per lane, so positions and weights are scalar loads
// and the k row loads of a lane are independent 16-byte loads.  Rows may start
// at any even address (odd N): gfx950's global loads take those at 16 bytes
// a lane too, and the last N % 8 columns go one by one.  All of it is touched
// once, so loads and stores are non-temporal (4096 tokens of 8 rows, N = 7168:
// 134 -> 96 us, 6.1 TB/s).
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));

namespace {

// Up to 8 bf16 at columns [c, c + 8) of a row of N, as fp32; 0 past N.
template <bool NT = true>
__device__ __forceinline__ void load8(const uint16_t *row, int64_t c, int64_t N, float *f) {
  if (c + 8 <= N) {
    v4u_any w;
    if constexpr (NT) w = __builtin_nontemporal_load(reinterpret_cast<const v4u_any *>(row + c));
    else w = *reinterpret_cast<const v4u_any *>(row + c);
    unpack8(make_uint4(w[0], w[1], w[2], w[3]), f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < N ? bf16_lo(row[c + i]) : 0.0f;
  }
}

template <bool NT = true>
__device__ __forceinline__ void store8(uint16_t *row, int64_t c, int64_t N, const float *f) {
  if (c + 8 <= N) {
    v4u_any w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<v4u_any *>(row + c));
    else *reinterpret_cast<v4u_any *>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < N) row[c + i] = to_bf16(f[i]);
  }
}

}  // namespace

constexpr int kCombineThreads = 256;
constexpr int kCombineCols = 512;   // columns of a wave
// Workgroups of one launch: a grid of 2^32 threads or more is not refused but
// wraps, so larger batches take several launches.
constexpr int64_t kCombineBlocks = int64_t(1) << 23;

__global__ __launch_bounds__(kCombineThreads) void combine_kernel(
    const uint16_t *__restrict__ y, int64_t R, const float *__restrict__ weights,
    const int32_t *__restrict__ positions, const uint16_t *base, int64_t T, int k, int64_t N,
    uint16_t *out,   // may be base: each lane reads its columns first
    int64_t block0) {
  const int lane = threadIdx.x & 63;
  const int64_t chunks = (N + kCombineCols - 1) / kCombineCols;
  const int64_t unit = (block0 + blockIdx.x) * (kCombineThreads / 64) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = unit / chunks;
  if (t >= T) return;
  const int64_t c = (unit - t * chunks) * kCombineCols + lane * 8;
  if (c >= N) return;
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (base) load8(base + t * N, c, N, acc);
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int p = positions[t * k + j];
    if (p < 0 || p >= R) continue;
    const float w = weights[t * k + j];
    float f[8];
    load8(y + (int64_t)p * N, c, N, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
  }
  store8(out + t * N, c, N, acc);
}

hipError_t launch_combine(const void *y, int64_t R, const float *weights, const int32_t *positions,
                          const void *base, int64_t T, int32_t k, int64_t N, void *out,
                          hipStream_t stream) {
  const int64_t units = T * ((N + kCombineCols - 1) / kCombineCols);
  const int64_t per = kCombineThreads / 64, blocks = (units + per - 1) / per;
  for (int64_t b = 0; b < blocks; b += kCombineBlocks) {
    const int64_t n = blocks - b < kCombineBlocks ? blocks - b : kCombineBlocks;
    combine_kernel<<<(unsigned)n, kCombineThreads, 0, stream>>>(
        static_cast<const uint16_t *>(y), R, weights, positions,
        static_cast<const uint16_t *>(base), T, k, N, static_cast<uint16_t *>(out), b);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

// Combine, backward: dy[pos] = bf16(w * d), dw = <d, y[pos]> (fp32, a fixed
// order), one workgroup per token; each column of d is read once per 8 slots
// and stays in registers while the slots' rows stream past.  Rows of dy past
// the last used one (n_used, in device memory) are zeroed.  Dropped slots get
// dw = 0.  A row below n_used that no slot names is not written, and one that two
// slots name gets either's gradient.  d_y is stored through the caches:
// non-temporal stores beside the non-temporal loads measured slower (203 against
// 191 us at 4096 tokens of 8 rows, N = 7168: 1.0 GB, 5.2 TB/s; 212 us in the
// kernel trace).
__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(
    const uint16_t *__restrict__ d_out, const uint16_t *__restrict__ y, int64_t R,
    const float *__restrict__ weights, const int32_t *__restrict__ positions,
    const int32_t *__restrict__ n_used, int64_t T, int k, int64_t N, uint16_t *__restrict__ dy,
    float *__restrict__ dw, int64_t t0) {
  constexpr int J = 8;
  __shared__ float sums[kCombineThreads / 64][J];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t = t0 + blockIdx.x;
  if (t < T) {
    for (int j0 = 0; j0 < k; j0 += J) {
      float acc[J];
#pragma unroll
      for (int j = 0; j < J; ++j) acc[j] = 0.0f;
      for (int64_t c = tid * 8; c < N; c += kCombineThreads * 8) {
        float d[8];
        load8(d_out + t * N, c, N, d);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j0 + j >= k) continue;
          const int p = positions[t * k + j0 + j];
          if (p < 0 || p >= R) continue;
          const float w = weights[t * k + j0 + j];
          float f[8];
          load8(y + (int64_t)p * N, c, N, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[j] = fmaf(d[i], f[i], acc[j]);
            f[i] = w * d[i];
          }
          store8<false>(dy + (int64_t)p * N, c, N, f);
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        acc[j] = row_sum<64>(acc[j]);
        if (lane == 0) sums[wave][j] = acc[j];
      }
      __syncthreads();
      if (tid < J && j0 + tid < k) {
        float s = 0.0f;
        for (int w = 0; w < kCombineThreads / 64; ++w) s += sums[w][tid];
        dw[t * k + j0 + tid] = s;
      }
      __syncthreads();
    }
  }
  if (t0) return;   // the first launch zeroes the rows past the used ones
  const int64_t used = max(*n_used, 0);
  const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t p = used + blockIdx.x; p < R; p += gridDim.x)
    for (int64_t c = tid * 8; c < N; c += kCombineThreads * 8) store8<false>(dy + p * N, c, N, zero);
}

hipError_t launch_combine_backward(const void *d_out, const void *y, int64_t R,
                                   const float *weights, const int32_t *positions,
                                   const int32_t *n_used, int64_t T, int32_t k, int64_t N,
                                   void *dy, float *dw, hipStream_t stream) {
  const int64_t blocks = T > 0 ? T : (R < 1024 ? R : 1024);
  for (int64_t t = 0; t < blocks; t += kCombineBlocks) {
    const int64_t n = blocks - t < kCombineBlocks ? blocks - t : kCombineBlocks;
    combine_backward_kernel<<<(unsigned)n, kCombineThreads, 0, stream>>>(
        static_cast<const uint16_t *>(d_out), static_cast<const uint16_t *>(y), R, weights,
        positions, n_used, T, k, N, static_cast<uint16_t *>(dy), dw, t);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace fp8blk
