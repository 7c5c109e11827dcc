// C ABI of fp8blk: argument validation (before any HIP runtime call), the
// gfx950 device check, and dispatch to the kernels.  Declared in fp8blk.h.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>
#include <initializer_list>

#include "../../include/fp8blk.h"
#include "fp8blk_launch.h"

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxK = int64_t(1) << 24;
constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int kMaxDevices = 64;

// 0 = unknown, 1 = gfx950, 2 = other / unusable
std::atomic<int> g_arch_state[kMaxDevices];

bool misaligned(const void *p, uintptr_t align = 16) {
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0;
}

fp8blk_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)hipGetLastError();
    return FP8BLK_ERR_DEVICE;
  }
  int st = g_arch_state[dev].load(std::memory_order_acquire);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return FP8BLK_ERR_DEVICE;
    }
    st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_arch_state[dev].store(st, std::memory_order_release);
  }
  return st == 1 ? FP8BLK_OK : FP8BLK_ERR_DEVICE;
}

fp8blk_status launched(hipError_t e) { return e == hipSuccess ? FP8BLK_OK : FP8BLK_ERR_LAUNCH; }

// Shape rules shared by the entry points: rows in [0, 2^31), K a positive
// multiple of 128 up to 2^24, element counts up to 2^40.
bool bad_rows(int64_t r) { return r < 0 || r > kMaxRows; }
bool bad_k(int64_t K) { return K <= 0 || K > kMaxK || (K % FP8BLK_BLOCK) != 0; }
bool too_big(int64_t rows, int64_t K) { return rows > 0 && K > 0 && rows > kMaxElems / K; }

// Validation of each operation, shared by its variants.  The scale arrays'
// alignment (bytes) depends on the variant: fp32 scale arrays 16, one
// static fp32 scale 4, E8M0 byte arrays 1 (none).
fp8blk_status check_quant(const void *in, int64_t rows, int64_t K, const void *q,
                          const void *scale, uintptr_t scale_align) {
  if (rows > 0 && (!in || !q || !scale)) return FP8BLK_ERR_NULL;
  if (bad_rows(rows) || bad_k(K) || too_big(rows, K)) return FP8BLK_ERR_SHAPE;
  if (rows > 0 && (misaligned(in) || misaligned(q) || misaligned(scale, scale_align)))
    return FP8BLK_ERR_ALIGN;
  return check_device();
}

// `work`: a workspace that the call will use (checked for 16-byte alignment
// with the other pointers), or NULL.
fp8blk_status check_gemm(const void *x_q, const void *x_scale, const void *w_q,
                         const void *w_scale, int64_t M, int64_t N, int64_t K, const void *y,
                         uintptr_t xs_align, uintptr_t ws_align, const void *work_buf = nullptr) {
  const bool work = M > 0 && N > 0;
  if (work && (!x_q || !x_scale || !w_q || !w_scale || !y)) return FP8BLK_ERR_NULL;
  if (bad_rows(M) || bad_rows(N) || bad_k(K) || too_big(M, K) || too_big(N, K) ||
      too_big(M, N))
    return FP8BLK_ERR_SHAPE;
  if (work && ((M + 127) / 128) * ((N + 127) / 128) > kMaxRows) return FP8BLK_ERR_SHAPE;
  if (work && (misaligned(x_q) || misaligned(w_q) || misaligned(y) ||
               misaligned(x_scale, xs_align) || misaligned(w_scale, ws_align) ||
               (work_buf && misaligned(work_buf))))
    return FP8BLK_ERR_ALIGN;
  return check_device();
}

fp8blk_status check_grouped(const void *x_q, const void *x_scale, const void *w_q,
                            const void *w_scale, const int32_t *offsets, int32_t E,
                            int64_t total_M, int64_t N, int64_t K, const void *y,
                            uintptr_t scale_align) {
  const bool work = E > 0 && total_M > 0 && N > 0;
  if (work && (!x_q || !x_scale || !w_q || !w_scale || !offsets || !y)) return FP8BLK_ERR_NULL;
  if (E < 0 || bad_rows(total_M) || bad_rows(N) || bad_k(K) || too_big(total_M, K) ||
      too_big(total_M, N) || (E > 0 && too_big(int64_t(E) * N, K)) || too_big(int64_t(E), N))
    return FP8BLK_ERR_SHAPE;
  if (work && ((total_M + 127) / 128 + E) * ((N + 127) / 128) > kMaxRows) return FP8BLK_ERR_SHAPE;
  if (work && (misaligned(x_q) || misaligned(w_q) || misaligned(y) ||
               misaligned(x_scale, scale_align) || misaligned(w_scale, scale_align)))
    return FP8BLK_ERR_ALIGN;
  return check_device();
}

fp8blk_status check_swiglu(const void *gate_up_bf16, int64_t M, int64_t I, const void *x_q,
                           const void *x_scale, uintptr_t scale_align) {
  if (M > 0 && (!gate_up_bf16 || !x_q || !x_scale)) return FP8BLK_ERR_NULL;
  if (bad_rows(M) || bad_k(I) || too_big(M, 2 * I) || M * (I / FP8BLK_BLOCK) > kMaxRows)
    return FP8BLK_ERR_SHAPE;
  if (M > 0 && (misaligned(gate_up_bf16) || misaligned(x_q) || misaligned(x_scale, scale_align)))
    return FP8BLK_ERR_ALIGN;
  return check_device();
}

}  // namespace

extern "C" {

const char *fp8blk_status_string(int s) {
  switch (s) {
    case FP8BLK_OK: return "FP8BLK_OK";
    case FP8BLK_ERR_NULL: return "FP8BLK_ERR_NULL: a required pointer is NULL";
    case FP8BLK_ERR_SHAPE: return "FP8BLK_ERR_SHAPE: bad size (negative, K not a positive multiple of 128, or over the limits)";
    case FP8BLK_ERR_ALIGN: return "FP8BLK_ERR_ALIGN: a base pointer is not 16-byte aligned";
    case FP8BLK_ERR_DEVICE: return "FP8BLK_ERR_DEVICE: no usable device, or the current device is not gfx950";
    case FP8BLK_ERR_LAUNCH: return "FP8BLK_ERR_LAUNCH: kernel launch failed";
    case FP8BLK_ERR_SCRATCH: return "FP8BLK_ERR_SCRATCH: the call needs more device scratch than the library holds (FP8BLK_SCRATCH_BYTES)";
    default: return "FP8BLK_ERR_UNKNOWN";
  }
}

int fp8blk_abi_version(void) { return FP8BLK_ABI_VERSION; }

fp8blk_status fp8_weight_block_quant(const void *w_bf16, int64_t N, int64_t K, void *w_q,
                                     float *w_scale, void *stream) {
  if (fp8blk_status c = check_quant(w_bf16, N, K, w_q, w_scale, 16)) return c;
  if (N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_weight_quant(w_bf16, N, K, w_q, w_scale,
                                              static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_act_quant_group(const void *x_bf16, int64_t M, int64_t K, void *x_q,
                                  float *x_scale, void *stream) {
  if (fp8blk_status c = check_quant(x_bf16, M, K, x_q, x_scale, 16)) return c;
  if (M == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_act_quant(x_bf16, M, K, x_q, x_scale,
                                           static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_block_gemm(const void *x_q, const float *x_scale, const void *w_q,
                             const float *w_scale, int64_t M, int64_t N, int64_t K, void *y_bf16,
                             void *stream) {
  if (fp8blk_status c = check_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, 16, 16)) return c;
  if (M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_block_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16,
                                            static_cast<hipStream_t>(stream)));
}

size_t fp8_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (bad_rows(M) || bad_rows(N) || bad_k(K) || too_big(M, K) || too_big(N, K) || too_big(M, N))
    return 0;
  return fp8blk::block_gemm_workspace_bytes(M, N, K);
}

fp8blk_status fp8_block_gemm_ws(const void *x_q, const float *x_scale, const void *w_q,
                                const float *w_scale, int64_t M, int64_t N, int64_t K,
                                void *y_bf16, void *workspace, size_t workspace_bytes,
                                void *stream) {
  // whether the workspace will be used (known before validation so that its
  // alignment is checked with the other pointers; check_gemm still rejects
  // bad sizes before anything runs)
  const size_t need = fp8blk::block_gemm_workspace_bytes(M, N, K);
  const bool use = need > 0 && workspace != nullptr && workspace_bytes >= need;
  if (fp8blk_status c = check_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, 16, 16,
                                   use ? workspace : nullptr))
    return c;
  if (M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_block_gemm_ws(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16,
                                               use ? workspace : nullptr, use ? workspace_bytes : 0,
                                               static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_grouped_block_gemm(const void *x_q, const float *x_scale, const void *w_q,
                                     const float *w_scale, const int32_t *expert_offsets,
                                     int32_t E, int64_t total_M, int64_t N, int64_t K,
                                     void *y_bf16, void *stream) {
  if (fp8blk_status c = check_grouped(x_q, x_scale, w_q, w_scale, expert_offsets, E, total_M, N,
                                      K, y_bf16, 16))
    return c;
  if (E == 0 || total_M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_grouped_gemm(x_q, x_scale, w_q, w_scale, expert_offsets, E,
                                              total_M, N, K, y_bf16,
                                              static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_act_quant_static(const void *x_bf16, int64_t M, int64_t K,
                                   const float *x_scale, void *x_q, void *stream) {
  if (fp8blk_status c = check_quant(x_bf16, M, K, x_q, x_scale, 4)) return c;
  if (M == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_act_quant_static(x_bf16, M, K, x_scale, x_q,
                                                  static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_block_gemm_static(const void *x_q, const float *x_scale, const void *w_q,
                                    const float *w_scale, int64_t M, int64_t N, int64_t K,
                                    void *y_bf16, void *stream) {
  if (fp8blk_status c = check_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, 4, 16)) return c;
  if (M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_block_gemm_static(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16,
                                                   static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_block_gemm_noalloc(const void *x_q, const float *x_scale, const void *w_q,
                                     const float *w_scale, int64_t M, int64_t N, int64_t K,
                                     void *y_bf16, void *stream) {
  static_assert(fp8blk::kScratchBytes == FP8BLK_SCRATCH_BYTES, "scratch size out of step");
  if (fp8blk_status c = check_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, 16, 16)) return c;
  if (M == 0 || N == 0) return FP8BLK_OK;
  if (fp8blk::block_gemm_split_workspace_bytes(M, N, K) > fp8blk::kScratchBytes)
    return FP8BLK_ERR_SCRATCH;
  return launched(fp8blk::launch_block_gemm_noalloc(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16,
                                                    static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_linear(const void *x_bf16, int64_t M, int64_t N, int64_t K, const void *w_q,
                         const float *w_scale, void *x_q_ws, float *x_scale_ws, void *y_bf16,
                         void *stream) {
  // The fused decode kernel re-quantizes x in every workgroup (each reads
  // all of x in bf16 from L2), once per K block for all the workgroup's
  // 16-column slabs.  With workspaces at hand it runs only where it beats
  // the two kernels: at M <= 16 for small weights (the second launch costs
  // more) and for K <= 8192 when the launcher packs two or more slabs per
  // workgroup; at M = 17-32 for weights of at most 2^24 elements; never
  // past M = 32.  Measured, weights streamed from HBM (fused against two
  // kernels), M = 16: 4096x4096 10.1 us / 19.4; 14336x4096 (4 slabs) 15.9 /
  // 19.5; 24576x1536 (2 slabs) 16.5 / 19.5; 4096x14336 (1 slab) 26.7 /
  // 21.1; 7168x16384 (2 slabs) 38.4 / 33.5; 18432x7168 (1 slab) 66.4 /
  // 47.2.  M = 17-32: 4096x4096 13.4-14.4 / 19.3-19.6; 1024x4096 11.4-12.6
  // / 19.1; 1536x7168 17.6-20.2 / 18.9-19.0; 14336x4096 27-31 / 23-24.
  // M = 33-64: 4096x4096 24.2-25.1 / 19.6-19.7; 1024x4096 21.1-23.1 /
  // 19.2-19.3; 1536x7168 35.7-39.1 / 19.3-25.7.
  constexpr int64_t kFusedMaxM = 64;
  constexpr int64_t kFusedMaxWeight = int64_t(1) << 25;     // N * K elements, M <= 16
  constexpr int64_t kFusedMaxWeight32 = int64_t(1) << 24;   // N * K elements, M <= 32
  constexpr int64_t kFusedSlabsMaxK = 8192;
  const bool work = M > 0 && N > 0;
  const bool have_ws = x_q_ws != nullptr && x_scale_ws != nullptr;
  // (N * K only for sizes within the limits, which keep it below 2^55;
  // others are refused below)
  const bool sized = !bad_rows(N) && !bad_k(K);
  const bool fused =
      M <= kFusedMaxM &&
      (!have_ws || !sized ||
       (M <= 16 && (N * K <= kFusedMaxWeight ||
                    (K <= kFusedSlabsMaxK && fp8blk::linear_decode_slabs(M, N) >= 2))) ||
       (M <= 32 && N * K <= kFusedMaxWeight32));
  if (work && (!x_bf16 || !w_q || !w_scale || !y_bf16 || (!fused && (!x_q_ws || !x_scale_ws))))
    return FP8BLK_ERR_NULL;
  if (bad_rows(M) || bad_rows(N) || bad_k(K) || too_big(M, K) || too_big(N, K) || too_big(M, N))
    return FP8BLK_ERR_SHAPE;
  if (work && ((M + 127) / 128) * ((N + 127) / 128) > kMaxRows) return FP8BLK_ERR_SHAPE;
  if (work && (misaligned(x_bf16) || misaligned(w_q) || misaligned(w_scale) ||
               misaligned(y_bf16) || (!fused && (misaligned(x_q_ws) || misaligned(x_scale_ws)))))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (!work) return FP8BLK_OK;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (fused) return launched(fp8blk::launch_linear_decode(x_bf16, w_q, w_scale, M, N, K, y_bf16, st));
  if (fp8blk_status e = launched(fp8blk::launch_act_quant(x_bf16, M, K, x_q_ws, x_scale_ws, st)))
    return e;
  return launched(fp8blk::launch_block_gemm(x_q_ws, x_scale_ws, w_q, w_scale, M, N, K, y_bf16, st));
}

fp8blk_status fp8_batched_block_gemm(const void *x_q, const float *x_scale, const void *w_q,
                                     const float *w_scale, const int32_t *expert_counts,
                                     int32_t E, int64_t capacity, int64_t N, int64_t K,
                                     void *y_bf16, void *stream) {
  const bool work = E > 0 && capacity > 0 && N > 0;
  if (work && (!x_q || !x_scale || !w_q || !w_scale || !expert_counts || !y_bf16))
    return FP8BLK_ERR_NULL;
  if (E < 0 || capacity < 0 || bad_rows(N) || bad_k(K) || (E > 0 && capacity > kMaxRows / E))
    return FP8BLK_ERR_SHAPE;
  const int64_t total = int64_t(E) * capacity;
  if (too_big(total, K) || too_big(total, N) || (E > 0 && too_big(int64_t(E) * N, K)) ||
      too_big(int64_t(E), N))
    return FP8BLK_ERR_SHAPE;
  if (work && int64_t(E) * ((capacity + 127) / 128) * ((N + 127) / 128) > kMaxRows)
    return FP8BLK_ERR_SHAPE;
  if (work && (misaligned(x_q) || misaligned(x_scale) || misaligned(w_q) || misaligned(w_scale) ||
               misaligned(y_bf16) || misaligned(expert_counts, 4)))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (!work) return FP8BLK_OK;
  return launched(fp8blk::launch_batched_gemm(x_q, x_scale, w_q, w_scale, expert_counts, E,
                                              capacity, N, K, y_bf16,
                                              static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_rowwise_quant(const void *in_bf16, int64_t R, int64_t K, void *q,
                                float *scale, void *stream) {
  if (fp8blk_status c = check_quant(in_bf16, R, K, q, scale, 16)) return c;
  if (R == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_rowwise_quant(in_bf16, R, K, q, scale,
                                               static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_rowwise_gemm(const void *x_q, const float *x_scale, const void *w_q,
                               const float *w_scale, int64_t M, int64_t N, int64_t K,
                               void *y_bf16, void *stream) {
  if (fp8blk_status c = check_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, 16, 16)) return c;
  if (M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_rowwise_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16,
                                              static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_swiglu_act_quant(const void *gate_up_bf16, int64_t M, int64_t I, void *x_q,
                                   float *x_scale, void *stream) {
  if (fp8blk_status c = check_swiglu(gate_up_bf16, M, I, x_q, x_scale, 16)) return c;
  if (M == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_swiglu_act_quant(gate_up_bf16, M, I, x_q, x_scale,
                                                  static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_swiglu_act_quant_ue8m0(const void *gate_up_bf16, int64_t M, int64_t I,
                                         void *x_q, uint8_t *x_scale, void *stream) {
  if (fp8blk_status c = check_swiglu(gate_up_bf16, M, I, x_q, x_scale, 1)) return c;
  if (M == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_swiglu_act_quant_e8m0(gate_up_bf16, M, I, x_q, x_scale,
                                                       static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_weight_block_quant_ue8m0(const void *w_bf16, int64_t N, int64_t K, void *w_q,
                                           uint8_t *w_scale, void *stream) {
  if (fp8blk_status c = check_quant(w_bf16, N, K, w_q, w_scale, 1)) return c;
  if (N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_weight_quant_e8m0(w_bf16, N, K, w_q, w_scale,
                                                   static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_act_quant_group_ue8m0(const void *x_bf16, int64_t M, int64_t K, void *x_q,
                                        uint8_t *x_scale, void *stream) {
  if (fp8blk_status c = check_quant(x_bf16, M, K, x_q, x_scale, 1)) return c;
  if (M == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_act_quant_e8m0(x_bf16, M, K, x_q, x_scale,
                                                static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_block_gemm_ue8m0(const void *x_q, const uint8_t *x_scale, const void *w_q,
                                   const uint8_t *w_scale, int64_t M, int64_t N, int64_t K,
                                   void *y_bf16, void *stream) {
  if (fp8blk_status c = check_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, 1, 1)) return c;
  if (M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_block_gemm_e8m0(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16,
                                                 static_cast<hipStream_t>(stream)));
}

size_t fp8_block_gemm_ue8m0_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (bad_rows(M) || bad_rows(N) || bad_k(K) || too_big(M, K) || too_big(N, K) || too_big(M, N))
    return 0;
  return fp8blk::block_gemm_e8m0_workspace_bytes(M, N, K);
}

fp8blk_status fp8_block_gemm_ue8m0_ws(const void *x_q, const uint8_t *x_scale, const void *w_q,
                                      const uint8_t *w_scale, int64_t M, int64_t N, int64_t K,
                                      void *y_bf16, void *workspace, size_t workspace_bytes,
                                      void *stream) {
  // as fp8_block_gemm_ws
  const size_t need = fp8blk::block_gemm_e8m0_workspace_bytes(M, N, K);
  const bool use = need > 0 && workspace != nullptr && workspace_bytes >= need;
  if (fp8blk_status c = check_gemm(x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, 1, 1,
                                   use ? workspace : nullptr))
    return c;
  if (M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_block_gemm_e8m0_ws(
      x_q, x_scale, w_q, w_scale, M, N, K, y_bf16, use ? workspace : nullptr,
      use ? workspace_bytes : 0, static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8_grouped_block_gemm_ue8m0(const void *x_q, const uint8_t *x_scale,
                                           const void *w_q, const uint8_t *w_scale,
                                           const int32_t *expert_offsets, int32_t E,
                                           int64_t total_M, int64_t N, int64_t K, void *y_bf16,
                                           void *stream) {
  if (fp8blk_status c = check_grouped(x_q, x_scale, w_q, w_scale, expert_offsets, E, total_M, N,
                                      K, y_bf16, 1))
    return c;
  if (E == 0 || total_M == 0 || N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_grouped_gemm_e8m0(x_q, x_scale, w_q, w_scale, expert_offsets, E,
                                                   total_M, N, K, y_bf16,
                                                   static_cast<hipStream_t>(stream)));
}

// ---- routing, rows by group, combine, adapters ---------------------------

namespace {

bool bad_groups(int32_t g) { return g < 1 || g > FP8BLK_MAX_GROUPS; }
// T rows of k slots with int32 slot numbers
bool bad_slots(int64_t T, int32_t k) {
  return bad_rows(T) || k < 1 || k > FP8BLK_MAX_TOPK || T > kMaxRows / k;
}
bool bad_route(int type, int64_t T, int32_t E, int32_t k) {
  return (type != FP8BLK_F32 && type != FP8BLK_BF16) || bad_groups(E) || bad_slots(T, k) || k > E;
}
bool any_misaligned(std::initializer_list<const void *> ps, uintptr_t align) {
  for (const void *p : ps)
    if (misaligned(p, align)) return true;
  return false;
}

}  // namespace

size_t fp8blk_moe_route_workspace_bytes(int64_t T, int32_t E) {
  return bad_rows(T) || bad_groups(E) ? 0 : fp8blk::route_workspace_bytes(T, E);
}

fp8blk_status fp8blk_moe_route(const void *logits, int logits_type, const uint8_t *mask, int64_t T,
                               int32_t E, int32_t k, int renormalize, float loss_coef,
                               int32_t *ids, float *weights, int32_t *counts, int32_t *rows,
                               float *loss, void *workspace, size_t workspace_bytes,
                               void *stream) {
  if (!counts || (T > 0 && (!logits || !ids || !weights))) return FP8BLK_ERR_NULL;
  if (bad_route(logits_type, T, E, k)) return FP8BLK_ERR_SHAPE;
  const size_t need = fp8blk::route_workspace_bytes(T, E);
  if (need > 0 && workspace == nullptr) return FP8BLK_ERR_NULL;
  if (workspace_bytes < need) return FP8BLK_ERR_SHAPE;
  if ((T > 0 && misaligned(logits)) || (need > 0 && misaligned(workspace)) ||
      any_misaligned({ids, weights, counts, rows, loss}, 4))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  return launched(fp8blk::launch_route(logits, logits_type == FP8BLK_BF16, mask, T, E, k,
                                       renormalize != 0, loss_coef, ids, weights, counts, rows,
                                       loss, workspace, static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8blk_moe_route_backward(const void *logits, int logits_type, int64_t T, int32_t E,
                                        int32_t k, int renormalize, float loss_coef,
                                        const int32_t *ids, const float *weights,
                                        const int32_t *counts, const int32_t *rows,
                                        const float *d_weights, const float *d_loss,
                                        void *d_logits, void *stream) {
  if (T > 0 && (!logits || !ids || !weights || !counts || !d_logits || (d_loss && !rows)))
    return FP8BLK_ERR_NULL;
  if (bad_route(logits_type, T, E, k)) return FP8BLK_ERR_SHAPE;
  if (T > 0 && (any_misaligned({logits, d_logits}, 16) ||
                any_misaligned({ids, weights, counts, rows, d_weights, d_loss}, 4)))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (T == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_route_backward(logits, logits_type == FP8BLK_BF16, T, E, k,
                                                renormalize != 0, loss_coef, ids, weights, counts,
                                                rows, d_weights, d_loss, d_logits,
                                                static_cast<hipStream_t>(stream)));
}

size_t fp8blk_group_rows_workspace_bytes(int64_t R, int32_t G) {
  return bad_rows(R) || bad_groups(G) ? 0 : fp8blk::group_workspace_bytes(R, G);
}

fp8blk_status fp8blk_group_rows(const int32_t *ids, int64_t R, int32_t G, int32_t *order,
                                int32_t *positions, int32_t *offsets, void *workspace,
                                size_t workspace_bytes, void *stream) {
  if (!offsets || (R > 0 && (!ids || !order || !positions))) return FP8BLK_ERR_NULL;
  if (bad_rows(R) || bad_groups(G)) return FP8BLK_ERR_SHAPE;
  const size_t need = fp8blk::group_workspace_bytes(R, G);
  if (need > 0 && workspace == nullptr) return FP8BLK_ERR_NULL;
  if (workspace_bytes < need) return FP8BLK_ERR_SHAPE;
  if ((need > 0 && misaligned(workspace)) || any_misaligned({ids, order, positions, offsets}, 4))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  return launched(fp8blk::launch_group_rows(ids, R, G, order, positions, offsets, workspace,
                                            static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8blk_moe_combine(const void *y_bf16, int64_t R, const float *weights,
                                 const int32_t *positions, const void *base_bf16, int64_t T,
                                 int32_t k, int64_t N, void *out_bf16, void *stream) {
  const bool work = T > 0 && N > 0;
  if (work && ((R > 0 && !y_bf16) || !weights || !positions || !out_bf16)) return FP8BLK_ERR_NULL;
  if (bad_slots(T, k) || bad_rows(R) || bad_rows(N) || too_big(T, N) || too_big(R, N))
    return FP8BLK_ERR_SHAPE;
  if (work && (any_misaligned({y_bf16, base_bf16, out_bf16}, 16) ||
               any_misaligned({weights, positions}, 4)))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (!work) return FP8BLK_OK;
  return launched(fp8blk::launch_combine(y_bf16, R, weights, positions, base_bf16, T, k, N,
                                         out_bf16, static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8blk_moe_combine_backward(const void *d_out_bf16, const void *y_bf16, int64_t R,
                                          const float *weights, const int32_t *positions,
                                          const int32_t *rows_used, int64_t T, int32_t k,
                                          int64_t N, void *d_y_bf16, float *d_weights,
                                          void *stream) {
  const bool work = T > 0 || (R > 0 && N > 0);
  if (work && (!rows_used || (R > 0 && N > 0 && (!y_bf16 || !d_y_bf16)) ||
               (T > 0 && (!weights || !positions || !d_weights || (N > 0 && !d_out_bf16)))))
    return FP8BLK_ERR_NULL;
  if (bad_slots(T, k) || bad_rows(R) || bad_rows(N) || too_big(T, N) || too_big(R, N))
    return FP8BLK_ERR_SHAPE;
  if (work && (any_misaligned({d_out_bf16, y_bf16, d_y_bf16}, 16) ||
               any_misaligned({weights, positions, rows_used, d_weights}, 4)))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (!work) return FP8BLK_OK;
  return launched(fp8blk::launch_combine_backward(d_out_bf16, y_bf16, R, weights, positions,
                                                  rows_used, T, k, N, d_y_bf16, d_weights,
                                                  static_cast<hipStream_t>(stream)));
}

namespace {
bool bad_lora(int64_t T, int64_t K, int32_t r, int32_t L) {
  return bad_rows(T) || bad_k(K) || too_big(T, K) || r < 8 || r > FP8BLK_MAX_RANK || r % 8 != 0 ||
         bad_groups(L);
}
}  // namespace

size_t fp8blk_lora_add_workspace_bytes(int64_t T, int64_t K, int32_t r, int32_t L, int listed) {
  return T == 0 || bad_lora(T, K, r, L) ? 0
                                        : fp8blk::lora_workspace_bytes(T, K, r, L, listed != 0);
}

fp8blk_status fp8blk_lora_add(const void *base_bf16, int64_t base_stride, const void *x_bf16,
                              int64_t x_stride, const void *a_bf16, const void *b_bf16,
                              const int32_t *ids, const float *scale, const int32_t *order,
                              const int32_t *offsets, int64_t T, int64_t K, int64_t N, int32_t r,
                              int32_t L, void *out_bf16, int64_t out_stride, void *workspace,
                              size_t workspace_bytes, void *stream) {
  const bool work = T > 0 && N > 0;
  if (work && (!x_bf16 || !a_bf16 || !b_bf16 || !ids || !out_bf16 ||
               (order == nullptr) != (offsets == nullptr)))
    return FP8BLK_ERR_NULL;
  if (bad_lora(T, K, r, L) || bad_rows(N) || x_stride < K || out_stride < N ||
      too_big(T, x_stride) || too_big(T, out_stride) || too_big(int64_t(L) * r, K) ||
      too_big(int64_t(L) * r, N) ||
      (base_bf16 && (base_stride < N || too_big(T, base_stride))) ||
      (base_bf16 && base_bf16 == out_bf16 && base_stride != out_stride) ||
      !fp8blk::lora_fits(T, K, N, r, L))
    return FP8BLK_ERR_SHAPE;
  if (work && !workspace) return FP8BLK_ERR_NULL;
  if (work && workspace_bytes < fp8blk::lora_workspace_bytes(T, K, r, L, order != nullptr))
    return FP8BLK_ERR_SHAPE;
  if (work && (any_misaligned({base_bf16, x_bf16, a_bf16, b_bf16, out_bf16, workspace}, 16) ||
               any_misaligned({ids, scale, order, offsets}, 4)))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (!work) return FP8BLK_OK;
  return launched(fp8blk::launch_lora_add(base_bf16, base_stride, x_bf16, x_stride, a_bf16, b_bf16,
                                          ids, scale, order, offsets, T, K, N, r, L, out_bf16,
                                          out_stride, workspace,
                                          static_cast<hipStream_t>(stream)));
}

// ---- gated projections -----------------------------------------------------

namespace {
constexpr int64_t kMaxWidth = int64_t(1) << 22;   // 256 rows stay below 2^32 bytes
bool bad_gated(int type, int act, int64_t M, int64_t I, int64_t K, int64_t x_stride) {
  return (type != FP8BLK_BF16 && type != FP8BLK_F16) || act < FP8BLK_SILU ||
         act > FP8BLK_GELU_TANH || bad_rows(M) || I < 0 || 2 * I > kMaxWidth || K < 1 ||
         K > kMaxWidth || x_stride < K || x_stride > kMaxWidth || !fp8blk::gated_fits(M, I, K);
}
}  // namespace

size_t fp8blk_gated_linear_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t x_stride) {
  if (bad_gated(FP8BLK_BF16, FP8BLK_SILU, M, I, K, x_stride) || M == 0 || I == 0) return 0;
  return fp8blk::gated_workspace_bytes(M, I, K, x_stride);
}

fp8blk_status fp8blk_gated_linear(const void *x, int64_t x_stride, const void *w, int type, int act,
                                  int64_t M, int64_t I, int64_t K, void *h, void *factors,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  const bool work = M > 0 && I > 0;
  if (work && (!x || !w || !h)) return FP8BLK_ERR_NULL;
  if (bad_gated(type, act, M, I, K, x_stride)) return FP8BLK_ERR_SHAPE;
  const size_t need = work ? fp8blk::gated_workspace_bytes(M, I, K, x_stride) : 0;
  if (need > 0 && !workspace) return FP8BLK_ERR_NULL;
  if (workspace_bytes < need) return FP8BLK_ERR_SHAPE;
  if (work && (any_misaligned({x, w, h, factors}, 16) || (need > 0 && misaligned(workspace))))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (!work) return FP8BLK_OK;
  const fp8blk::GatedCall c{x, w, x_stride, M, I, K, type == FP8BLK_BF16, act};
  return launched(
      fp8blk::launch_gated(c, h, factors, workspace, static_cast<hipStream_t>(stream)));
}

size_t fp8blk_gated_linear_backward_workspace_bytes(int64_t M, int64_t I, int64_t K,
                                                    int64_t x_stride, int want_d_x, int want_d_w) {
  if (bad_gated(FP8BLK_BF16, FP8BLK_SILU, M, I, K, x_stride) || M == 0 || I == 0) return 0;
  return fp8blk::gated_backward_workspace_bytes(M, I, K, x_stride, want_d_x != 0, want_d_w != 0);
}

fp8blk_status fp8blk_gated_linear_backward(const void *d_h, const void *x, int64_t x_stride,
                                           const void *w, const void *factors, int type, int act,
                                           int64_t M, int64_t I, int64_t K, void *d_x, void *d_w,
                                           void *workspace, size_t workspace_bytes, void *stream) {
  const bool work = M > 0 && I > 0 && (d_x || d_w);
  if (work && (!d_h || !x || !w)) return FP8BLK_ERR_NULL;
  if (bad_gated(type, act, M, I, K, x_stride)) return FP8BLK_ERR_SHAPE;
  const size_t need = work ? fp8blk::gated_backward_workspace_bytes(M, I, K, x_stride,
                                                                    d_x != nullptr, d_w != nullptr)
                           : 0;
  if (need > 0 && !workspace) return FP8BLK_ERR_NULL;
  if (workspace_bytes < need) return FP8BLK_ERR_SHAPE;
  if (any_misaligned({d_x, d_w}, 16) ||
      (work && (any_misaligned({d_h, x, w, factors}, 16) || (need > 0 && misaligned(workspace)))))
    return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (!d_x && !d_w) return FP8BLK_OK;
  const fp8blk::GatedCall c{x, w, x_stride, M, I, K, type == FP8BLK_BF16, act};
  return launched(fp8blk::launch_gated_backward(c, d_h, factors, d_x, d_w, workspace,
                                                static_cast<hipStream_t>(stream)));
}

// ---- 4-bit weights ---------------------------------------------------------

namespace {
bool bad_w4(int type, int group, int64_t rows, int64_t K) {
  return (type != FP8BLK_BF16 && type != FP8BLK_F16) ||
         (group != 32 && group != 64 && group != 128) || bad_rows(rows) || K < group ||
         K > kMaxWidth || K % group != 0;
}
bool bad_w4_product(int type, int group, int64_t M, int64_t rows, int64_t K, int64_t x_stride) {
  return bad_w4(type, group, rows, K) || bad_rows(M) || x_stride < K || x_stride > kMaxWidth ||
         !fp8blk::w4_fits(M, rows);
}
// Arguments of the two products; `need` is the workspace they take.
fp8blk_status check_w4(const fp8blk::W4Call &c, int type, const void *out, const void *workspace,
                       size_t workspace_bytes, size_t need) {
  const bool work = c.M > 0 && c.rows > 0;
  if (work && (!c.x || !c.codes || !c.scale || !out)) return FP8BLK_ERR_NULL;
  if (bad_w4_product(type, c.group, c.M, c.rows, c.K, c.ldx)) return FP8BLK_ERR_SHAPE;
  if (need > 0 && !workspace) return FP8BLK_ERR_NULL;
  if (workspace_bytes < need) return FP8BLK_ERR_SHAPE;
  if (work && (any_misaligned({c.x, c.codes, c.scale, c.zeros, out}, 16) ||
               (need > 0 && misaligned(workspace))))
    return FP8BLK_ERR_ALIGN;
  return check_device();
}
}  // namespace

fp8blk_status fp8blk_w4_quant(const void *w, int type, int64_t N, int64_t K, int group, void *codes,
                              void *scale, void *zeros, void *stream) {
  if (N > 0 && (!w || !codes || !scale)) return FP8BLK_ERR_NULL;
  if (bad_w4(type, group, N, K)) return FP8BLK_ERR_SHAPE;
  if (N > 0 && any_misaligned({w, codes, scale, zeros}, 16)) return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (N == 0) return FP8BLK_OK;
  return launched(fp8blk::launch_w4_quant(w, type == FP8BLK_BF16, N, K, group, codes, scale, zeros,
                                          static_cast<hipStream_t>(stream)));
}

fp8blk_status fp8blk_w4_dequant(const void *codes, const void *scale, const void *zeros, int type,
                                int64_t N, int64_t K, int group, void *w, void *stream) {
  if (N > 0 && (!w || !codes || !scale)) return FP8BLK_ERR_NULL;
  if (bad_w4(type, group, N, K)) return FP8BLK_ERR_SHAPE;
  if (N > 0 && any_misaligned({w, codes, scale, zeros}, 16)) return FP8BLK_ERR_ALIGN;
  if (fp8blk_status d = check_device()) return d;
  if (N == 0) return FP8BLK_OK;
  const fp8blk::W4Call c{nullptr, K, 0, codes, scale, zeros, N, K, group, type == FP8BLK_BF16};
  return launched(fp8blk::launch_w4_dequant(c, w, static_cast<hipStream_t>(stream)));
}

size_t fp8blk_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t x_stride) {
  if (M == 0 || N == 0 || bad_w4_product(FP8BLK_BF16, 32, M, N, K, x_stride)) return 0;
  return fp8blk::w4_linear_workspace_bytes(M, N, K, x_stride);
}

fp8blk_status fp8blk_w4_linear(const void *x, int64_t x_stride, const void *codes,
                               const void *scale, const void *zeros, int type, int group, int64_t M,
                               int64_t N, int64_t K, void *y, void *workspace,
                               size_t workspace_bytes, void *stream) {
  const fp8blk::W4Call c{x, x_stride, M, codes, scale, zeros, N, K, group, type == FP8BLK_BF16};
  if (fp8blk_status e = check_w4(c, type, y, workspace, workspace_bytes,
                                 fp8blk_w4_linear_workspace_bytes(M, N, K, x_stride)))
    return e;
  if (M == 0 || N == 0) return FP8BLK_OK;
  return launched(
      fp8blk::launch_w4_linear(c, y, workspace, static_cast<hipStream_t>(stream)));
}

size_t fp8blk_w4_gated_linear_workspace_bytes(int64_t M, int64_t I, int64_t K, int64_t x_stride) {
  if (M == 0 || I <= 0 || I > kMaxRows / 2 ||
      bad_w4_product(FP8BLK_BF16, 32, M, 2 * I, K, x_stride))
    return 0;
  return fp8blk::w4_gated_workspace_bytes(M, I, K, x_stride);
}

fp8blk_status fp8blk_w4_gated_linear(const void *x, int64_t x_stride, const void *codes,
                                     const void *scale, const void *zeros, int type, int group,
                                     int act, int64_t M, int64_t I, int64_t K, void *h,
                                     void *workspace, size_t workspace_bytes, void *stream) {
  // (a negative or too large I stays one through the doubling)
  const int64_t rows = I < 0 ? -1 : I > kMaxRows / 2 ? kMaxRows + 1 : 2 * I;
  const fp8blk::W4Call c{x, x_stride, M, codes, scale, zeros, rows, K, group, type == FP8BLK_BF16};
  if (act < FP8BLK_SILU || act > FP8BLK_GELU_TANH) return FP8BLK_ERR_SHAPE;
  if (fp8blk_status e = check_w4(c, type, h, workspace, workspace_bytes,
                                 fp8blk_w4_gated_linear_workspace_bytes(M, I, K, x_stride)))
    return e;
  if (M == 0 || I == 0) return FP8BLK_OK;
  return launched(
      fp8blk::launch_w4_gated(c, act, h, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
