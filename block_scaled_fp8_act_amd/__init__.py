"""Python binding of libfp8blk: block-scaled ("fine-grained") FP8 linear
layers on AMD MI355X (gfx950).

Argument marshalling only.  Every step of the computation runs in the HIP
kernels of libfp8blk.so; torch provides device memory and the current
stream.  There is no fallback: if the library is missing or the device is
not a gfx950, calls raise.

Low-level entry points carry the C names and take torch tensors for every
buffer (inputs and preallocated outputs):

    fp8_weight_block_quant(w, w_q, w_scale)
    fp8_act_quant_group(x, x_q, x_scale)
    fp8_block_gemm(x_q, x_scale, w_q, w_scale, y)
    fp8_grouped_block_gemm(x_q, x_scale, w_q, w_scale, offsets, y)

their power-of-two-scale twins (scales as E8M0 bytes, uint8 or
torch.float8_e8m0fnu tensors): fp8_weight_block_quant_ue8m0,
fp8_act_quant_group_ue8m0, fp8_block_gemm_ue8m0, fp8_grouped_block_gemm_ue8m0,
and the static-activation-scale pair (one fp32 scale in a 1-element device
tensor): fp8_act_quant_static(x, x_scale, x_q),
fp8_block_gemm_static(x_q, x_scale, w_q, w_scale, y); the batched expert
layout fp8_batched_block_gemm(x_q, x_scale, w_q, w_scale, counts, y) with
x_q [E, C, K]; row-wise scales fp8_rowwise_quant(x, q, scale),
fp8_rowwise_gemm(x_q, x_scale, w_q, w_scale, y); and SwiGLU ahead of the
activation quantizer fp8_swiglu_act_quant(gate_up, x_q, x_scale) (the
input of a mixture-of-experts down projection, gate_up [M, 2I] with the
gate first).

Convenience wrappers allocate the outputs; ``scale_fmt`` is "float" (fp32
scales) or "ue8m0" (E8M0 bytes), and the GEMMs pick the path from the scale
tensors' dtype:

    weight_block_quant(w, scale_fmt) -> (w_q uint8 [N,K], w_scale [ceil(N/128), K/128])
    act_quant_group(x, scale_fmt)    -> (x_q uint8 [M,K], x_scale [M, K/128])
    block_gemm(x_q, x_scale, w_q, w_scale) -> y bf16 [M,N]
    grouped_block_gemm(x_q, x_scale, w_q, w_scale, offsets) -> y bf16 [sum M_e, N]
    linear(x, w_q, w_scale) -> y bf16 [M,N]   (dynamic act quant, then GEMM)
    act_quant_static(x, x_scale) -> x_q uint8 [M,K]
    block_gemm_static(x_q, x_scale, w_q, w_scale) -> y bf16 [M,N]
    linear_static(x, x_scale, w_q, w_scale) -> y bf16 [M,N]
    batched_block_gemm(x_q, x_scale, w_q, w_scale, counts) -> y bf16 [E,C,N]
    rowwise_quant(x) -> (q uint8 [R,K], scale fp32 [R])
    rowwise_gemm(x_q, x_scale, w_q, w_scale) -> y bf16 [M,N]
    linear_rowwise(x, w_q, w_scale) -> y bf16 [M,N]
    swiglu_act_quant(gate_up, scale_fmt) -> (x_q uint8 [M,I], x_scale [M, I/128])

Around the expert products and the shared projections (low-level names
fp8blk_*, same order of arguments as the wrappers' with the outputs last):

    moe_route(logits, k, mask, renormalize, loss_coef) -> Routing(ids, weights, counts, rows, loss, ...)
    moe_route_backward(logits, routing, d_weights, d_loss) -> d_logits [T,E]
    group_rows(ids, groups) -> RowGroups(order, positions, offsets)   (offsets feed grouped_block_gemm)
    moe_combine(y, weights, positions, base) -> out bf16 [T,N]
    moe_combine_backward(d_out, y, weights, positions, offsets) -> (d_y, d_weights)
    lora_add(base, x, a, b, ids, scale, groups, out) -> out bf16 [T,N]
    lora_linear(x, w_q, w_scale, a, b, ids, scale, groups) -> y bf16 [M,N]   (linear, then its adapters)
    moe_experts(x, routing, gate_up_q, gate_up_s, down_q, down_s, base) -> y bf16 [T,N]

The gated feed-forward block in 16 bits (bf16 or fp16), with its gradients, and
weights in 4 bits (low-level names fp8blk_*, as above); act is one of ACTS:

    gated_linear(x, w, act, save) -> h [M,I]   (and with save the factors), w [2I,K] gates first
    gated_linear_backward(d_h, x, w, factors, act, need_x, need_w) -> (d_x, d_w)
    w4_quant(w, group, zeros) -> W4Weight(codes, scale, zeros)
    w4_dequant(codes, scale, zeros) -> w [N,K]
    w4_linear(x, codes, scale, zeros) -> y [M,N]
    w4_gated_linear(x, codes, scale, zeros, act) -> h [M,I]
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

__all__ = [
    "Fp8BlkError", "BLOCK", "lib_path", "load_library", "status_string",
    "fp8_weight_block_quant", "fp8_act_quant_group", "fp8_block_gemm",
    "fp8_grouped_block_gemm", "fp8_block_gemm_ws", "fp8_block_gemm_workspace_bytes",
    "fp8_block_gemm_ue8m0_ws", "fp8_block_gemm_noalloc", "SCRATCH_BYTES",
    "fp8_weight_block_quant_ue8m0", "fp8_act_quant_group_ue8m0",
    "fp8_block_gemm_ue8m0", "fp8_grouped_block_gemm_ue8m0", "fp8_act_quant_static",
    "fp8_block_gemm_static", "act_quant_static", "block_gemm_static", "linear_static",
    "fp8_linear", "fp8_batched_block_gemm", "batched_block_gemm", "fp8_rowwise_quant", "fp8_rowwise_gemm",
    "rowwise_quant", "rowwise_gemm", "linear_rowwise", "fp8_swiglu_act_quant",
    "fp8_swiglu_act_quant_ue8m0", "swiglu_act_quant",
    "weight_block_quant",
    "act_quant_group", "block_gemm", "grouped_block_gemm", "linear", "SCALE_FMTS",
    "Routing", "RowGroups", "fp8blk_moe_route", "fp8blk_moe_route_backward",
    "fp8blk_group_rows", "fp8blk_moe_combine", "fp8blk_moe_combine_backward",
    "fp8blk_lora_add", "moe_route", "moe_route_backward", "group_rows", "moe_combine",
    "moe_combine_backward", "lora_add", "lora_linear", "moe_experts",
    "MAX_GROUPS", "MAX_TOPK", "MAX_RANK",
    "ACTS", "factor_row", "fp8blk_gated_linear", "fp8blk_gated_linear_backward", "gated_linear",
    "gated_linear_backward",
    "W4_GROUPS", "W4Weight", "fp8blk_w4_quant", "fp8blk_w4_dequant", "fp8blk_w4_linear",
    "fp8blk_w4_gated_linear", "w4_quant", "w4_dequant", "w4_linear", "w4_gated_linear",
]

BLOCK = 128
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "lib", "libfp8blk.so")
_lib = None

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DEVICE, ERR_LAUNCH, ERR_SCRATCH = range(7)
SCRATCH_BYTES = 16 * 1024 * 1024 + 64 * 1024     # FP8BLK_SCRATCH_BYTES
MAX_GROUPS, MAX_TOPK, MAX_RANK = 1024, 32, 256   # FP8BLK_MAX_*


class Fp8BlkError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class Fp8BlkValueError(Fp8BlkError, ValueError):
    pass


def lib_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libfp8blk.so (built in-tree by block_scaled_fp8_act_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"libfp8blk.so not found at {_LIB_PATH}; build it with "
            "`python -m block_scaled_fp8_act_amd.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    ci, sz = ctypes.c_int, ctypes.c_size_t
    sigs = {
        "fp8_weight_block_quant": [vp, i64, i64, vp, vp, vp],
        "fp8_act_quant_group": [vp, i64, i64, vp, vp, vp],
        "fp8_block_gemm": [vp, vp, vp, vp, i64, i64, i64, vp, vp],
        "fp8_block_gemm_ws": [vp, vp, vp, vp, i64, i64, i64, vp, vp, ctypes.c_size_t, vp],
        "fp8_block_gemm_noalloc": [vp, vp, vp, vp, i64, i64, i64, vp, vp],
        "fp8_grouped_block_gemm": [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, vp],
        "fp8_linear": [vp, i64, i64, i64, vp, vp, vp, vp, vp, vp],
        "fp8_batched_block_gemm": [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, vp],
        "fp8_rowwise_quant": [vp, i64, i64, vp, vp, vp],
        "fp8_swiglu_act_quant": [vp, i64, i64, vp, vp, vp],
        "fp8_swiglu_act_quant_ue8m0": [vp, i64, i64, vp, vp, vp],
        "fp8_rowwise_gemm": [vp, vp, vp, vp, i64, i64, i64, vp, vp],
        "fp8_act_quant_static": [vp, i64, i64, vp, vp, vp],
        "fp8_block_gemm_static": [vp, vp, vp, vp, i64, i64, i64, vp, vp],
        "fp8_weight_block_quant_ue8m0": [vp, i64, i64, vp, vp, vp],
        "fp8_act_quant_group_ue8m0": [vp, i64, i64, vp, vp, vp],
        "fp8_block_gemm_ue8m0": [vp, vp, vp, vp, i64, i64, i64, vp, vp],
        "fp8_block_gemm_ue8m0_ws": [vp, vp, vp, vp, i64, i64, i64, vp, vp, ctypes.c_size_t, vp],
        "fp8_grouped_block_gemm_ue8m0": [vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, vp],
        "fp8blk_moe_route": [vp, ci, vp, i64, i32, i32, ci, ctypes.c_float, vp, vp, vp, vp, vp,
                             vp, sz, vp],
        "fp8blk_moe_route_backward": [vp, ci, i64, i32, i32, ci, ctypes.c_float, vp, vp, vp, vp,
                                      vp, vp, vp, vp],
        "fp8blk_group_rows": [vp, i64, i32, vp, vp, vp, vp, sz, vp],
        "fp8blk_moe_combine": [vp, i64, vp, vp, vp, i64, i32, i64, vp, vp],
        "fp8blk_moe_combine_backward": [vp, vp, i64, vp, vp, vp, i64, i32, i64, vp, vp, vp],
        "fp8blk_lora_add": [vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32,
                            vp, i64, vp, sz, vp],
        "fp8blk_gated_linear": [vp, i64, vp, ci, ci, i64, i64, i64, vp, vp, vp, sz, vp],
        "fp8blk_gated_linear_backward": [vp, vp, i64, vp, vp, ci, ci, i64, i64, i64, vp, vp, vp,
                                         sz, vp],
        "fp8blk_w4_quant": [vp, ci, i64, i64, ci, vp, vp, vp, vp],
        "fp8blk_w4_dequant": [vp, vp, vp, ci, i64, i64, ci, vp, vp],
        "fp8blk_w4_linear": [vp, i64, vp, vp, vp, ci, ci, i64, i64, i64, vp, vp, sz, vp],
        "fp8blk_w4_gated_linear": [vp, i64, vp, vp, vp, ci, ci, ci, i64, i64, i64, vp, vp, sz, vp],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("fp8_block_gemm_workspace_bytes", "fp8_block_gemm_ue8m0_workspace_bytes"):
        getattr(lib, name).argtypes = [i64, i64, i64]
        getattr(lib, name).restype = ctypes.c_size_t
    for name, args in {"fp8blk_moe_route_workspace_bytes": [i64, i32],
                       "fp8blk_group_rows_workspace_bytes": [i64, i32],
                       "fp8blk_lora_add_workspace_bytes": [i64, i64, i32, i32, ci],
                       "fp8blk_gated_linear_workspace_bytes": [i64, i64, i64, i64],
                       "fp8blk_gated_linear_backward_workspace_bytes": [i64, i64, i64, i64, ci,
                                                                        ci],
                       "fp8blk_w4_linear_workspace_bytes": [i64, i64, i64, i64],
                       "fp8blk_w4_gated_linear_workspace_bytes": [i64, i64, i64, i64]}.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = sz
    lib.fp8blk_status_string.argtypes = [ctypes.c_int]
    lib.fp8blk_status_string.restype = ctypes.c_char_p
    lib.fp8blk_abi_version.argtypes = []
    lib.fp8blk_abi_version.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().fp8blk_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status == OK:
        return
    msg = f"{what}: {status_string(status)}"
    if status in (ERR_SHAPE, ERR_DEVICE):
        raise Fp8BlkValueError(status, msg)
    raise Fp8BlkError(status, msg)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


# The current stream's handle without a Stream object around it: 0.3 us a call
# against 2.9 us (host-bound decode steps make several).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _need(t: torch.Tensor, name: str, dtypes, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (cuda/hip) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")


_CODES = (torch.uint8, torch.float8_e4m3fn)


def _shape_eq(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


# --------------------------------------------------------------------------
# low-level entry points (same names as the C ABI)

_F32 = (torch.float32,)
_E8M0 = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())
SCALE_FMTS = ("float", "ue8m0")


def _weight_quant(cname, sdt, w, w_q, w_scale):
    _need(w, "w", (torch.bfloat16,), 2)
    N, K = w.shape
    _need(w_q, "w_q", _CODES); _need(w_scale, "w_scale", sdt)
    _shape_eq(w_q, (N, K), "w_q")
    if K % BLOCK == 0:
        _shape_eq(w_scale, (-(-N // BLOCK), K // BLOCK), "w_scale")
    _check(getattr(load_library(), cname)(_ptr(w), N, K, _ptr(w_q), _ptr(w_scale), _stream()),
           cname)


def _act_quant(cname, sdt, x, x_q, x_scale):
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    _need(x_q, "x_q", _CODES); _need(x_scale, "x_scale", sdt)
    _shape_eq(x_q, (M, K), "x_q")
    if K % BLOCK == 0:
        _shape_eq(x_scale, (M, K // BLOCK), "x_scale")
    _check(getattr(load_library(), cname)(_ptr(x), M, K, _ptr(x_q), _ptr(x_scale), _stream()),
           cname)


def _gemm(cname, sdt, x_q, x_scale, w_q, w_scale, y):
    _need(x_q, "x_q", _CODES, 2); _need(w_q, "w_q", _CODES, 2)
    _need(x_scale, "x_scale", sdt, 2); _need(w_scale, "w_scale", sdt, 2)
    _need(y, "y", (torch.bfloat16,), 2)
    M, K = x_q.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("x_q and w_q disagree on K")
    if K % BLOCK == 0:
        _shape_eq(x_scale, (M, K // BLOCK), "x_scale")
        _shape_eq(w_scale, (-(-N // BLOCK), K // BLOCK), "w_scale")
    _shape_eq(y, (M, N), "y")
    _check(getattr(load_library(), cname)(_ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale),
                                          M, N, K, _ptr(y), _stream()), cname)


def _grouped(cname, sdt, x_q, x_scale, w_q, w_scale, offsets, y):
    _need(x_q, "x_q", _CODES, 2); _need(w_q, "w_q", _CODES, 3)
    _need(x_scale, "x_scale", sdt, 2); _need(w_scale, "w_scale", sdt, 3)
    _need(offsets, "offsets", (torch.int32,), 1); _need(y, "y", (torch.bfloat16,), 2)
    total, K = x_q.shape
    E, N, K2 = w_q.shape
    if K2 != K:
        raise ValueError("x_q and w_q disagree on K")
    if offsets.numel() != E + 1:
        raise ValueError("offsets must have E+1 entries")
    if K % BLOCK == 0:
        _shape_eq(x_scale, (total, K // BLOCK), "x_scale")
        _shape_eq(w_scale, (E, -(-N // BLOCK), K // BLOCK), "w_scale")
    _shape_eq(y, (total, N), "y")
    _check(getattr(load_library(), cname)(
        _ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale), _ptr(offsets), E, total, N, K,
        _ptr(y), _stream()), cname)


def fp8_weight_block_quant(w, w_q, w_scale):
    _weight_quant("fp8_weight_block_quant", _F32, w, w_q, w_scale)


def fp8_act_quant_group(x, x_q, x_scale):
    _act_quant("fp8_act_quant_group", _F32, x, x_q, x_scale)


def fp8_block_gemm(x_q, x_scale, w_q, w_scale, y):
    _gemm("fp8_block_gemm", _F32, x_q, x_scale, w_q, w_scale, y)


def fp8_block_gemm_noalloc(x_q, x_scale, w_q, w_scale, y):
    """fp8_block_gemm_ws with the library's own device scratch: no
    workspace, no allocation (callers that cannot allocate)."""
    _gemm("fp8_block_gemm_noalloc", _F32, x_q, x_scale, w_q, w_scale, y)


def fp8_block_gemm_workspace_bytes(M, N, K, scale_fmt="float"):
    """Workspace bytes fp8_block_gemm_ws (scale_fmt "ue8m0":
    fp8_block_gemm_ue8m0_ws) splits K with for these sizes (0: no split; the
    call is then the plain GEMM)."""
    name = ("fp8_block_gemm_ue8m0_workspace_bytes" if scale_fmt == "ue8m0"
            else "fp8_block_gemm_workspace_bytes")
    return int(getattr(load_library(), name)(int(M), int(N), int(K)))


def fp8_block_gemm_ws(x_q, x_scale, w_q, w_scale, y, workspace=None):
    """fp8_block_gemm with K split over workgroups through ``workspace`` (a
    device tensor of at least fp8_block_gemm_workspace_bytes bytes) for
    grids that would leave most CUs idle; without a large enough workspace
    it is fp8_block_gemm."""
    _gemm_ws("fp8_block_gemm_ws", _F32, x_q, x_scale, w_q, w_scale, y, workspace)


def fp8_block_gemm_ue8m0_ws(x_q, x_scale, w_q, w_scale, y, workspace=None):
    """fp8_block_gemm_ue8m0 with K split over workgroups (as fp8_block_gemm_ws)."""
    _gemm_ws("fp8_block_gemm_ue8m0_ws", _E8M0, x_q, x_scale, w_q, w_scale, y, workspace)


def _gemm_ws(cname, sdt, x_q, x_scale, w_q, w_scale, y, workspace):
    _need(x_q, "x_q", _CODES, 2); _need(w_q, "w_q", _CODES, 2)
    _need(x_scale, "x_scale", sdt, 2); _need(w_scale, "w_scale", sdt, 2)
    _need(y, "y", (torch.bfloat16,), 2)
    M, K = x_q.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("x_q and w_q disagree on K")
    if K % BLOCK == 0:
        _shape_eq(x_scale, (M, K // BLOCK), "x_scale")
        _shape_eq(w_scale, (-(-N // BLOCK), K // BLOCK), "w_scale")
    _shape_eq(y, (M, N), "y")
    wbytes = 0
    if workspace is not None:
        _need(workspace, "workspace", (workspace.dtype,))
        wbytes = workspace.numel() * workspace.element_size()
    _check(getattr(load_library(), cname)(_ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale),
                                          M, N, K, _ptr(y), _ptr(workspace), wbytes, _stream()),
           cname)


def fp8_grouped_block_gemm(x_q, x_scale, w_q, w_scale, offsets, y):
    _grouped("fp8_grouped_block_gemm", _F32, x_q, x_scale, w_q, w_scale, offsets, y)


def _static_scale(x_scale):
    _need(x_scale, "x_scale", _F32)
    if x_scale.numel() != 1:
        raise ValueError("the static activation scale is one fp32 value")


def fp8_act_quant_static(x, x_scale, x_q):
    _need(x, "x", (torch.bfloat16,), 2)
    M, K = x.shape
    _static_scale(x_scale)
    _need(x_q, "x_q", _CODES)
    _shape_eq(x_q, (M, K), "x_q")
    _check(load_library().fp8_act_quant_static(_ptr(x), M, K, _ptr(x_scale), _ptr(x_q), _stream()),
           "fp8_act_quant_static")


def fp8_block_gemm_static(x_q, x_scale, w_q, w_scale, y):
    _need(x_q, "x_q", _CODES, 2); _need(w_q, "w_q", _CODES, 2)
    _static_scale(x_scale); _need(w_scale, "w_scale", _F32, 2)
    _need(y, "y", (torch.bfloat16,), 2)
    M, K = x_q.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("x_q and w_q disagree on K")
    if K % BLOCK == 0:
        _shape_eq(w_scale, (-(-N // BLOCK), K // BLOCK), "w_scale")
    _shape_eq(y, (M, N), "y")
    _check(load_library().fp8_block_gemm_static(_ptr(x_q), _ptr(x_scale), _ptr(w_q),
                                                _ptr(w_scale), M, N, K, _ptr(y), _stream()),
           "fp8_block_gemm_static")


FUSED_MAX_M = 64


def fp8_linear(x, w_q, w_scale, y, x_q_ws=None, x_scale_ws=None):
    """One C call for the linear layer: fused in one kernel for M <= 64 when
    no workspaces are given, and with workspaces where that is faster (M <= 16
    with N * K <= 2^25 or with several 16-column slabs per workgroup at
    K <= 8192; 16 < M <= 32 with N * K <= 2^24); else quantization into the
    workspaces (required for M > 64) and the GEMM."""
    _need(x, "x", (torch.bfloat16,), 2); _need(w_q, "w_q", _CODES, 2)
    _need(w_scale, "w_scale", _F32, 2); _need(y, "y", (torch.bfloat16,), 2)
    M, K = x.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("x and w_q disagree on K")
    if K % BLOCK == 0:
        _shape_eq(w_scale, (-(-N // BLOCK), K // BLOCK), "w_scale")
    _shape_eq(y, (M, N), "y")
    if M > FUSED_MAX_M:
        if x_q_ws is None or x_scale_ws is None:
            raise ValueError("M > 64 needs the x_q_ws / x_scale_ws workspaces")
        _need(x_q_ws, "x_q_ws", _CODES); _need(x_scale_ws, "x_scale_ws", _F32)
        _shape_eq(x_q_ws, (M, K), "x_q_ws")
        if K % BLOCK == 0:
            _shape_eq(x_scale_ws, (M, K // BLOCK), "x_scale_ws")
    _check(load_library().fp8_linear(_ptr(x), M, N, K, _ptr(w_q), _ptr(w_scale), _ptr(x_q_ws),
                                     _ptr(x_scale_ws), _ptr(y), _stream()), "fp8_linear")


def fp8_batched_block_gemm(x_q, x_scale, w_q, w_scale, counts, y):
    _need(x_q, "x_q", _CODES, 3); _need(w_q, "w_q", _CODES, 3)
    _need(x_scale, "x_scale", _F32, 3); _need(w_scale, "w_scale", _F32, 3)
    _need(counts, "counts", (torch.int32,), 1); _need(y, "y", (torch.bfloat16,), 3)
    E, C, K = x_q.shape
    E2, N, K2 = w_q.shape
    if E2 != E or K2 != K:
        raise ValueError("x_q [E,C,K] and w_q [E,N,K] disagree")
    if counts.numel() != E:
        raise ValueError("counts must have E entries")
    if K % BLOCK == 0:
        _shape_eq(x_scale, (E, C, K // BLOCK), "x_scale")
        _shape_eq(w_scale, (E, -(-N // BLOCK), K // BLOCK), "w_scale")
    _shape_eq(y, (E, C, N), "y")
    _check(load_library().fp8_batched_block_gemm(
        _ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale), _ptr(counts), E, C, N, K, _ptr(y),
        _stream()), "fp8_batched_block_gemm")


def fp8_rowwise_quant(x, q, scale):
    _need(x, "x", (torch.bfloat16,), 2)
    R, K = x.shape
    _need(q, "q", _CODES); _need(scale, "scale", _F32)
    _shape_eq(q, (R, K), "q")
    _shape_eq(scale, (R,), "scale")
    _check(load_library().fp8_rowwise_quant(_ptr(x), R, K, _ptr(q), _ptr(scale), _stream()),
           "fp8_rowwise_quant")


def _swiglu(cname, sdt, gate_up, x_q, x_scale):
    _need(gate_up, "gate_up", (torch.bfloat16,), 2)
    M, two_i = gate_up.shape
    if two_i % 2:
        raise ValueError("gate_up must hold 2I columns")
    I = two_i // 2
    _need(x_q, "x_q", _CODES); _need(x_scale, "x_scale", sdt)
    _shape_eq(x_q, (M, I), "x_q")
    if I % BLOCK == 0:
        _shape_eq(x_scale, (M, I // BLOCK), "x_scale")
    _check(getattr(load_library(), cname)(_ptr(gate_up), M, I, _ptr(x_q), _ptr(x_scale),
                                          _stream()), cname)


def fp8_swiglu_act_quant(gate_up, x_q, x_scale):
    """gate_up bf16 [M, 2I] (gate in columns [0, I), up in [I, 2I)) ->
    codes of h = bf16(SiLU(gate) * up) in x_q [M, I] and fp32 group scales
    in x_scale [M, I/128]."""
    _swiglu("fp8_swiglu_act_quant", _F32, gate_up, x_q, x_scale)


def fp8_swiglu_act_quant_ue8m0(gate_up, x_q, x_scale):
    """As fp8_swiglu_act_quant with E8M0 scale bytes (uint8 or float8_e8m0fnu)."""
    _swiglu("fp8_swiglu_act_quant_ue8m0", _E8M0, gate_up, x_q, x_scale)


def fp8_rowwise_gemm(x_q, x_scale, w_q, w_scale, y):
    _need(x_q, "x_q", _CODES, 2); _need(w_q, "w_q", _CODES, 2)
    _need(x_scale, "x_scale", _F32, 1); _need(w_scale, "w_scale", _F32, 1)
    _need(y, "y", (torch.bfloat16,), 2)
    M, K = x_q.shape
    N = w_q.shape[0]
    if w_q.shape[1] != K:
        raise ValueError("x_q and w_q disagree on K")
    _shape_eq(x_scale, (M,), "x_scale"); _shape_eq(w_scale, (N,), "w_scale")
    _shape_eq(y, (M, N), "y")
    _check(load_library().fp8_rowwise_gemm(_ptr(x_q), _ptr(x_scale), _ptr(w_q), _ptr(w_scale),
                                           M, N, K, _ptr(y), _stream()), "fp8_rowwise_gemm")


def fp8_weight_block_quant_ue8m0(w, w_q, w_scale):
    _weight_quant("fp8_weight_block_quant_ue8m0", _E8M0, w, w_q, w_scale)


def fp8_act_quant_group_ue8m0(x, x_q, x_scale):
    _act_quant("fp8_act_quant_group_ue8m0", _E8M0, x, x_q, x_scale)


def fp8_block_gemm_ue8m0(x_q, x_scale, w_q, w_scale, y):
    _gemm("fp8_block_gemm_ue8m0", _E8M0, x_q, x_scale, w_q, w_scale, y)


def fp8_grouped_block_gemm_ue8m0(x_q, x_scale, w_q, w_scale, offsets, y):
    _grouped("fp8_grouped_block_gemm_ue8m0", _E8M0, x_q, x_scale, w_q, w_scale, offsets, y)


# --------------------------------------------------------------------------
# convenience wrappers (allocate outputs with torch.empty)

def _scale_dtype(scale_fmt):
    if scale_fmt not in SCALE_FMTS:
        raise ValueError(f"scale_fmt must be one of {SCALE_FMTS}, got {scale_fmt!r}")
    return torch.float32 if scale_fmt == "float" else torch.uint8


def _is_e8m0(t):
    return t.dtype in _E8M0


def weight_block_quant(w, scale_fmt="float"):
    N, K = w.shape
    w_q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    w_s = torch.empty((-(-N // BLOCK), max(K // BLOCK, 0)), dtype=_scale_dtype(scale_fmt),
                      device=w.device)
    (fp8_weight_block_quant if scale_fmt == "float" else fp8_weight_block_quant_ue8m0)(w, w_q, w_s)
    return w_q, w_s


def act_quant_group(x, scale_fmt="float"):
    M, K = x.shape
    x_q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    x_s = torch.empty((M, max(K // BLOCK, 0)), dtype=_scale_dtype(scale_fmt), device=x.device)
    (fp8_act_quant_group if scale_fmt == "float" else fp8_act_quant_group_ue8m0)(x, x_q, x_s)
    return x_q, x_s


def block_gemm(x_q, x_scale, w_q, w_scale):
    """y = x * W^T in bf16.  fp32 scales: with K split over workgroups (and a
    workspace from torch's allocator) when the library asks for one."""
    M, N, K = x_q.shape[0], w_q.shape[0], x_q.shape[1]
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x_q.device)
    e8m0 = _is_e8m0(w_scale)
    need = fp8_block_gemm_workspace_bytes(M, N, K, "ue8m0" if e8m0 else "float")
    if need:
        work = torch.empty(need, dtype=torch.uint8, device=x_q.device)
        (fp8_block_gemm_ue8m0_ws if e8m0 else fp8_block_gemm_ws)(x_q, x_scale, w_q, w_scale, y, work)
    else:
        (fp8_block_gemm_ue8m0 if e8m0 else fp8_block_gemm)(x_q, x_scale, w_q, w_scale, y)
    return y


def grouped_block_gemm(x_q, x_scale, w_q, w_scale, offsets):
    y = torch.empty((x_q.shape[0], w_q.shape[1]), dtype=torch.bfloat16, device=x_q.device)
    fn = fp8_grouped_block_gemm_ue8m0 if _is_e8m0(w_scale) else fp8_grouped_block_gemm
    fn(x_q, x_scale, w_q, w_scale, offsets, y)
    return y


def linear(x, w_q, w_scale):
    """The FP8 linear layer: dynamic per-token-group quantization of x, then
    the block-scaled GEMM on the current stream (fp32 scales: one C call,
    fused into one kernel where the library finds that faster, M <= 32; the
    quantizer then the GEMM with a workspace when the library asks for one:
    output grids too small to fill the chip (K split over workgroups, or
    stream-K with long K), a partly empty last round of tiles, and 9 <= M <=
    16 or 33 <= M <= 64 with long K, where re-reading x per column slab costs
    more than the separate quantizer and the split).  E8M0 weight scales
    select power-of-two activation scales as well."""
    if _is_e8m0(w_scale):
        x_q, x_s = act_quant_group(x, "ue8m0")
        return block_gemm(x_q, x_s, w_q, w_scale)
    M, K = x.shape
    if fp8_block_gemm_workspace_bytes(M, w_q.shape[0], K):
        x_q, x_s = act_quant_group(x)
        return block_gemm(x_q, x_s, w_q, w_scale)
    y = torch.empty((M, w_q.shape[0]), dtype=torch.bfloat16, device=x.device)
    x_q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    x_s = torch.empty((M, max(K // BLOCK, 0)), dtype=torch.float32, device=x.device)
    fp8_linear(x, w_q, w_scale, y, x_q, x_s)   # the library picks fused or two kernels
    return y


def act_quant_static(x, x_scale):
    x_q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    fp8_act_quant_static(x, x_scale, x_q)
    return x_q


def block_gemm_static(x_q, x_scale, w_q, w_scale):
    y = torch.empty((x_q.shape[0], w_q.shape[0]), dtype=torch.bfloat16, device=x_q.device)
    fp8_block_gemm_static(x_q, x_scale, w_q, w_scale, y)
    return y


def linear_static(x, x_scale, w_q, w_scale):
    """The FP8 linear layer with a static (calibrated, per-tensor) activation
    scale: quantization of x, then the block-scaled GEMM."""
    return block_gemm_static(act_quant_static(x, x_scale), x_scale, w_q, w_scale)


def batched_block_gemm(x_q, x_scale, w_q, w_scale, counts):
    """Rows past an expert's count are left as torch.empty returned them."""
    y = torch.empty((x_q.shape[0], x_q.shape[1], w_q.shape[1]), dtype=torch.bfloat16,
                    device=x_q.device)
    fp8_batched_block_gemm(x_q, x_scale, w_q, w_scale, counts, y)
    return y


def rowwise_quant(x):
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty((x.shape[0],), dtype=torch.float32, device=x.device)
    fp8_rowwise_quant(x, q, s)
    return q, s


def swiglu_act_quant(gate_up, scale_fmt="float"):
    M, I = gate_up.shape[0], gate_up.shape[1] // 2
    q = torch.empty((M, I), dtype=torch.uint8, device=gate_up.device)
    s = torch.empty((M, I // BLOCK), dtype=_scale_dtype(scale_fmt), device=gate_up.device)
    (fp8_swiglu_act_quant if scale_fmt == "float" else fp8_swiglu_act_quant_ue8m0)(gate_up, q, s)
    return q, s


def rowwise_gemm(x_q, x_scale, w_q, w_scale):
    y = torch.empty((x_q.shape[0], w_q.shape[0]), dtype=torch.bfloat16, device=x_q.device)
    fp8_rowwise_gemm(x_q, x_scale, w_q, w_scale, y)
    return y


def linear_rowwise(x, w_q, w_scale):
    """Row-wise ("fp8r") linear layer: per-token quantization of x, then the
    row-scaled GEMM."""
    x_q, x_s = rowwise_quant(x)
    return rowwise_gemm(x_q, x_s, w_q, w_scale)


# --------------------------------------------------------------------------
# routing, rows by group, combine, adapters

class Routing(NamedTuple):
    """What moe_route found, as moe_route_backward and group_rows take it."""
    ids: torch.Tensor        # [T,k] int32, -1 in unused slots
    weights: torch.Tensor    # [T,k] fp32
    counts: torch.Tensor     # [E] int32
    rows: torch.Tensor | None   # [1] int32: rows routed (with the loss)
    loss: torch.Tensor | None   # fp32 scalar
    loss_coef: float
    renormalize: bool


class RowGroups(NamedTuple):
    """Rows listed by group: order[offsets[g]:offsets[g+1]] are group g's."""
    order: torch.Tensor      # [R] int32
    positions: torch.Tensor  # as the ids' shape, int32, -1 for rows of no group
    offsets: torch.Tensor    # [G+1] int32


_LOGITS = {torch.float32: 0, torch.bfloat16: 1}    # FP8BLK_F32, FP8BLK_BF16
_LOGIT_TYPES = tuple(_LOGITS)
_I32 = (torch.int32,)
_BF16 = (torch.bfloat16,)
_MASK = (torch.bool, torch.uint8)


def _rows_2d(t, name, dtypes=(torch.bfloat16,)):
    """A matrix whose rows are contiguous and a fixed stride apart; the stride."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a torch.Tensor of a type in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (cuda/hip) tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    if t.is_contiguous():
        return t.shape[1]
    rows, cols = t.shape
    if rows <= 1 or cols == 0:
        if cols > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}'s rows must be contiguous")
        return cols
    if (cols > 1 and t.stride(1) != 1) or t.stride(0) < cols:
        raise ValueError(f"{name}'s rows must be contiguous and not overlap")
    return t.stride(0)


def _same_device(first, *others):
    """All on the current device, where the kernels are launched."""
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError("all tensors must be on one device")
    if d != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{d}, which is not the current device")


def _plain(device, *specs):
    """Whether every (tensor, dtype, shape) is just that, contiguous and on the
    device: the one quick look that most calls need; where it is not so, the
    checks one by one accept it or say what is wrong."""
    for t, dtype, shape in specs:
        if (t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != device
                               or not t.is_contiguous())):
            return False
    return device == torch.cuda.current_device()


def _at(t):
    return t.data_ptr() if t is not None else None


def _work(need, like):
    return like.new_empty((need,), dtype=torch.uint8) if need else None


def _bytes(t):
    return t.numel() * t.element_size() if t is not None else 0


def _need_work(t):
    """A caller's workspace: contiguous, so that its size is what it covers."""
    if t is not None:
        _need(t, "workspace", (t.dtype,))


# Each operator's call of the library, its arguments checked: the low-level entry
# points check every buffer, the wrappers what the caller gave them.

def _route_in(logits, mask):
    _need(logits, "logits", _LOGIT_TYPES, 2)
    if mask is not None:
        _need(mask, "mask", _MASK, 1)
        _shape_eq(mask, (logits.shape[0],), "mask")


def _route_call(logits, mask, k, renormalize, coef, ids, weights, counts, rows, loss, workspace):
    T, E = logits.shape
    _check(load_library().fp8blk_moe_route(
        logits.data_ptr(), _LOGITS[logits.dtype], _at(mask), T, E, k, renormalize, coef,
        ids.data_ptr(), weights.data_ptr(), counts.data_ptr(), _at(rows), _at(loss),
        _at(workspace), _bytes(workspace), _stream()), "fp8blk_moe_route")


def fp8blk_moe_route(logits, mask, renormalize, loss_coef, ids, weights, counts, rows, loss,
                     workspace=None):
    """Routing into preallocated outputs; k is ids' width, ``mask`` (uint8 or
    bool [T]), ``rows`` (int32) and ``loss`` (fp32, one value each) may be None,
    ``workspace`` holds fp8blk_moe_route_workspace_bytes(T, E) bytes."""
    _route_in(logits, mask)
    T, E = logits.shape
    _need(ids, "ids", _I32, 2); _need(weights, "weights", _F32, 2)
    _need(counts, "counts", _I32, 1)
    k = ids.shape[1]
    _shape_eq(ids, (T, k), "ids"); _shape_eq(weights, (T, k), "weights")
    _shape_eq(counts, (E,), "counts")
    for t, name, dtype in ((rows, "rows", _I32), (loss, "loss", _F32)):
        if t is not None:
            _need(t, name, dtype)
            if t.numel() != 1:
                raise ValueError(f"{name} holds one value")
    _need_work(workspace)
    _same_device(logits, mask, ids, weights, counts, rows, loss, workspace)
    _route_call(logits, mask, k, bool(renormalize), loss_coef, ids, weights, counts, rows, loss,
                workspace)


def _route_back_in(logits, routing, d_weights, d_loss):
    _need(logits, "logits", _LOGIT_TYPES, 2)
    T, E = logits.shape
    ids, weights, counts = routing.ids, routing.weights, routing.counts
    _need(ids, "routing.ids", _I32, 2); _need(weights, "routing.weights", _F32, 2)
    _need(counts, "routing.counts", _I32, 1)
    k = ids.shape[1]
    _shape_eq(ids, (T, k), "routing.ids"); _shape_eq(weights, (T, k), "routing.weights")
    _shape_eq(counts, (E,), "routing.counts")
    if d_weights is not None:
        _need(d_weights, "d_weights", _F32, 2)
        _shape_eq(d_weights, (T, k), "d_weights")
    if d_loss is not None:
        _need(d_loss, "d_loss", _F32)
        if d_loss.numel() != 1:
            raise ValueError("d_loss holds one value")
        if routing.rows is None:
            raise ValueError("d_loss needs a routing that computed the loss")
        _need(routing.rows, "routing.rows", _I32)
        if routing.rows.numel() != 1:
            raise ValueError("routing.rows holds one value")


def _route_back_call(logits, routing, d_weights, d_loss, d_logits):
    T, E = logits.shape
    _check(load_library().fp8blk_moe_route_backward(
        logits.data_ptr(), _LOGITS[logits.dtype], T, E, routing.ids.shape[1], routing.renormalize,
        routing.loss_coef, routing.ids.data_ptr(), routing.weights.data_ptr(),
        routing.counts.data_ptr(), _at(routing.rows), _at(d_weights), _at(d_loss),
        d_logits.data_ptr(), _stream()), "fp8blk_moe_route_backward")


def fp8blk_moe_route_backward(logits, routing, d_weights, d_loss, d_logits):
    """Gradient of the logits into d_logits; d_weights [T,k] or d_loss (one
    value) may be None."""
    _route_back_in(logits, routing, d_weights, d_loss)
    _need(d_logits, "d_logits", (logits.dtype,), 2)
    _shape_eq(d_logits, logits.shape, "d_logits")
    _same_device(logits, routing.ids, routing.weights, routing.counts, routing.rows, d_weights,
                 d_loss, d_logits)
    _route_back_call(logits, routing, d_weights, d_loss, d_logits)


def _group_call(ids, groups, order, positions, offsets, workspace):
    _check(load_library().fp8blk_group_rows(
        ids.data_ptr(), ids.numel(), groups, order.data_ptr(), positions.data_ptr(),
        offsets.data_ptr(), _at(workspace), _bytes(workspace), _stream()), "fp8blk_group_rows")


def fp8blk_group_rows(ids, order, positions, offsets, workspace=None):
    """Rows by group into preallocated outputs; G is offsets' length less one,
    ``workspace`` holds fp8blk_group_rows_workspace_bytes(R, G) bytes."""
    _need(ids, "ids", _I32); _need(order, "order", _I32)
    _need(positions, "positions", _I32); _need(offsets, "offsets", _I32, 1)
    R = ids.numel()
    if order.numel() != R or positions.numel() != R:
        raise ValueError("order and positions have an entry per row")
    _need_work(workspace)
    _same_device(ids, order, positions, offsets, workspace)
    _group_call(ids, offsets.numel() - 1, order, positions, offsets, workspace)


def _combine_in(y, weights, positions, base):
    _need(y, "y", _BF16, 2); _need(weights, "weights", _F32, 2)
    _need(positions, "positions", _I32, 2)
    _shape_eq(positions, weights.shape, "positions")
    if base is not None:
        _need(base, "base", _BF16, 2)
        _shape_eq(base, (weights.shape[0], y.shape[1]), "base")


def _combine_call(y, weights, positions, base, out):
    T, k = weights.shape
    R, N = y.shape
    _check(load_library().fp8blk_moe_combine(
        y.data_ptr(), R, weights.data_ptr(), positions.data_ptr(), _at(base), T, k, N,
        out.data_ptr(), _stream()), "fp8blk_moe_combine")


def fp8blk_moe_combine(y, weights, positions, base, out):
    """Weighted sums of y's rows into out; base may be None or out itself."""
    _combine_in(y, weights, positions, base)
    _need(out, "out", _BF16, 2)
    _shape_eq(out, (weights.shape[0], y.shape[1]), "out")
    _same_device(y, weights, positions, base, out)
    _combine_call(y, weights, positions, base, out)


def _combine_back_in(d_out, y, weights, positions, rows_used):
    _combine_in(y, weights, positions, None)
    _need(d_out, "d_out", _BF16, 2); _need(rows_used, "rows_used", _I32)
    _shape_eq(d_out, (weights.shape[0], y.shape[1]), "d_out")
    if rows_used.numel() < 1:
        raise ValueError("rows_used holds one value at least")


def _combine_back_call(d_out, y, weights, positions, rows_used, d_y, d_weights):
    T, k = weights.shape
    R, N = y.shape
    _check(load_library().fp8blk_moe_combine_backward(
        d_out.data_ptr(), y.data_ptr(), R, weights.data_ptr(), positions.data_ptr(),
        rows_used.data_ptr() + 4 * (rows_used.numel() - 1), T, k, N, d_y.data_ptr(),
        d_weights.data_ptr(), _stream()), "fp8blk_moe_combine_backward")


def fp8blk_moe_combine_backward(d_out, y, weights, positions, rows_used, d_y, d_weights):
    """Gradients into d_y and d_weights; the last entry of ``rows_used`` (an
    int32 tensor, e.g. RowGroups.offsets) is the number of y's rows in use."""
    _combine_back_in(d_out, y, weights, positions, rows_used)
    _need(d_y, "d_y", _BF16, 2); _need(d_weights, "d_weights", _F32, 2)
    _shape_eq(d_y, y.shape, "d_y"); _shape_eq(d_weights, weights.shape, "d_weights")
    _same_device(d_out, y, weights, positions, rows_used, d_y, d_weights)
    _combine_back_call(d_out, y, weights, positions, rows_used, d_y, d_weights)


def _lora_in(base, x, a, b, ids, scale, groups, out):
    """Row strides of base, x and out."""
    ldx, ldo = _rows_2d(x, "x"), _rows_2d(out, "out")
    _need(a, "a", _BF16, 3); _need(b, "b", _BF16, 3); _need(ids, "ids", _I32, 1)
    T, K = x.shape
    L, r, K2 = a.shape
    N = out.shape[1]
    if K2 != K:
        raise ValueError("x and a disagree on K")
    _shape_eq(b, (L, N, r), "b"); _shape_eq(ids, (T,), "ids")
    _shape_eq(out, (T, N), "out")
    ldb = 0
    if base is not None:
        ldb = _rows_2d(base, "base")
        _shape_eq(base, (T, N), "base")
    if scale is not None:
        _need(scale, "scale", _F32, 1)
        _shape_eq(scale, (L,), "scale")
    order = offsets = None
    if groups is not None:
        order, offsets = groups.order, groups.offsets
        _need(order, "groups.order", _I32, 1); _need(offsets, "groups.offsets", _I32, 1)
        _shape_eq(order, (T,), "groups.order"); _shape_eq(offsets, (L + 1,), "groups.offsets")
    _same_device(x, base, a, b, ids, scale, order, offsets, out)
    return ldb, ldx, ldo


def _lora_call(base, x, a, b, ids, scale, groups, out, workspace, strides):
    T, K = x.shape
    L, r = a.shape[:2]
    order, offsets = (groups.order, groups.offsets) if groups is not None else (None, None)
    _check(load_library().fp8blk_lora_add(
        _at(base), strides[0], x.data_ptr(), strides[1], a.data_ptr(), b.data_ptr(),
        ids.data_ptr(), _at(scale), _at(order), _at(offsets), T, K, out.shape[1], r, L,
        out.data_ptr(), strides[2], _at(workspace), _bytes(workspace), _stream()),
        "fp8blk_lora_add")


def fp8blk_lora_add(base, x, a, b, ids, scale, groups, out, workspace):
    """Adapters into out; base, scale and groups may be None; base and out, and
    x, may be column slices of wider matrices.  ``workspace`` holds
    fp8blk_lora_add_workspace_bytes(T, K, r, L, listed) bytes."""
    strides = _lora_in(base, x, a, b, ids, scale, groups, out)
    _need_work(workspace)
    _same_device(x, workspace)
    _lora_call(base, x, a, b, ids, scale, groups, out, workspace, strides)


def moe_route(logits, k, mask=None, renormalize=True, loss_coef=None):
    """The k experts of each token with their softmax weights, and how many
    rows each expert gets; with ``loss_coef`` also the balance loss
    loss_coef * sum_e (counts_e E / (k n)) * mean_t p_te.  Rows with mask 0,
    and experts with logit -inf, are left out; unused slots have id -1 and
    weight 0."""
    _route_in(logits, mask)
    _same_device(logits, mask)
    T, E = logits.shape
    if not 1 <= k <= E:
        raise ValueError(f"k must be between 1 and the number of experts, got {k}")
    ids = logits.new_empty((T, k), dtype=torch.int32)
    weights = logits.new_empty((T, k), dtype=torch.float32)
    counts = logits.new_empty((E,), dtype=torch.int32)
    rows = loss = None
    if loss_coef is not None:
        rows = logits.new_empty((1,), dtype=torch.int32)
        loss = logits.new_empty((), dtype=torch.float32)
    coef, renormalize = float(loss_coef or 0.0), bool(renormalize)
    _route_call(logits, mask, k, renormalize, coef, ids, weights, counts, rows, loss,
                _work(load_library().fp8blk_moe_route_workspace_bytes(T, E), logits))
    return Routing(ids, weights, counts, rows, loss, coef, renormalize)


def moe_route_backward(logits, routing, d_weights=None, d_loss=None):
    """Gradient of the logits (in their type) from those of the weights and of
    the loss; the choice itself has none."""
    T, E = logits.shape
    slots = (T, routing.ids.shape[1])
    if not (logits.dtype in _LOGITS and (d_loss is None or d_loss.dim() == 0) and routing.rows is not None
            and _plain(logits.get_device(), (logits, logits.dtype, (T, E)),
                       (routing.ids, torch.int32, slots), (routing.weights, torch.float32, slots),
                       (routing.counts, torch.int32, (E,)), (routing.rows, torch.int32, (1,)),
                       (d_weights, torch.float32, slots), (d_loss, torch.float32, ()))):
        _route_back_in(logits, routing, d_weights, d_loss)
        _same_device(logits, routing.ids, routing.weights, routing.counts, routing.rows, d_weights,
                     d_loss)
    d_logits = torch.empty_like(logits)
    _route_back_call(logits, routing, d_weights, d_loss, d_logits)
    return d_logits


def group_rows(ids, groups):
    """Rows (entries of ids, any shape) listed by group, in their own order
    within a group; entries outside [0, groups) belong to none and come last."""
    _need(ids, "ids", _I32)
    _same_device(ids)
    R = ids.numel()
    order, positions = ids.new_empty((R,)), torch.empty_like(ids)
    offsets = ids.new_empty((groups + 1,))
    _group_call(ids, groups, order, positions, offsets,
                _work(load_library().fp8blk_group_rows_workspace_bytes(R, groups), ids))
    return RowGroups(order, positions, offsets)


def moe_combine(y, weights, positions, base=None):
    """out[t] = base[t] + sum_j weights[t,j] * y[positions[t,j]] in bf16;
    slots with position -1 add nothing."""
    slots = weights.shape
    if not (len(slots) == 2 and y.dim() == 2 and
            _plain(y.get_device(), (y, torch.bfloat16, y.shape), (weights, torch.float32, slots),
                   (positions, torch.int32, slots), (base, torch.bfloat16, (slots[0], y.shape[1])))):
        _combine_in(y, weights, positions, base)
        _same_device(y, weights, positions, base)
    out = y.new_empty((weights.shape[0], y.shape[1]))
    _combine_call(y, weights, positions, base, out)
    return out


def moe_combine_backward(d_out, y, weights, positions, offsets):
    """(d_y, d_weights) of moe_combine; the last entry of offsets is the number
    of y's rows in use (rows past it get 0).  positions names each row in use
    once, as group_rows gives them: one that no slot names is left unwritten."""
    _combine_back_in(d_out, y, weights, positions, offsets)
    _same_device(d_out, y, weights, positions, offsets)
    d_y, d_weights = torch.empty_like(y), torch.empty_like(weights)
    _combine_back_call(d_out, y, weights, positions, offsets, d_y, d_weights)
    return d_y, d_weights


def lora_add(base, x, a, b, ids, scale=None, groups=None, out=None):
    """out = base + scale[g] * (x a[g]^T) b[g]^T, g = ids[t] the row's adapter
    (none outside [0, L)); ``out`` may be base (in place).  ``groups`` =
    group_rows(ids, L) saves listing the rows again in every projection."""
    T, K = x.shape
    L, r, N = a.shape[0], a.shape[1], b.shape[1]
    if out is None:
        out = x.new_empty((T, N))
    bf = torch.bfloat16
    if groups is None and _plain(x.get_device(), (x, bf, (T, K)), (a, bf, (L, r, K)),
                                 (b, bf, (L, N, r)), (ids, torch.int32, (T,)), (base, bf, (T, N)),
                                 (out, bf, (T, N)), (scale, torch.float32, (L,))):
        strides = N, K, N
    else:
        strides = _lora_in(base, x, a, b, ids, scale, groups, out)
    need = load_library().fp8blk_lora_add_workspace_bytes(T, K, r, L, groups is not None)
    _lora_call(base, x, a, b, ids, scale, groups, out, _work(need, x), strides)
    return out


def lora_linear(x, w_q, w_scale, a, b, ids, scale=None, groups=None):
    """The FP8 linear layer with the adapters of a batch's requests added."""
    y = linear(x, w_q, w_scale)
    return lora_add(y, x, a, b, ids, scale, groups, out=y)


def moe_experts(x, routing, gate_up_q, gate_up_s, down_q, down_s, base=None):
    """The routed experts of a mixture-of-experts layer: x's rows listed by
    expert and quantized, the gate/up product, SwiGLU, the down product, and
    the weighted sum back to the tokens, on top of ``base`` (the shared
    expert's output).  Scale formats as the weights'; the routing is that of x's
    rows over the weights' experts."""
    (T, k), E = routing.ids.shape, gate_up_q.shape[0]
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError(f"x has shape {tuple(x.shape)}, the routing is of {T} rows")
    if down_q.shape[0] != E or (routing.counts is not None and routing.counts.numel() != E):
        raise ValueError("the routing and the weights have different numbers of experts")
    if gate_up_q.shape[2] != x.shape[1]:
        raise ValueError("x and gate_up_q disagree on K")
    if gate_up_q.shape[1] != 2 * down_q.shape[2]:
        raise ValueError("gate_up_q's rows are not twice down_q's columns")
    if base is not None:
        _shape_eq(base, (T, down_q.shape[1]), "base")
    groups = group_rows(routing.ids, E)
    fmt = "ue8m0" if _is_e8m0(gate_up_s) else "float"
    # rows past the last used one belong to no expert; no product reads them
    x_q, x_s = act_quant_group(x.index_select(0, groups.order // k), fmt)
    h = grouped_block_gemm(x_q, x_s, gate_up_q, gate_up_s, groups.offsets)
    h_q, h_s = swiglu_act_quant(h, fmt)
    y = grouped_block_gemm(h_q, h_s, down_q, down_s, groups.offsets)
    return moe_combine(y, routing.weights, groups.positions, base)


# --------------------------------------------------------------------------
# gated projections in 16 bits

_HALF = {torch.bfloat16: 1, torch.float16: 2}      # FP8BLK_BF16, FP8BLK_F16
_HALF_TYPES = tuple(_HALF)
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}      # FP8BLK_SILU, ...


def _stream_of(t):
    """The current stream of t's device, which is the current one (checked)."""
    return _raw_stream(t.get_device()) if _raw_stream is not None else _stream()


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {tuple(ACTS)}, got {act!r}")
    return ACTS[act]


def factor_row(I):
    """Bytes of a row of factors that gated_linear saves for I outputs."""
    return -(-I // 4) * 24


def _gated_in(x, w, *more, factors=None):
    """Row stride of x, sizes (M, I, K); ``more`` are (tensor, name) of [M,I]."""
    if (not more and isinstance(x, torch.Tensor) and isinstance(w, torch.Tensor) and
            x.dim() == 2 and w.dim() == 2 and x.dtype in _HALF):
        (M, K), rows = x.shape, w.shape[0]
        if K and rows % 2 == 0 and _plain(x.get_device(), (x, x.dtype, (M, K)),
                                          (w, x.dtype, (rows, K))):
            return K, M, rows // 2, K
    ldx = _rows_2d(x, "x", _HALF_TYPES)
    _need(w, "w", (x.dtype,), 2)
    M, K = x.shape
    if w.shape[1] != K:
        raise ValueError("x and w disagree on K")
    if K == 0:
        raise ValueError("K must be positive")
    if w.shape[0] % 2:
        raise ValueError("w must hold 2I rows, the gates' first")
    I = w.shape[0] // 2
    for t, name in more:
        _need(t, name, (x.dtype,), 2)
        _shape_eq(t, (M, I), name)
    if factors is not None:
        _need(factors, "factors", (torch.uint8,), 2)
        _shape_eq(factors, (M, factor_row(I)), "factors")
    _same_device(x, w, factors, *(t for t, _ in more))
    return ldx, M, I, K


def _gated_call(x, ldx, w, act, M, I, K, h, factors, workspace):
    _check(load_library().fp8blk_gated_linear(
        x.data_ptr(), ldx, w.data_ptr(), _HALF[x.dtype], act, M, I, K, h.data_ptr(), _at(factors),
        _at(workspace), _bytes(workspace), _stream_of(x)), "fp8blk_gated_linear")


def fp8blk_gated_linear(x, w, act, h, factors, workspace=None):
    """The gated projections into h [M,I]; ``factors`` uint8 [M,factor_row(I)]
    (for the backward pass) may be None, x may be a column slice of a wider matrix.  ``workspace``
    holds fp8blk_gated_linear_workspace_bytes(M, I, K, x's row stride) bytes."""
    ldx, M, I, K = _gated_in(x, w, (h, "h"), factors=factors)
    _need_work(workspace)
    _same_device(x, workspace)
    _gated_call(x, ldx, w, _act(act), M, I, K, h, factors, workspace)


def _gated_back_call(d_h, x, ldx, w, factors, act, M, I, K, d_x, d_w, workspace):
    _check(load_library().fp8blk_gated_linear_backward(
        d_h.data_ptr(), x.data_ptr(), ldx, w.data_ptr(), _at(factors), _HALF[x.dtype], act, M, I, K,
        _at(d_x), _at(d_w), _at(workspace), _bytes(workspace), _stream_of(x)),
        "fp8blk_gated_linear_backward")


def fp8blk_gated_linear_backward(d_h, x, w, factors, act, d_x, d_w, workspace=None):
    """Gradients into d_x [M,K] and d_w [2I,K], either may be None; ``factors``
    None: the projections are computed again.  ``workspace`` holds
    fp8blk_gated_linear_backward_workspace_bytes(M, I, K, x's row stride,
    d_x wanted, d_w wanted) bytes."""
    ldx, M, I, K = _gated_in(x, w, (d_h, "d_h"), factors=factors)
    for t, like, name in ((d_x, x, "d_x"), (d_w, w, "d_w")):
        if t is not None:
            _need(t, name, (x.dtype,), 2)
            _shape_eq(t, like.shape, name)
    _need_work(workspace)
    _same_device(x, d_x, d_w, workspace)
    _gated_back_call(d_h, x, ldx, w, factors, _act(act), M, I, K, d_x, d_w, workspace)


def gated_linear(x, w, act="silu", save=False):
    """h = act(x Wg^T) * (x Wu^T), w [2I,K] with the gate rows first, in x's type
    (bf16 or fp16).  With ``save`` also the factors that gated_linear_backward
    takes (bytes, 6 an output; without them it computes the projections again)."""
    ldx, M, I, K = _gated_in(x, w)
    act = _act(act)
    h = x.new_empty((M, I))
    factors = x.new_empty((M, factor_row(I)), dtype=torch.uint8) if save else None
    need = load_library().fp8blk_gated_linear_workspace_bytes(M, I, K, ldx)
    _gated_call(x, ldx, w, act, M, I, K, h, factors, _work(need, x))
    return (h, factors) if save else h


def gated_linear_backward(d_h, x, w, factors=None, act="silu", need_x=True, need_w=True):
    """(d_x, d_w) of gated_linear; None in the place of one that is not needed.
    Between d_h and the results stands dgu, the gradient of x W^T, rounded once to
    x's type: in fp16 it is infinite past 65504 and zero below 2^-25."""
    ldx, M, I, K = _gated_in(x, w, (d_h, "d_h"), factors=factors)
    act = _act(act)
    d_x = x.new_empty((M, K)) if need_x else None
    d_w = torch.empty_like(w) if need_w else None
    need = load_library().fp8blk_gated_linear_backward_workspace_bytes(M, I, K, ldx, bool(need_x),
                                                                       bool(need_w))
    _gated_back_call(d_h, x, ldx, w, factors, act, M, I, K, d_x, d_w, _work(need, x))
    return d_x, d_w


# --------------------------------------------------------------------------
# 4-bit weights

W4_GROUPS = (32, 64, 128)


class W4Weight(NamedTuple):
    """Weights W[n,k] = (q - z) * s in 4 bits, as w4_linear takes them."""
    codes: torch.Tensor          # [N, K/2] uint8: two codes q, the even k in the low half
    scale: torch.Tensor          # [N, K/group] in the weights' type: s
    zeros: torch.Tensor | None   # [N, K/group] uint8: z (None: 8)


def _w4_in(codes, scale, zeros):
    """Sizes (N, K, group)."""
    _need(codes, "codes", (torch.uint8,), 2)
    _need(scale, "scale", _HALF_TYPES, 2)
    N, K = codes.shape[0], 2 * codes.shape[1]
    groups = scale.shape[1]
    if scale.shape[0] != N or groups < 1 or K % groups or K // groups not in W4_GROUPS:
        raise ValueError(f"scale has shape {tuple(scale.shape)}, which is no scale per group of "
                         f"{W4_GROUPS} for codes of shape {tuple(codes.shape)}")
    if zeros is not None:
        _need(zeros, "zeros", (torch.uint8,), 2)
        _shape_eq(zeros, scale.shape, "zeros")
    return N, K, K // groups


def _w4_product_in(x, codes, scale, zeros):
    """Row stride of x, sizes (M, N, K, group)."""
    if (isinstance(x, torch.Tensor) and isinstance(codes, torch.Tensor) and
            isinstance(scale, torch.Tensor) and (zeros is None or isinstance(zeros, torch.Tensor)) and
            x.dim() == 2 and codes.dim() == 2 and scale.dim() == 2 and x.dtype in _HALF):
        (M, K), (N, groups) = x.shape, scale.shape
        if (groups and K % groups == 0 and K // groups in W4_GROUPS and
                _plain(x.get_device(), (x, x.dtype, (M, K)), (codes, torch.uint8, (N, K // 2)),
                       (scale, x.dtype, (N, groups)), (zeros, torch.uint8, (N, groups)))):
            return K, M, N, K, K // groups
    N, K, group = _w4_in(codes, scale, zeros)
    ldx = _rows_2d(x, "x", (scale.dtype,))
    if x.shape[1] != K:
        raise ValueError("x and codes disagree on K")
    _same_device(x, codes, scale, zeros)
    return ldx, x.shape[0], N, K, group


def _w4_quant_call(w, group, codes, scale, zeros):
    _check(load_library().fp8blk_w4_quant(
        w.data_ptr(), _HALF[w.dtype], w.shape[0], w.shape[1], group, codes.data_ptr(),
        scale.data_ptr(), _at(zeros), _stream_of(w)), "fp8blk_w4_quant")


def fp8blk_w4_quant(w, codes, scale, zeros):
    """Weights w [N,K] to 4 bits into codes, scale and (None: no zero points)
    zeros; the group is K over scale's columns."""
    N, K, group = _w4_in(codes, scale, zeros)
    _need(w, "w", (scale.dtype,), 2)
    _shape_eq(w, (N, K), "w")
    _same_device(w, codes, scale, zeros)
    _w4_quant_call(w, group, codes, scale, zeros)


def _w4_dequant_call(codes, scale, zeros, N, K, group, w):
    _check(load_library().fp8blk_w4_dequant(
        codes.data_ptr(), scale.data_ptr(), _at(zeros), _HALF[w.dtype], N, K, group, w.data_ptr(),
        _stream_of(w)), "fp8blk_w4_dequant")


def fp8blk_w4_dequant(codes, scale, zeros, w):
    """The weights that codes stand for into w [N,K] (scale's type)."""
    N, K, group = _w4_in(codes, scale, zeros)
    _need(w, "w", (scale.dtype,), 2)
    _shape_eq(w, (N, K), "w")
    _same_device(w, codes, scale, zeros)
    _w4_dequant_call(codes, scale, zeros, N, K, group, w)


def _w4_call(x, sizes, codes, scale, zeros, y, workspace):
    ldx, M, N, K, group = sizes
    _check(load_library().fp8blk_w4_linear(
        x.data_ptr(), ldx, codes.data_ptr(), scale.data_ptr(), _at(zeros), _HALF[x.dtype], group, M,
        N, K, y.data_ptr(), _at(workspace), _bytes(workspace), _stream_of(x)), "fp8blk_w4_linear")


def fp8blk_w4_linear(x, codes, scale, zeros, y, workspace=None):
    """y [M,N] = x W^T with 4-bit weights; zeros may be None, x a column slice of
    a wider matrix.  ``workspace`` holds fp8blk_w4_linear_workspace_bytes(M, N, K,
    x's row stride) bytes."""
    sizes = _w4_product_in(x, codes, scale, zeros)
    _need(y, "y", (x.dtype,), 2)
    _shape_eq(y, sizes[1:3], "y")
    _need_work(workspace)
    _same_device(x, y, workspace)
    _w4_call(x, sizes, codes, scale, zeros, y, workspace)


def _w4_half(N):
    if N % 2:
        raise ValueError("codes must hold 2I rows, the gates' first")
    return N // 2


def _w4_gated_call(x, sizes, codes, scale, zeros, act, h, workspace):
    ldx, M, N, K, group = sizes
    _check(load_library().fp8blk_w4_gated_linear(
        x.data_ptr(), ldx, codes.data_ptr(), scale.data_ptr(), _at(zeros), _HALF[x.dtype], group, act,
        M, N // 2, K, h.data_ptr(), _at(workspace), _bytes(workspace), _stream_of(x)),
        "fp8blk_w4_gated_linear")


def fp8blk_w4_gated_linear(x, codes, scale, zeros, act, h, workspace=None):
    """h [M,I] = act(x Wg^T) * (x Wu^T) with 4-bit weights [2I,K].  ``workspace``
    holds fp8blk_w4_gated_linear_workspace_bytes(M, I, K, x's row stride) bytes."""
    sizes = _w4_product_in(x, codes, scale, zeros)
    _need(h, "h", (x.dtype,), 2)
    _shape_eq(h, (sizes[1], _w4_half(sizes[2])), "h")
    _need_work(workspace)
    _same_device(x, h, workspace)
    _w4_gated_call(x, sizes, codes, scale, zeros, _act(act), h, workspace)


def w4_quant(w, group=128, zeros=False):
    """Weights [N,K] (bf16 or fp16) to 4 bits with a scale, and with ``zeros`` a
    zero point, per ``group`` of K: W4Weight(codes, scale, zeros)."""
    _need(w, "w", _HALF_TYPES, 2)
    _same_device(w)
    N, K = w.shape
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, got {group}")
    if K == 0 or K % group:
        raise ValueError(f"K must be a positive multiple of the group, got {K}")
    q = W4Weight(w.new_empty((N, K // 2), dtype=torch.uint8), w.new_empty((N, K // group)),
                 w.new_empty((N, K // group), dtype=torch.uint8) if zeros else None)
    _w4_quant_call(w, group, *q)
    return q


def w4_dequant(codes, scale, zeros=None):
    """The weights [N,K] that 4-bit codes stand for, in the scales' type."""
    N, K, group = _w4_in(codes, scale, zeros)
    _same_device(codes, scale, zeros)
    w = scale.new_empty((N, K))
    _w4_dequant_call(codes, scale, zeros, N, K, group, w)
    return w


def w4_linear(x, codes, scale, zeros=None):
    """y = x W^T with 4-bit weights (w4_linear(x, *w4_quant(w))), from one row,
    where it reads a quarter of a 16-bit weight's bytes, to many."""
    sizes = ldx, M, N, K, _ = _w4_product_in(x, codes, scale, zeros)
    y = x.new_empty((M, N))
    need = load_library().fp8blk_w4_linear_workspace_bytes(M, N, K, ldx)
    _w4_call(x, sizes, codes, scale, zeros, y, _work(need, x))
    return y


def w4_gated_linear(x, codes, scale, zeros=None, act="silu"):
    """gated_linear with 4-bit weights [2I,K], the gate rows first: h [M,I]."""
    sizes = ldx, M, N, K, _ = _w4_product_in(x, codes, scale, zeros)
    h = x.new_empty((M, _w4_half(N)))
    need = load_library().fp8blk_w4_gated_linear_workspace_bytes(M, N // 2, K, ldx)
    _w4_gated_call(x, sizes, codes, scale, zeros, _act(act), h, _work(need, x))
    return h
