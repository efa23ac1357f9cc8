"""Thin Python binding of the C ABI in include/nvfp4.h (ctypes; marshalling only).

Every function here checks tensor placement, dtype, shape and contiguity,
allocates outputs with torch (device memory is torch's job), passes raw
device pointers and the current HIP stream to libnvfp4.so, and raises
NVFP4Error on a non-zero status.  All arithmetic runs in the library's HIP
kernels; there is no fallback: without the built library (or without a GPU)
these functions raise.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

NVFP4_OK, NVFP4_ERR_NULL, NVFP4_ERR_SHAPE, NVFP4_ERR_ALIGN, NVFP4_ERR_DTYPE, NVFP4_ERR_HIP, NVFP4_ERR_SCRATCH = range(7)
SCRATCH_BYTES = 4 << 20  # NVFP4_SCRATCH_BYTES
NVFP4_F32, NVFP4_BF16 = 0, 1
PATH_AUTO, PATH_SKINNY, PATH_TILED = 0, 1, 2
# kernel selectors of nvfp4_gemm_ex (and values of nvfp4_gemm_dispatch)
(KERNEL_GEMV_FP4, KERNEL_GEMV_FLAT, KERNEL_M16, KERNEL_SKINNY256, KERNEL_SKINNY16,
 KERNEL_TILED_PERSISTENT, KERNEL_TILED, KERNEL_M16_STREAM) = range(3, 11)
KERNEL_NAMES = {KERNEL_GEMV_FP4: "gemv_fp4_kernel", KERNEL_GEMV_FLAT: "gemv_flat_kernel", KERNEL_M16: "gemm_m16_kernel",
                KERNEL_SKINNY256: "gemm_skinny256_kernel", KERNEL_SKINNY16: "gemm_skinny_kernel",
                KERNEL_TILED_PERSISTENT: "gemm_wg_tiled_kernel", KERNEL_TILED: "gemm_tiled_kernel",
                KERNEL_M16_STREAM: "gemm_m16_stream_kernel"}

EXPORTS = ("nvfp4_abi_version", "nvfp4_act_global_scale", "nvfp4_delta_commit", "nvfp4_delta_commit_counts",
           "nvfp4_delta_rule", "nvfp4_delta_rule_workspace_bytes", "nvfp4_delta_tree", "nvfp4_gemm",
           "nvfp4_gemm_dispatch", "nvfp4_gemm_ex",
           "nvfp4_gemm_quantize_output", "nvfp4_gemm_scratch", "nvfp4_gemm_workspace_bytes", "nvfp4_gemm_ws",
           "nvfp4_kv_append", "nvfp4_kv_append_rope", "nvfp4_kv_attention", "nvfp4_kv_attention_workspace_bytes", "nvfp4_kv_compact",
           "nvfp4_kv_fork", "nvfp4_kv_fp8_decode", "nvfp4_kv_fp8_encode", "nvfp4_kv_resize",
           "nvfp4_quantize_act",
           "nvfp4_quantize_gemm", "nvfp4_quantize_gemm_dynamic", "nvfp4_quantize_weights", "nvfp4_status_string",
           "nvfp4_stream_read", "nvfp4_token_logprobs", "nvfp4_token_logprobs_workspace_bytes",
           "nvfp4_tree_accept",
           "nvfp4_tree_verify")

_lib: Optional[ctypes.CDLL] = None


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


def load() -> ctypes.CDLL:
    """Loads libnvfp4.so and declares the signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing; build it with `python -m nvfp4_w4a4_block_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.nvfp4_quantize_weights.argtypes = [p, i32, i64, i64, p, p, p, p]
    lib.nvfp4_quantize_act.argtypes = [p, i32, i64, i64, p, p, p, p]
    lib.nvfp4_gemm.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, i32, p]
    lib.nvfp4_gemm_ex.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, i32, i32, p]
    lib.nvfp4_gemm_ws.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, i32, p, i64, p]
    lib.nvfp4_gemm_scratch.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, i32, p]
    lib.nvfp4_gemm_quantize_output.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, i32, p, p, p, p]
    lib.nvfp4_gemm_workspace_bytes.argtypes = [i64, i64, i64]
    lib.nvfp4_gemm_workspace_bytes.restype = i64
    lib.nvfp4_gemm_dispatch.argtypes = [i64, i64, i64, i64]
    lib.nvfp4_stream_read.argtypes = [p, i64, p, i64, p, ctypes.c_uint32, p]
    lib.nvfp4_gemm_dispatch.restype = i32
    lib.nvfp4_quantize_gemm.argtypes = [i64, i64, i64, p, i32, p, p, p, p, p, i32, p, p, p]
    lib.nvfp4_quantize_gemm_dynamic.argtypes = [i64, i64, i64, p, i32, p, p, p, p, p, i32, p, p, p]
    lib.nvfp4_tree_accept.argtypes = [i64, p, p, p, p, p]
    lib.nvfp4_kv_fp8_encode.argtypes = [p, i32, i64, p, p, p]
    lib.nvfp4_act_global_scale.argtypes = [p, i32, i64, i64, p, p]
    lib.nvfp4_kv_fp8_decode.argtypes = [p, i64, p, p, i32, p]
    lib.nvfp4_tree_verify.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, p, p, p, p, p, p]
    f32 = ctypes.c_float
    lib.nvfp4_kv_append.argtypes = [i64] * 7 + [p, p, i32, i64, i64, p, p, p, p, i64, p, p, p, p]
    lib.nvfp4_kv_attention_workspace_bytes.argtypes = [i64] * 7 + [i32]
    lib.nvfp4_kv_attention_workspace_bytes.restype = i64
    lib.nvfp4_kv_attention.argtypes = [i64] * 8 + [p, i32, i64, f32, p, p, p, p, i64, p, p, p, p, p, p, p, i64, p]
    lib.nvfp4_kv_compact.argtypes = [i64] * 8 + [p, p, i64, i64, p, p, p, p, p]
    lib.nvfp4_kv_resize.argtypes = [i64] * 5 + [p] * 8
    lib.nvfp4_kv_fork.argtypes = [i64] * 5 + [p] * 9 + [i64] * 3 + [p, p, i64, i64, p]
    lib.nvfp4_kv_append_rope.argtypes = [i64] * 9 + [p, p, p, i32, i64, i64, i64, p, ctypes.c_double, i32, p, p, p, p, i64,
                                                     p, p, p, p, p, p]
    lib.nvfp4_delta_rule_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.nvfp4_delta_rule_workspace_bytes.restype = i64
    lib.nvfp4_delta_rule.argtypes = [i64] * 7 + [p, p, p, i32, i64, i64, i64, p, p, f32, f32, p, p, p, p, p, p, i64, p]
    lib.nvfp4_delta_tree.argtypes = [i64] * 7 + [p, p, p, i32, i64, i64, i64, p, p, f32, f32, p, p, p, p, p, p, p, p]
    lib.nvfp4_delta_commit.argtypes = [i64] * 8 + [p] * 8
    lib.nvfp4_delta_commit_counts.argtypes = [i64] * 8 + [p] * 9
    lib.nvfp4_token_logprobs_workspace_bytes.argtypes = [i64] * 3 + [i32]
    lib.nvfp4_token_logprobs_workspace_bytes.restype = i64
    lib.nvfp4_token_logprobs.argtypes = [i64] * 3 + [p, i32, i64, p, p, p, p, p, p, i64, p]
    for f in ("nvfp4_kv_append_rope", "nvfp4_delta_rule", "nvfp4_delta_tree", "nvfp4_delta_commit",
              "nvfp4_delta_commit_counts", "nvfp4_token_logprobs", "nvfp4_kv_append", "nvfp4_kv_attention", "nvfp4_kv_compact", "nvfp4_kv_resize", "nvfp4_kv_fork",
              "nvfp4_quantize_weights", "nvfp4_quantize_act", "nvfp4_gemm", "nvfp4_gemm_ex", "nvfp4_gemm_ws",
              "nvfp4_gemm_scratch",
              "nvfp4_gemm_quantize_output",
              "nvfp4_quantize_gemm", "nvfp4_tree_accept", "nvfp4_tree_verify", "nvfp4_kv_fp8_encode",
              "nvfp4_kv_fp8_decode", "nvfp4_act_global_scale", "nvfp4_stream_read"):
        getattr(lib, f).restype = i32
    lib.nvfp4_status_string.argtypes = [i32]
    lib.nvfp4_status_string.restype = ctypes.c_char_p
    lib.nvfp4_abi_version.argtypes = []
    lib.nvfp4_abi_version.restype = i32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().nvfp4_status_string(status).decode()


def _dt(t: torch.dtype) -> int:
    if t == torch.float32:
        return NVFP4_F32
    if t == torch.bfloat16:
        return NVFP4_BF16
    raise TypeError(f"unsupported dtype {t} (float32 or bfloat16)")


def _dev(*ts: torch.Tensor) -> torch.device:
    dev = ts[0].device
    for t in ts:
        if t.device.type != "cuda" or t.device != dev:
            raise ValueError("all tensors must be on the same GPU")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    return dev


# The raw handle without a Stream object around it, where torch offers it (2 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: torch.device) -> int:
    return _raw_stream(dev.index) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _check(status: int, where: str) -> None:
    if status != NVFP4_OK:
        raise NVFP4Error(status, where)


def nvfp4_quantize_weights(w: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """w [N, K] float32/bfloat16 -> (codes uint8 [N, K/2], scales uint8 [N, K/16], g_w float32 [1])."""
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    dev = _dev(w)
    N, K = w.shape
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=dev)
    g = torch.empty((1,), dtype=torch.float32, device=dev)
    _check(load().nvfp4_quantize_weights(w.data_ptr(), _dt(w.dtype), N, K, codes.data_ptr(),
                                         scales.data_ptr(), g.data_ptr(), _stream(dev)),
           "nvfp4_quantize_weights")
    return codes, scales, g


def nvfp4_quantize_act(a: torch.Tensor, g_a: torch.Tensor, codes: Optional[torch.Tensor] = None,
                       scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """a [M, K] float32/bfloat16 with device decode scale g_a [1] -> (codes [M, K/2], scales [M, K/16])."""
    if a.dim() != 2:
        raise ValueError("a must be [M, K]")
    if g_a.dtype != torch.float32 or g_a.numel() != 1:
        raise ValueError("g_a must be a float32 tensor of one element")
    dev = _dev(a, g_a)
    M, K = a.shape
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
    _dev(a, codes, scales)
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or \
            codes.numel() != M * (K // 2) or scales.numel() != M * (K // 16):
        raise ValueError("codes/scales must be uint8 of [M, K/2] / [M, K/16] elements")
    _check(load().nvfp4_quantize_act(a.data_ptr(), _dt(a.dtype), M, K, g_a.data_ptr(),
                                     codes.data_ptr(), scales.data_ptr(), _stream(dev)),
           "nvfp4_quantize_act")
    return codes, scales


_gemm_workspaces: dict = {}


def gemm_workspace(M: int, K: int, N: int, dev: torch.device) -> Optional[torch.Tensor]:
    """A zeroed workspace of at least nvfp4_gemm_workspace_bytes(M, K, N) bytes on `dev`, or None
    when the product needs none.  Cached per device and grown when too small; every call leaves
    its counters zero, so it is zeroed only when allocated.  Shared by the calls of this module:
    keep them on one stream, or pass a workspace of your own."""
    need = int(load().nvfp4_gemm_workspace_bytes(M, K, N))
    if need <= 0:
        return None
    ws = _gemm_workspaces.get(dev)
    if ws is None or ws.numel() < need:
        ws = _gemm_workspaces[dev] = torch.zeros((need,), dtype=torch.uint8, device=dev)
    return ws


def gemm_dispatch(M: int, K: int, N: int, workspace_bytes: int = 0) -> int:
    """The kernel selector (KERNEL_*) the automatic path runs for an (M, K, N) product with a
    workspace of that size (nvfp4_gemm_dispatch); 0 for an empty or invalid product."""
    return int(load().nvfp4_gemm_dispatch(M, K, N, workspace_bytes))


def nvfp4_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, g_a: torch.Tensor,
               w_codes: torch.Tensor, w_scales: torch.Tensor, g_w: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               path: int = PATH_AUTO, workspace=None) -> torch.Tensor:
    """NVFP4 W4A4 product: out [M, N] = dequant(A) @ dequant(W)^T, fp32 accumulation.
    workspace: None (nvfp4_gemm_ex with `path`), "auto" (gemm_workspace(), nvfp4_gemm_ws) or a
    uint8 device tensor (nvfp4_gemm_ws; zero before its first use)."""
    if a_codes.dim() != 2 or w_codes.dim() != 2:
        raise ValueError("codes must be 2-D")
    M, K2 = a_codes.shape
    N = w_codes.shape[0]
    K = 2 * K2
    if w_codes.shape[1] != K2 or a_scales.shape != (M, K // 16) or w_scales.shape != (N, K // 16):
        raise ValueError("inconsistent operand shapes")
    for t in (a_codes, a_scales, w_codes, w_scales):
        if t.dtype != torch.uint8:
            raise ValueError("codes and scales must be uint8")
    for g in (g_a, g_w):
        if g.dtype != torch.float32 or g.numel() != 1:
            raise ValueError("tensor scales must be float32 tensors of one element")
    dev = _dev(a_codes, a_scales, g_a, w_codes, w_scales, g_w)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    elif out.shape != (M, N) or out.dtype != out_dtype:
        raise ValueError("out must be [M, N] of out_dtype")
    _dev(a_codes, out)
    if workspace is None:
        _check(load().nvfp4_gemm_ex(M, K, N, a_codes.data_ptr(), a_scales.data_ptr(), g_a.data_ptr(),
                                    w_codes.data_ptr(), w_scales.data_ptr(), g_w.data_ptr(),
                                    out.data_ptr(), _dt(out_dtype), path, _stream(dev)),
               "nvfp4_gemm")
        return out
    if path != PATH_AUTO:
        raise ValueError("a workspace is used by the automatic path only")
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be None, "auto" or a uint8 tensor')
        workspace = gemm_workspace(M, K, N, dev)
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != dev or
                                  not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
    _check(load().nvfp4_gemm_ws(M, K, N, a_codes.data_ptr(), a_scales.data_ptr(), g_a.data_ptr(),
                                w_codes.data_ptr(), w_scales.data_ptr(), g_w.data_ptr(),
                                out.data_ptr(), _dt(out_dtype),
                                workspace.data_ptr() if workspace is not None else None,
                                workspace.numel() if workspace is not None else 0, _stream(dev)),
           "nvfp4_gemm_ws")
    return out


def nvfp4_gemm_quantize_output(a_codes: torch.Tensor, a_scales: torch.Tensor, g_a: torch.Tensor,
                               w_codes: torch.Tensor, w_scales: torch.Tensor, g_w: torch.Tensor,
                               g_y: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                               out: Optional[torch.Tensor] = None, y_codes: Optional[torch.Tensor] = None,
                               y_scales: Optional[torch.Tensor] = None
                               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """NVFP4 product whose output is also quantized with the device scale g_y [1]: returns
    (out [M, N], y_codes [M, N/2], y_scales [M, N/16])."""
    if a_codes.dim() != 2 or w_codes.dim() != 2:
        raise ValueError("codes must be 2-D")
    M, K2 = a_codes.shape
    N = w_codes.shape[0]
    K = 2 * K2
    if w_codes.shape[1] != K2 or a_scales.shape != (M, K // 16) or w_scales.shape != (N, K // 16):
        raise ValueError("inconsistent operand shapes")
    for t in (a_codes, a_scales, w_codes, w_scales):
        if t.dtype != torch.uint8:
            raise ValueError("codes and scales must be uint8")
    for g in (g_a, g_w, g_y):
        if g.dtype != torch.float32 or g.numel() != 1:
            raise ValueError("tensor scales must be float32 tensors of one element")
    dev = _dev(a_codes, a_scales, g_a, w_codes, w_scales, g_w, g_y)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    elif out.shape != (M, N) or out.dtype != out_dtype:
        raise ValueError("out must be [M, N] of out_dtype")
    if y_codes is None:
        y_codes = torch.empty((M, N // 2), dtype=torch.uint8, device=dev)
    if y_scales is None:
        y_scales = torch.empty((M, N // 16), dtype=torch.uint8, device=dev)
    if y_codes.dtype != torch.uint8 or y_scales.dtype != torch.uint8 or \
            y_codes.numel() != M * (N // 2) or y_scales.numel() != M * (N // 16):
        raise ValueError("y_codes/y_scales must be uint8 of [M, N/2] / [M, N/16] elements")
    _dev(a_codes, out, y_codes, y_scales)
    _check(load().nvfp4_gemm_quantize_output(M, K, N, a_codes.data_ptr(), a_scales.data_ptr(), g_a.data_ptr(),
                                             w_codes.data_ptr(), w_scales.data_ptr(), g_w.data_ptr(),
                                             out.data_ptr(), _dt(out_dtype), g_y.data_ptr(), y_codes.data_ptr(),
                                             y_scales.data_ptr(), _stream(dev)),
           "nvfp4_gemm_quantize_output")
    return out, y_codes, y_scales


def nvfp4_quantize_gemm(a: torch.Tensor, g_a: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                        g_w: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None, a_codes: Optional[torch.Tensor] = None,
                        a_scales: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Raw activations a [M, K] (float32/bfloat16) with device scale g_a [1] times the NVFP4
    weights: returns (out [M, N], a_codes [M, K/2], a_scales [M, K/16])."""
    if a.dim() != 2 or w_codes.dim() != 2:
        raise ValueError("a and w_codes must be 2-D")
    M, K = a.shape
    N = w_codes.shape[0]
    if w_codes.shape[1] != K // 2 or w_scales.shape != (N, K // 16):
        raise ValueError("inconsistent operand shapes")
    if w_codes.dtype != torch.uint8 or w_scales.dtype != torch.uint8:
        raise ValueError("codes and scales must be uint8")
    for g in (g_a, g_w):
        if g.dtype != torch.float32 or g.numel() != 1:
            raise ValueError("tensor scales must be float32 tensors of one element")
    dev = _dev(a, g_a, w_codes, w_scales, g_w)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    elif out.shape != (M, N) or out.dtype != out_dtype:
        raise ValueError("out must be [M, N] of out_dtype")
    if a_codes is None:
        a_codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if a_scales is None:
        a_scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
    if a_codes.dtype != torch.uint8 or a_scales.dtype != torch.uint8 or \
            a_codes.numel() != M * (K // 2) or a_scales.numel() != M * (K // 16):
        raise ValueError("a_codes/a_scales must be uint8 of [M, K/2] / [M, K/16] elements")
    _dev(a, out, a_codes, a_scales)
    _check(load().nvfp4_quantize_gemm(M, K, N, a.data_ptr(), _dt(a.dtype), g_a.data_ptr(),
                                      w_codes.data_ptr(), w_scales.data_ptr(), g_w.data_ptr(),
                                      out.data_ptr(), _dt(out_dtype), a_codes.data_ptr(),
                                      a_scales.data_ptr(), _stream(dev)),
           "nvfp4_quantize_gemm")
    return out, a_codes, a_scales


def nvfp4_quantize_gemm_dynamic(a: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, g_w: torch.Tensor,
                                out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                                a_codes: Optional[torch.Tensor] = None, a_scales: Optional[torch.Tensor] = None,
                                g_a: Optional[torch.Tensor] = None
                                ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Raw activations a [M, K] times the NVFP4 weights with the activations' tensor scale
    computed on the device: returns (out [M, N], a_codes, a_scales, g_a [1])."""
    if a.dim() != 2 or w_codes.dim() != 2:
        raise ValueError("a and w_codes must be 2-D")
    M, K = a.shape
    N = w_codes.shape[0]
    if w_codes.shape[1] != K // 2 or w_scales.shape != (N, K // 16):
        raise ValueError("inconsistent operand shapes")
    if w_codes.dtype != torch.uint8 or w_scales.dtype != torch.uint8:
        raise ValueError("codes and scales must be uint8")
    if g_w.dtype != torch.float32 or g_w.numel() != 1:
        raise ValueError("tensor scales must be float32 tensors of one element")
    dev = _dev(a, w_codes, w_scales, g_w)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    elif out.shape != (M, N) or out.dtype != out_dtype:
        raise ValueError("out must be [M, N] of out_dtype")
    if a_codes is None:
        a_codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    if a_scales is None:
        a_scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
    if g_a is None:
        g_a = torch.empty((1,), dtype=torch.float32, device=dev)
    if g_a.dtype != torch.float32 or g_a.numel() != 1:
        raise ValueError("g_a must be a float32 tensor of one element")
    if a_codes.dtype != torch.uint8 or a_scales.dtype != torch.uint8 or \
            a_codes.numel() != M * (K // 2) or a_scales.numel() != M * (K // 16):
        raise ValueError("a_codes/a_scales must be uint8 of [M, K/2] / [M, K/16] elements")
    _dev(a, out, a_codes, a_scales, g_a)
    _check(load().nvfp4_quantize_gemm_dynamic(M, K, N, a.data_ptr(), _dt(a.dtype), g_a.data_ptr(),
                                              w_codes.data_ptr(), w_scales.data_ptr(), g_w.data_ptr(),
                                              out.data_ptr(), _dt(out_dtype), a_codes.data_ptr(),
                                              a_scales.data_ptr(), _stream(dev)),
           "nvfp4_quantize_gemm_dynamic")
    return out, a_codes, a_scales, g_a


def _int32_vec(t: torch.Tensor, n: int, name: str) -> None:
    if t.dtype != torch.int32 or t.dim() != 1 or t.numel() != n:
        raise ValueError(f"{name} must be an int32 vector of {n} elements")


def nvfp4_tree_accept(parent: torch.Tensor, draft: torch.Tensor, greedy: torch.Tensor) -> torch.Tensor:
    """Greedy acceptance of a candidate tree: returns result int32 [3 + n] = (end node, accepted
    count L, bonus token, L path nodes, -1 padding)."""
    n = parent.numel()
    for t, name in ((parent, "parent"), (draft, "draft"), (greedy, "greedy")):
        _int32_vec(t, n, name)
    dev = _dev(parent, draft, greedy)
    result = torch.empty((3 + n,), dtype=torch.int32, device=dev)
    _check(load().nvfp4_tree_accept(n, parent.data_ptr(), draft.data_ptr(), greedy.data_ptr(),
                                    result.data_ptr(), _stream(dev)), "nvfp4_tree_accept")
    return result


_key_workspaces: dict = {}


def tree_key_workspace(dev: torch.device) -> torch.Tensor:
    """The argmax-key workspace of nvfp4_tree_verify for `dev` (1024 int64, zeroed once; every
    call leaves it zeroed).  Shared by the calls of this module: keep them on one stream, or
    pass a workspace of your own."""
    ws = _key_workspaces.get(dev)
    if ws is None:
        ws = _key_workspaces[dev] = torch.zeros((1024,), dtype=torch.int64, device=dev)
    return ws


def nvfp4_tree_verify(a_codes: torch.Tensor, a_scales: torch.Tensor, g_a: torch.Tensor,
                      w_codes: torch.Tensor, w_scales: torch.Tensor, g_w: torch.Tensor,
                      parent: torch.Tensor, draft: torch.Tensor, want_logits: bool = False,
                      keys: Optional[torch.Tensor] = None):
    """LM head over the M tree nodes plus greedy acceptance: returns (greedy int32 [M],
    result int32 [3 + M], logits fp32 [M, N] or None)."""
    M, K2 = a_codes.shape
    N = w_codes.shape[0]
    K = 2 * K2
    if w_codes.shape[1] != K2 or a_scales.shape != (M, K // 16) or w_scales.shape != (N, K // 16):
        raise ValueError("inconsistent operand shapes")
    _int32_vec(parent, M, "parent")
    _int32_vec(draft, M, "draft")
    dev = _dev(a_codes, a_scales, g_a, w_codes, w_scales, g_w, parent, draft)
    greedy = torch.empty((M,), dtype=torch.int32, device=dev)
    result = torch.empty((3 + M,), dtype=torch.int32, device=dev)
    if keys is None:
        keys = tree_key_workspace(dev)
    elif keys.dtype != torch.int64 or keys.numel() != 1024 or keys.device != dev:
        raise ValueError("keys must be 1024 int64 on the operands' device, zero on entry")
    logits = torch.empty((M, N), dtype=torch.float32, device=dev) if want_logits else None
    _check(load().nvfp4_tree_verify(M, K, N, a_codes.data_ptr(), a_scales.data_ptr(), g_a.data_ptr(),
                                    w_codes.data_ptr(), w_scales.data_ptr(), g_w.data_ptr(),
                                    parent.data_ptr(), draft.data_ptr(),
                                    logits.data_ptr() if logits is not None else None,
                                    greedy.data_ptr(), result.data_ptr(), keys.data_ptr(), _stream(dev)),
           "nvfp4_tree_verify")
    return greedy, result, logits


def nvfp4_kv_fp8_encode(x: torch.Tensor, scale: torch.Tensor, q: Optional[torch.Tensor] = None) -> torch.Tensor:
    """KV values x (float32/bfloat16, any shape, contiguous) with device decode scale [1] -> E4M3
    bytes (uint8, same shape)."""
    if scale.dtype != torch.float32 or scale.numel() != 1:
        raise ValueError("scale must be a float32 tensor of one element")
    dev = _dev(x, scale)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=dev)
    elif q.dtype != torch.uint8 or q.numel() != x.numel():
        raise ValueError("q must be uint8 with x's element count")
    _dev(x, q)
    _check(load().nvfp4_kv_fp8_encode(x.data_ptr(), _dt(x.dtype), x.numel(), scale.data_ptr(), q.data_ptr(),
                                      _stream(dev)), "nvfp4_kv_fp8_encode")
    return q


def nvfp4_kv_fp8_decode(q: torch.Tensor, scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """E4M3 bytes q (uint8) with device decode scale [1] -> values (out_dtype, same shape)."""
    if q.dtype != torch.uint8:
        raise ValueError("q must be uint8")
    if scale.dtype != torch.float32 or scale.numel() != 1:
        raise ValueError("scale must be a float32 tensor of one element")
    dev = _dev(q, scale)
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=dev)
    elif out.dtype != out_dtype or out.numel() != q.numel():
        raise ValueError("out must have q's element count and out_dtype")
    _dev(q, out)
    _check(load().nvfp4_kv_fp8_decode(q.data_ptr(), q.numel(), scale.data_ptr(), out.data_ptr(), _dt(out_dtype),
                                      _stream(dev)), "nvfp4_kv_fp8_decode")
    return out


def nvfp4_act_global_scale(a: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dynamic activation decode scale g_a = amax|a| / 2688 of a [M, K] float32/bfloat16 tensor,
    computed on the device -> float32 [1] (device)."""
    if a.dim() != 2:
        raise ValueError("a must be [M, K]")
    dev = _dev(a)
    if out is None:
        out = torch.empty((1,), dtype=torch.float32, device=dev)
    elif out.dtype != torch.float32 or out.numel() != 1:
        raise ValueError("out must be a float32 tensor of one element")
    M, K = a.shape
    _check(load().nvfp4_act_global_scale(a.data_ptr(), _dt(a.dtype), M, K, out.data_ptr(), _stream(dev)),
           "nvfp4_act_global_scale")
    return out


def nvfp4_stream_read(a: torch.Tensor, b: torch.Tensor, sink: Optional[torch.Tensor] = None,
                      magic: int = 0x9E3779B9) -> torch.Tensor:
    """Reads every byte of a and b once (the read-only streaming ceiling of nvfp4_stream_read);
    returns the sink (int32 [1] on the device, written only by a lane whose XOR fold of the words
    it read equals `magic`)."""
    dev = _dev(a, b)
    if sink is None:
        sink = torch.zeros((1,), dtype=torch.int32, device=dev)
    _dev(a, sink)
    _check(load().nvfp4_stream_read(a.data_ptr(), a.numel() * a.element_size(), b.data_ptr(),
                                    b.numel() * b.element_size(), sink.data_ptr(), magic, _stream(dev)),
           "nvfp4_stream_read")
    return sink


# Paged FP8 KV cache.  Pages are uint8 [P, H, page_size, D] per layer ([L, P, H, page_size, D] for
# all layers), tables int32 [B, W], lengths int32 [B]; include/nvfp4.h states the layout.
# A small call is bound by its host time (an append: 4 us for the launch, 5 for what is here), so the
# checks compare device indices and bound names.

_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(on: int, where: str, fn, *args) -> None:
    """Calls fn(*args, stream) with GPU `on` current and its current stream."""
    if on == _current_device() and _raw_stream is not None:
        status = fn(*args, _raw_stream(on))
    else:
        with torch.cuda.device(on):
            status = fn(*args, torch.cuda.current_stream(on).cuda_stream)
    if status != NVFP4_OK:
        raise NVFP4Error(status, where)


def _ints(on: int, names: str, *ts: torch.Tensor) -> None:
    for t in ts:
        if t.dtype is not _I32 or t.get_device() != on or not t.is_contiguous():
            raise ValueError(f"{names} must be contiguous int32 tensors on cuda:{on}")


def _kv_scale(on: int, k_scale: torch.Tensor, v_scale: torch.Tensor) -> None:
    if k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or k_scale.get_device() != on or \
            v_scale.get_device() != on or k_scale.numel() != 1 or v_scale.numel() != 1:
        raise ValueError(f"k_scale and v_scale must be float32 tensors of one element on cuda:{on}")


def _kv_pages(k_pages: torch.Tensor, v_pages: torch.Tensor, dim: int) -> Tuple[int, torch.Size, int, int]:
    """Checks a pair of page tensors of `dim` dimensions (same shape and strides, whole pages);
    returns their GPU and shape and the bytes from a layer to the next and from a page to the next."""
    on = k_pages.get_device()
    if k_pages.dtype is not _U8 or v_pages.dtype is not _U8 or on < 0 or v_pages.get_device() != on:
        raise ValueError("pages must be uint8 tensors on one GPU")
    shape = k_pages.shape
    dense = k_pages.is_contiguous() and v_pages.is_contiguous()
    if len(shape) != dim or shape != v_pages.shape or not (dense or k_pages.stride() == v_pages.stride()):
        raise ValueError("k_pages and v_pages must have the same shape "
                         + ("[L, P, H, page_size, D]" if dim == 5 else "[P, H, page_size, D]") + " and strides")
    P, H, page, D = shape[-4:]
    if dense:
        return on, shape, P * H * page * D if dim == 5 and shape[0] > 1 else 0, H * page * D
    st = k_pages.stride()
    if (st[-1] != 1 and D > 1) or (st[-2] != D and page > 1) or (st[-3] != page * D and H > 1):
        raise ValueError("a page must be contiguous [H, page_size, D]")
    return on, shape, st[0] if dim == 5 and shape[0] > 1 else 0, st[-4] if P > 1 else H * page * D


def _kv_rows(x: torch.Tensor, shape: torch.Size, on: int, name: str) -> int:
    """x of shape [B, M, heads, D] whose rows are contiguous; returns the values from a row to the next."""
    if x.get_device() != on:
        raise ValueError(f"{name} must be on cuda:{on}")
    B, M, H, D = shape
    if x.is_contiguous():
        return H * D
    sb, sm, sh, sd = x.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"the rows of {name} must be contiguous [heads, D]")
    row = sm if M > 1 else sb if B > 1 else H * D
    if B > 1 and M > 1 and sb != M * sm:
        raise ValueError(f"the rows of {name} must be equally spaced")
    return row


def nvfp4_kv_append(k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                    k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                    counts: Optional[torch.Tensor] = None) -> None:
    """Writes k and v [B, M, H, D] (float32/bfloat16; rows may be column ranges of a wider tensor) as
    E4M3 bytes at tokens lens[b] .. lens[b] + M - 1 (counts[b] of them) of the sequences' pages, which
    must not be shared (refs 1): a sequence cut back into a shared page goes on as a fork of itself."""
    on, (P, Hp, page, Dp), _, page_stride = _kv_pages(k_pages, v_pages, 4)
    shape, entries = k.shape, table.shape
    if len(shape) != 4 or shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must be [B, M, H, D] of one dtype")
    B, M, H, D = shape
    if H != Hp or D != Dp or len(entries) != 2 or entries[0] != B or lens.shape != (B,):
        raise ValueError("k, pages [P, H, page_size, D], table [B, W] and lens [B] do not fit together")
    _ints(on, "table and lens", table, lens)
    if counts is not None:
        _ints(on, "counts", counts)
        if counts.shape != (B,):
            raise ValueError("counts must be [B]")
    _kv_scale(on, k_scale, v_scale)
    _call(on, "nvfp4_kv_append", load().nvfp4_kv_append, B, M, H, D, page, P, entries[1], k.data_ptr(),
          v.data_ptr(), _dt(k.dtype), _kv_rows(k, shape, on, "k"), _kv_rows(v, shape, on, "v"), k_scale.data_ptr(),
          v_scale.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_stride, table.data_ptr(),
          lens.data_ptr(), counts.data_ptr() if counts is not None else None)


def nvfp4_kv_attention(q: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, k_pages: torch.Tensor,
                       v_pages: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                       parent: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                       sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None, want_lse: bool = False,
                       workspace: Optional[torch.Tensor] = None):
    """Attention of the nodes q [B, M, Hq, D] (float32/bfloat16) over one layer of the cache, in which
    the nodes' own keys and values already stand behind lens[b].  parent int32 [B, M]: drafted trees (M <=
    64); None: a chain.  sm_scale defaults to 1/sqrt(D).  Returns out [B, M, Hq, D] of q's dtype, or
    (out, lse float32 [B, M, Hq]) with want_lse.  workspace: uint8 scratch; None allocates it."""
    on, (P, H, page, Dp), _, page_stride = _kv_pages(k_pages, v_pages, 4)
    shape, entries = q.shape, table.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, M, Hq, D]")
    B, M, Hq, D = shape
    if D != Dp or H < 1 or Hq % H or len(entries) != 2 or entries[0] != B or lens.shape != (B,):
        raise ValueError("q, pages [P, H, page_size, D], table [B, W] and lens [B] do not fit together")
    _ints(on, "table and lens", table, lens)
    if parent is not None:
        _ints(on, "parent", parent)
        if parent.shape != (B, M):
            raise ValueError("parent must be [B, M]")
    if counts is not None:
        _ints(on, "counts", counts)
        if counts.shape != (B,):
            raise ValueError("counts must be [B]")
    _kv_scale(on, k_scale, v_scale)
    stride = _kv_rows(q, shape, on, "q")
    dt, W = _dt(q.dtype), entries[1]
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.shape != shape or out.dtype != q.dtype or out.get_device() != on or not out.is_contiguous():
        raise ValueError("out must be a contiguous [B, M, Hq, D] of q's dtype on its GPU")
    lse = k_scale.new_empty((B, M, Hq)) if want_lse else None
    lib = load()
    if workspace is None:
        if on == _current_device():
            need = lib.nvfp4_kv_attention_workspace_bytes(B, M, Hq, H, D, page, W, dt)
        else:
            with torch.cuda.device(on):
                need = lib.nvfp4_kv_attention_workspace_bytes(B, M, Hq, H, D, page, W, dt)
        workspace = k_pages.new_empty((need,)) if need else None
    elif workspace.dtype is not _U8 or workspace.get_device() != on or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
    _call(on, "nvfp4_kv_attention", lib.nvfp4_kv_attention, B, M, Hq, H, D, page, P, W, q.data_ptr(), dt, stride,
          1.0 / math.sqrt(D) if sm_scale is None else sm_scale, k_scale.data_ptr(), v_scale.data_ptr(),
          k_pages.data_ptr(), v_pages.data_ptr(), page_stride, table.data_ptr(), lens.data_ptr(),
          parent.data_ptr() if parent is not None else None, counts.data_ptr() if counts is not None else None,
          out.data_ptr(), lse.data_ptr() if lse is not None else None,
          workspace.data_ptr() if workspace is not None else None,
          workspace.numel() if workspace is not None else 0)
    return (out, lse) if want_lse else out


def nvfp4_kv_compact(k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                     result: torch.Tensor, new_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Moves the accepted path of each sequence's tree to the front in all layers of pages [L, P, H,
    page_size, D]; result int32 [B, 3 + M]: rows of nvfp4_tree_accept / nvfp4_tree_verify.  Returns
    new_lens int32 [B] = lens + 1 + accepted (a tensor of its own: lens is not changed)."""
    on, (L, P, H, page, D), layer_stride, page_stride = _kv_pages(k_pages, v_pages, 5)
    entries, paths = table.shape, result.shape
    if len(entries) != 2 or len(paths) != 2 or lens.shape != entries[:1] or paths[0] != entries[0]:
        raise ValueError("table [B, W], lens [B] and result [B, 3 + M] do not fit together")
    B, W = entries
    _ints(on, "table, lens and result", table, lens, result)
    if new_lens is None:
        new_lens = torch.empty_like(lens)
    else:
        _ints(on, "new_lens", new_lens)
        if new_lens.shape != lens.shape:
            raise ValueError("new_lens must be [B]")
    _call(on, "nvfp4_kv_compact", load().nvfp4_kv_compact, L, B, paths[1] - 3, H, D, page, P, W,
          k_pages.data_ptr(), v_pages.data_ptr(), layer_stride, page_stride, table.data_ptr(),
          lens.data_ptr(), result.data_ptr(), new_lens.data_ptr())
    return new_lens


def kv_pool(seqs: int, width: int, pages: int, dev) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """An empty page pool on `dev`: (table [seqs, width], held [seqs], refs [pages], free_list [1 +
    pages]); pages are handed out in ascending order."""
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=dev)
    held = torch.zeros((seqs,), dtype=torch.int32, device=dev)
    refs = torch.zeros((pages,), dtype=torch.int32, device=dev)
    return table, held, refs, torch.arange(pages, -1, -1, dtype=torch.int32, device=dev)


def _pool(table: torch.Tensor, held: torch.Tensor, refs: torch.Tensor,
          free_list: torch.Tensor) -> Tuple[int, int, int, int]:
    """Checks a pool; returns its GPU, sequences, width and pages."""
    on, shape, seqs, pages = table.get_device(), table.shape, held.shape, refs.shape
    if on < 0:
        raise ValueError("the page pool must be on a GPU")
    _ints(on, "table, held, refs and free_list", table, held, refs, free_list)
    if len(shape) != 2 or seqs != shape[:1] or len(pages) != 1 or free_list.shape != (pages[0] + 1,):
        raise ValueError("table [S, W], held [S], refs [P] and free_list [1 + P] do not fit together")
    return on, shape[0], shape[1], pages[0]


def _shortage(on: int, shortage: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    if shortage is None:
        return like.new_empty((1,))
    _ints(on, "shortage", shortage)
    if shortage.numel() != 1:
        raise ValueError("shortage must have one element")
    return shortage


def nvfp4_kv_resize(table: torch.Tensor, held: torch.Tensor, refs: torch.Tensor, free_list: torch.Tensor,
                    page_size: int, seqs: torch.Tensor, tokens: torch.Tensor,
                    shortage: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Lets each sequence of seqs int32 [n] hold the pages of tokens int32 [n] tokens (0 frees it).  One
    cut back into a page that others hold too must not be appended to: fork it to an unused one first.
    Returns shortage int32 [1]: 0, or how many pages were missing (then nothing is changed)."""
    on, S, W, P = _pool(table, held, refs, free_list)
    _ints(on, "seqs and tokens", seqs, tokens)
    entries = seqs.shape
    if len(entries) != 1 or tokens.shape != entries:
        raise ValueError("seqs and tokens must be [n]")
    shortage = _shortage(on, shortage, table)
    _call(on, "nvfp4_kv_resize", load().nvfp4_kv_resize, entries[0], S, W, P, page_size,
          table.data_ptr(), held.data_ptr(), refs.data_ptr(), free_list.data_ptr(), seqs.data_ptr(),
          tokens.data_ptr(), shortage.data_ptr())
    return shortage


def nvfp4_kv_fork(table: torch.Tensor, held: torch.Tensor, refs: torch.Tensor, free_list: torch.Tensor,
                  k_pages: torch.Tensor, v_pages: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
                  tokens: torch.Tensor, shortage: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Sequence dst[i] becomes the first tokens[i] committed tokens of src[i] (int32 [n] each): whole pages are
    shared, a partial one is copied in all layers of pages [L, P, H, page_size, D], what dst held is
    given up.  Returns shortage as nvfp4_kv_resize."""
    on, S, W, pages = _pool(table, held, refs, free_list)
    at, (L, P, H, page, D), layer_stride, page_stride = _kv_pages(k_pages, v_pages, 5)
    if at != on or P != pages:
        raise ValueError("pages must be [L, P, H, page_size, D] of the pool's P pages, on its GPU")
    _ints(on, "src, dst and tokens", src, dst, tokens)
    entries = src.shape
    if len(entries) != 1 or dst.shape != entries or tokens.shape != entries:
        raise ValueError("src, dst and tokens must be [n]")
    shortage = _shortage(on, shortage, table)
    n = entries[0]
    moves = table.new_empty((3 * n,))
    _call(on, "nvfp4_kv_fork", load().nvfp4_kv_fork, n, S, W, P, page, table.data_ptr(), held.data_ptr(),
          refs.data_ptr(), free_list.data_ptr(), src.data_ptr(), dst.data_ptr(), tokens.data_ptr(),
          shortage.data_ptr(), moves.data_ptr(), L, H, D, k_pages.data_ptr(), v_pages.data_ptr(), layer_stride,
          page_stride)
    return shortage


def rope_frequencies(rotary: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained: int = 8192, fast: float = 32.0, slow: float = 1.0,
                     device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq float64 [rotary / 2] on `device`, rope_scale) for nvfp4_kv_append_rope.  scaling stretches a
    context of `trained` tokens by `factor`: "none"; "linear" (positions divided by it); "ntk" (a larger base, so
    that the slowest pair alone is stretched in full); "yarn" (pairs that turn more than `fast` times within the
    trained length stay, those that turn less than `slow` times are stretched in full, the others by a part
    between; rotated values times 0.1 ln factor + 1)."""
    if rotary < 16 or rotary % 16 or not 1.0 < base < math.inf or not 1.0 <= factor < math.inf or \
            not 1 <= trained < math.inf or not math.inf > fast > slow > 0.0:
        raise ValueError("rotary must be a multiple of 16, base above 1, factor at least 1, fast above slow above 0, "
                         "all finite")
    if scaling == "ntk":
        base *= factor ** (rotary / (rotary - 2))
    elif scaling not in ("none", "linear", "yarn"):
        raise ValueError("scaling must be none, linear, ntk or yarn")
    f = float(base) ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        # the pair that turns n times within the trained length; those between are mixed by their index
        at = [rotary * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary - 1)
        part = ((torch.arange(rotary // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - part) + f / factor * part
        scale = 0.1 * math.log(factor) + 1.0
    return f.to(device), scale


def nvfp4_kv_append_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, inv_freq: torch.Tensor,
                         k_scale: torch.Tensor, v_scale: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                         table: torch.Tensor, lens: torch.Tensor, parent: Optional[torch.Tensor] = None,
                         counts: Optional[torch.Tensor] = None, interleaved: bool = False, rope_scale: float = 1.0,
                         q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """nvfp4_kv_append with rotary positions: keys k [B, M, H, D] are turned on the way into the cache, the
    queries q [B, M, Hq, D] into q_out (returned; it may be a contiguous q).  inv_freq float64 [R / 2]: radians
    per position of the first R values' pairs (rope_frequencies).  parent int32 [B, M]: drafted trees, whose
    nodes stand at lens[b] + depth; None: a chain."""
    on, (P, Hp, page, Dp), _, page_stride = _kv_pages(k_pages, v_pages, 4)
    shape, rows, entries = q.shape, k.shape, table.shape
    if len(shape) != 4 or len(rows) != 4 or rows != v.shape or not q.dtype == k.dtype == v.dtype:
        raise ValueError("q must be [B, M, Hq, D], k and v [B, M, H, D], all of one dtype")
    B, M, Hq, D = shape
    H = rows[2]
    if rows != (B, M, Hp, Dp) or D != Dp or len(entries) != 2 or entries[0] != B or lens.shape != (B,):
        raise ValueError("q, k, pages [P, H, page_size, D], table [B, W] and lens [B] do not fit together")
    _ints(on, "table and lens", table, lens)
    if parent is not None:
        _ints(on, "parent", parent)
        if parent.shape != (B, M):
            raise ValueError("parent must be [B, M]")
    if counts is not None:
        _ints(on, "counts", counts)
        if counts.shape != (B,):
            raise ValueError("counts must be [B]")
    _kv_scale(on, k_scale, v_scale)
    if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != on or inv_freq.dim() != 1 or \
            not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous float64 [R / 2] on cuda:{on}")
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif q_out.shape != shape or q_out.dtype != q.dtype or q_out.get_device() != on or not q_out.is_contiguous():
        raise ValueError("q_out must be a contiguous [B, M, Hq, D] of q's dtype on its GPU")
    _call(on, "nvfp4_kv_append_rope", load().nvfp4_kv_append_rope, B, M, Hq, H, D, 2 * inv_freq.shape[0], page, P,
          entries[1], q.data_ptr(), k.data_ptr(), v.data_ptr(), _dt(q.dtype), _kv_rows(q, shape, on, "q"),
          _kv_rows(k, rows, on, "k"), _kv_rows(v, rows, on, "v"), inv_freq.data_ptr(), rope_scale, interleaved,
          k_scale.data_ptr(), v_scale.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_stride,
          table.data_ptr(), lens.data_ptr(), parent.data_ptr() if parent is not None else None,
          counts.data_ptr() if counts is not None else None, q_out.data_ptr())
    return q_out


# Gated delta rule.  States are float32 [S, H, Dv, Dk] per layer ([L, S, H, Dv, Dk] for all layers).


def _floats(on: int, shape, name: str, t: torch.Tensor) -> None:
    if t.dtype is not _F32 or t.get_device() != on or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 {list(shape)} on cuda:{on}")


def _delta_rows(q, k, v, g, beta, states, src, counts, out):
    """Checks a step's rows and slots; returns the GPU, the shape arguments, the rows' arguments and out."""
    on, rows, values, slots = states.get_device(), k.shape, v.shape, states.shape
    if on < 0 or states.dtype is not _F32 or len(slots) != 4 or not states.is_contiguous():
        raise ValueError("states must be a contiguous float32 [S, H, Dv, Dk] on a GPU")
    if len(rows) != 4 or q.shape != rows or len(values) != 4 or not q.dtype == k.dtype == v.dtype:
        raise ValueError("q and k must be [B, M, Hk, Dk], v [B, M, H, Dv], all of one dtype")
    B, M, Hk, Dk = rows
    S, H, Dv, _ = slots
    if values != (B, M, H, Dv) or slots[3] != Dk or Hk < 1 or H % Hk or src.shape != (B,):
        raise ValueError("q, k, v, states [S, H, Dv, Dk] and src [B] do not fit together")
    _ints(on, "src", src)
    if counts is not None:
        _ints(on, "counts", counts)
        if counts.shape != (B,):
            raise ValueError("counts must be [B]")
    _floats(on, (B, M, H), "g", g)
    _floats(on, (B, M, H), "beta", beta)
    if out is None:
        out = torch.empty_like(v, memory_format=torch.contiguous_format)
    elif out.shape != values or out.dtype != v.dtype or out.get_device() != on or not out.is_contiguous():
        raise ValueError("out must be a contiguous [B, M, H, Dv] of v's dtype on its GPU")
    return on, (B, M, Hk, H, Dk, Dv, S), (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _dt(q.dtype), _kv_rows(q, rows, on, "q"), _kv_rows(k, rows, on, "k"),
        _kv_rows(v, values, on, "v"), g.data_ptr(), beta.data_ptr()), out


def nvfp4_delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                     states: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
                     counts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     norm_eps: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gated delta rule over chains of tokens: q, k [B, M, Hk, Dk] and v [B, M, H, Dv] (float32/bfloat16; rows
    may be column ranges of a wider tensor), log decays g and rates beta float32 [B, M, H].  Sequence b begins with
    slot src[b] of states float32 [S, H, Dv, Dk] (-1: with zeros) and leaves its state in slot dst[b] (int32 [B]
    each).  scale defaults to 1/sqrt(Dk); norm_eps: q and k are normalised with it (None: used as they are).
    Returns out [B, M, H, Dv] of v's dtype.  workspace: uint8 scratch; None allocates it."""
    on, dims, rows, out = _delta_rows(q, k, v, g, beta, states, src, counts, out)
    B, M, Hk, H, Dk, Dv, _ = dims
    _ints(on, "dst", dst)
    if dst.shape != (B,):
        raise ValueError("dst must be [B]")
    lib = load()
    if workspace is None:
        need = lib.nvfp4_delta_rule_workspace_bytes(B, M, Hk, H, Dk, Dv, rows[3])
        workspace = states.new_empty((need,), dtype=_U8) if need else None
    elif workspace.dtype is not _U8 or workspace.get_device() != on or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
    _call(on, "nvfp4_delta_rule", lib.nvfp4_delta_rule, *dims, *rows,
          1.0 / math.sqrt(Dk) if scale is None else scale, -1.0 if norm_eps is None else norm_eps, states.data_ptr(),
          src.data_ptr(), dst.data_ptr(), counts.data_ptr() if counts is not None else None, out.data_ptr(),
          workspace.data_ptr() if workspace is not None else None, workspace.numel() if workspace is not None else 0)
    return out


def nvfp4_delta_tree(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                     states: torch.Tensor, src: torch.Tensor, parent: torch.Tensor,
                     counts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                     norm_eps: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     keys: Optional[torch.Tensor] = None, updates: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The gated delta rule over drafted trees (parent int32 [B, M], M <= 64), which leaves the states as they are.
    Arguments as nvfp4_delta_rule.  Returns out, and what nvfp4_delta_commit takes: keys float32 [B, M, Hk, Dk] and
    updates float32 [B, M, H, Dv] (one layer's part of tensors for all layers may be given)."""
    on, dims, rows, out = _delta_rows(q, k, v, g, beta, states, src, counts, out)
    B, M, Hk, H, Dk, Dv, _ = dims
    _ints(on, "parent", parent)
    if parent.shape != (B, M):
        raise ValueError("parent must be [B, M]")
    if keys is None:
        keys = states.new_empty((B, M, Hk, Dk))
    else:
        _floats(on, (B, M, Hk, Dk), "keys", keys)
    if updates is None:
        updates = states.new_empty((B, M, H, Dv))
    else:
        _floats(on, (B, M, H, Dv), "updates", updates)
    _call(on, "nvfp4_delta_tree", load().nvfp4_delta_tree, *dims, *rows,
          1.0 / math.sqrt(Dk) if scale is None else scale, -1.0 if norm_eps is None else norm_eps, states.data_ptr(),
          src.data_ptr(), parent.data_ptr(), counts.data_ptr() if counts is not None else None, out.data_ptr(),
          keys.data_ptr(), updates.data_ptr())
    return out, keys, updates


def nvfp4_delta_commit(states: torch.Tensor, keys: torch.Tensor, updates: torch.Tensor, g: torch.Tensor,
                       result: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
                       counts: Optional[torch.Tensor] = None) -> None:
    """Takes each sequence's state through the root and the accepted path of its tree, in all layers: states [L, S,
    H, Dv, Dk], slot src[b] to slot dst[b]; keys [L, B, M, Hk, Dk] and updates [L, B, M, H, Dv] as nvfp4_delta_tree
    gives them, g float32 [L, B, M, H] the layers' log decays, result int32 [B, 3 + M]: rows of nvfp4_tree_accept /
    nvfp4_tree_verify.  counts int32 [B]: those of the tree; nodes that are no tokens change nothing."""
    on, slots, rows, paths = states.get_device(), states.shape, keys.shape, result.shape
    if on < 0 or states.dtype is not _F32 or len(slots) != 5 or not states.is_contiguous():
        raise ValueError("states must be a contiguous float32 [L, S, H, Dv, Dk] on a GPU")
    if len(rows) != 5 or len(paths) != 2:
        raise ValueError("keys must be [L, B, M, Hk, Dk] and result [B, 3 + M]")
    L, S, H, Dv, Dk = slots
    B, M, Hk = rows[1:4]
    if paths != (B, 3 + M) or Hk < 1 or H % Hk or src.shape != (B,) or dst.shape != (B,):
        raise ValueError("states, keys, result [B, 3 + M], src [B] and dst [B] do not fit together")
    _floats(on, (L, B, M, Hk, Dk), "keys", keys)
    _floats(on, (L, B, M, H, Dv), "updates", updates)
    _floats(on, (L, B, M, H), "g", g)
    _ints(on, "result, src and dst", result, src, dst)
    if counts is not None:
        _ints(on, "counts", counts)
        if counts.shape != (B,):
            raise ValueError("counts must be [B]")
    _call(on, "nvfp4_delta_commit", load().nvfp4_delta_commit_counts, L, B, M, Hk, H, Dk, Dv, S,
          states.data_ptr(), keys.data_ptr(), updates.data_ptr(), g.data_ptr(), result.data_ptr(), src.data_ptr(),
          dst.data_ptr(), counts.data_ptr() if counts is not None else None)


def nvfp4_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0,
                         workspace: Optional[torch.Tensor] = None
                         ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Under the rows of logits [M, N] (float32/bfloat16; rows may be spaced): the log probabilities of tokens int32
    [M], the entropies, and the `top` most probable tokens with their log probabilities, in descending order:
    (float32 [M], float32 [M], float32 [M, top], int32 [M, top]).  workspace: uint8 scratch; None allocates it."""
    on, shape = logits.get_device(), logits.shape
    if on < 0 or len(shape) != 2 or (logits.stride(1) != 1 and shape[1] > 1):
        raise ValueError("logits must be [M, N] on a GPU, rows contiguous")
    M, N = shape
    _ints(on, "tokens", tokens)
    if tokens.shape != (M,):
        raise ValueError("tokens must be [M]")
    dt = _dt(logits.dtype)
    numbers = torch.empty((2, M), dtype=_F32, device=logits.device)
    best = torch.empty((M, top), dtype=_F32, device=logits.device)
    ids = tokens.new_empty((M, top))
    lib = load()
    if workspace is None:
        workspace = torch.empty((lib.nvfp4_token_logprobs_workspace_bytes(M, N, top, dt),), dtype=_U8,
                                device=logits.device)
    elif workspace.dtype is not _U8 or workspace.get_device() != on or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")
    _call(on, "nvfp4_token_logprobs", lib.nvfp4_token_logprobs, M, N, top, logits.data_ptr(), dt,
          logits.stride(0) if M > 1 else N, tokens.data_ptr(), numbers[0].data_ptr(),
          numbers[1].data_ptr(), best.data_ptr(), ids.data_ptr(), workspace.data_ptr(), workspace.numel())
    return numbers[0], numbers[1], best, ids
