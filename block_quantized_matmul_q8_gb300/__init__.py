"""Python binding of libqmm (the C ABI in include/qmm.h).

Argument marshalling only: every step of the matmul runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  The functions keep the C
names; tensors are passed as device pointers of contiguous CUDA tensors and the
current torch stream is used unless one is given.

If libqmm.so is missing or cannot be loaded, every call raises QMMError; there is
no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

TYPES = {"q4_0": 2, "q8_0": 8, "q4_K": 12, "q5_K": 13, "q6_K": 14}
BLOCK = {"q4_0": (32, 18), "q8_0": (32, 34), "q4_K": (256, 144), "q5_K": (256, 176), "q6_K": (256, 210)}
STATUS = {0: "QMM_OK", 1: "QMM_ERR_ARG", 2: "QMM_ERR_SHAPE", 3: "QMM_ERR_TYPE", 4: "QMM_ERR_ALIGN",
          5: "QMM_ERR_WORKSPACE", 6: "QMM_ERR_CUDA", 7: "QMM_ERR_IDS", 8: "QMM_ERR_DEVICE"}
PATH_AUTO, PATH_GEMV, PATH_GEMM_DP4A, PATH_GEMM_TC, PATH_GEMV_DIRECT, PATH_GEMV_TC, PATH_GEMV_MMA = 0, 1, 2, 3, 4, 5, 6

# Every function that include/qmm.h declares.
EXPORTS = ("qmm_status_string", "qmm_q8_1_bytes", "qmm_row_bytes", "qmm_workspace_bytes", "qmm_quantize_q8_1",
           "qmm_mul_mat", "qmm_mul_mat_id", "qmm_read_device_status", "qmm_tile_efficiency_percent",
           "qmm_plan_gemm", "qmm_plan_cta_range", "qmm_set_force_path", "qmm_set_stream_k_mode",
           "qmm_mul_mat_id_noalloc", "qmm_noalloc_scratch_bytes", "qmm_workspace_bytes_f32", "qmm_mul_mat_f32",
           "qmm_mul_mat_id_slot", "qmm_workspace_bytes_glu", "qmm_mul_mat_glu", "qmm_gemv_ring_stages",
           "qmm_repack_glu", "qmm_mul_mat_glu_packed", "qmm_workspace_bytes_f32_host", "qmm_mul_mat_f32_host",
           "qmm_get_device_status", "qmm_set_test_fault", "qmm_aligned_row_bytes", "qmm_repack_aligned",
           "qmm_workspace_bytes_aligned", "qmm_mul_mat_aligned", "qmm_workspace_bytes_id_glu", "qmm_mul_mat_id_glu",
           "qmm_qk_norm_rope", "qmm_workspace_bytes_attn_prompt", "qmm_attn_prompt",
           "qmm_workspace_bytes_attn_decode", "qmm_attn_decode", "qmm_kv_page_bytes", "qmm_kv_append", "qmm_kv_read",
           "qmm_workspace_bytes_attn_decode_kv", "qmm_attn_decode_kv", "qmm_take_attn_error")


class QMMError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = int(code)
        super().__init__(f"{what}: {STATUS.get(self.code, self.code)}" if what else STATUS.get(self.code, str(code)))


class GemmPlan(ctypes.Structure):
    _fields_ = [("tiles_n", ctypes.c_int64), ("tiles_m", ctypes.c_int64), ("ntiles", ctypes.c_int64),
                ("iters_per_tile", ctypes.c_int64), ("nwork", ctypes.c_int64), ("ctas", ctypes.c_int32),
                ("stream_k", ctypes.c_int32), ("fixup", ctypes.c_int32), ("efficiency_percent", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("iter_k", ctypes.c_int32)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class Heads(ctypes.Structure):
    """A [tokens][heads][head_dim] view (qmm_heads): data pointer and strides in elements."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Cache(ctypes.Structure):
    """A paged key/value cache (qmm_kv_cache)."""
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("type", ctypes.c_int32)]


FLOATS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 30}

_lib = None


def lib():
    """The loaded libqmm (ctypes.CDLL).  Raises QMMError if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise QMMError(6, f"libqmm.so not found at {LIB_PATH}; run block_quantized_matmul_q8_gb300._build.build()")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    L.qmm_status_string.restype = ctypes.c_char_p
    L.qmm_status_string.argtypes = [ctypes.c_int]
    L.qmm_q8_1_bytes.restype = SZ
    L.qmm_q8_1_bytes.argtypes = [I64, I64]
    L.qmm_row_bytes.restype = SZ
    L.qmm_row_bytes.argtypes = [ctypes.c_int, I64]
    L.qmm_workspace_bytes.restype = SZ
    L.qmm_workspace_bytes.argtypes = [ctypes.c_int, I64, I64, I64, I64, I64]
    L.qmm_quantize_q8_1.restype = ctypes.c_int
    L.qmm_quantize_q8_1.argtypes = [P, I64, I64, P, P]
    L.qmm_mul_mat.restype = ctypes.c_int
    L.qmm_mul_mat.argtypes = [P, ctypes.c_int, I64, I64, P, I64, P, P, SZ, P]
    L.qmm_mul_mat_id.restype = ctypes.c_int
    L.qmm_mul_mat_id.argtypes = [P, ctypes.c_int, I64, I64, I64, P, P, I64, I64, P, P, SZ, P]
    L.qmm_read_device_status.restype = ctypes.c_int
    L.qmm_read_device_status.argtypes = [P, ctypes.POINTER(I32), P]
    L.qmm_get_device_status.restype = ctypes.c_int
    L.qmm_get_device_status.argtypes = [P, P]
    L.qmm_tile_efficiency_percent.restype = ctypes.c_int
    L.qmm_tile_efficiency_percent.argtypes = [I64, I64]
    L.qmm_gemv_ring_stages.restype = ctypes.c_int
    L.qmm_gemv_ring_stages.argtypes = [ctypes.c_int, I64, I64, I32, I64]
    L.qmm_plan_gemm.restype = ctypes.c_int
    L.qmm_plan_gemm.argtypes = [ctypes.c_int, I64, I64, I64, I32, I32, ctypes.POINTER(GemmPlan)]
    L.qmm_plan_cta_range.restype = None
    L.qmm_plan_cta_range.argtypes = [ctypes.POINTER(GemmPlan), I32, ctypes.POINTER(I64), ctypes.POINTER(I64)]
    L.qmm_set_force_path.restype = None
    L.qmm_set_force_path.argtypes = [ctypes.c_int]
    L.qmm_aligned_row_bytes.restype = SZ
    L.qmm_aligned_row_bytes.argtypes = [ctypes.c_int, I64]
    L.qmm_repack_aligned.restype = ctypes.c_int
    L.qmm_repack_aligned.argtypes = [P, ctypes.c_int, I64, I64, P, P]
    L.qmm_workspace_bytes_aligned.restype = SZ
    L.qmm_workspace_bytes_aligned.argtypes = [ctypes.c_int, I64, I64, I64]
    L.qmm_mul_mat_aligned.restype = ctypes.c_int
    L.qmm_mul_mat_aligned.argtypes = [P, ctypes.c_int, I64, I64, P, I64, P, P, SZ, P]
    L.qmm_set_test_fault.restype = None
    L.qmm_set_test_fault.argtypes = [ctypes.c_int]
    L.qmm_set_stream_k_mode.restype = None
    L.qmm_set_stream_k_mode.argtypes = [ctypes.c_int]
    L.qmm_mul_mat_id_noalloc.restype = ctypes.c_int
    L.qmm_mul_mat_id_noalloc.argtypes = [P, ctypes.c_int, I64, I64, I64, P, P, I64, I64, P, P]
    L.qmm_workspace_bytes_glu.restype = ctypes.c_size_t
    L.qmm_workspace_bytes_glu.argtypes = [ctypes.c_int, I64, I64, I64]
    L.qmm_mul_mat_glu.restype = ctypes.c_int
    L.qmm_mul_mat_glu.argtypes = [P, P, ctypes.c_int, I64, I64, P, I64, P, P, ctypes.c_size_t, P]
    L.qmm_mul_mat_glu_packed.restype = ctypes.c_int
    L.qmm_mul_mat_glu_packed.argtypes = [P, ctypes.c_int, I64, I64, P, I64, P, P, ctypes.c_size_t, P]
    L.qmm_repack_glu.restype = ctypes.c_int
    L.qmm_repack_glu.argtypes = [P, P, ctypes.c_int, I64, I64, P, P]
    L.qmm_mul_mat_id_slot.restype = ctypes.c_int
    L.qmm_mul_mat_id_slot.argtypes = [P, ctypes.c_int, I64, I64, I64, P, P, I64, I64, P, P, ctypes.c_size_t, P]
    L.qmm_workspace_bytes_id_glu.restype = SZ
    L.qmm_workspace_bytes_id_glu.argtypes = [ctypes.c_int, I64, I64, I64, I64, I64]
    L.qmm_mul_mat_id_glu.restype = ctypes.c_int
    L.qmm_mul_mat_id_glu.argtypes = [P, P, ctypes.c_int, I64, I64, I64, P, P, I64, I64, P, P, ctypes.c_size_t, P]
    L.qmm_noalloc_scratch_bytes.restype = SZ
    L.qmm_noalloc_scratch_bytes.argtypes = []
    L.qmm_workspace_bytes_f32.restype = SZ
    L.qmm_workspace_bytes_f32_host.restype = SZ
    L.qmm_workspace_bytes_f32_host.argtypes = [ctypes.c_int, I64, I64, I64]
    L.qmm_mul_mat_f32_host.restype = ctypes.c_int
    L.qmm_mul_mat_f32_host.argtypes = [P, ctypes.c_int, I64, I64, P, I64, P, P, SZ, P]
    L.qmm_workspace_bytes_f32.argtypes = [ctypes.c_int, I64, I64, I64]
    L.qmm_mul_mat_f32.restype = ctypes.c_int
    L.qmm_mul_mat_f32.argtypes = [P, ctypes.c_int, I64, I64, P, I64, P, P, SZ, P]
    HP, F32 = ctypes.POINTER(Heads), ctypes.c_float
    L.qmm_qk_norm_rope.restype = ctypes.c_int
    L.qmm_qk_norm_rope.argtypes = [HP, HP, HP, ctypes.c_int, I64, I64, I64, I64, P, P, F32, P, P, I64, ctypes.c_int,
                                   HP, HP, HP, ctypes.c_int, P]
    L.qmm_workspace_bytes_attn_prompt.restype = SZ
    L.qmm_workspace_bytes_attn_prompt.argtypes = [I64] * 6
    L.qmm_attn_prompt.restype = ctypes.c_int
    L.qmm_attn_prompt.argtypes = [HP, HP, HP, ctypes.c_int, I64, I64, I64, I64, I64, P, P, I64, ctypes.c_int, F32, HP,
                                  P, P, SZ, P]
    L.qmm_workspace_bytes_attn_decode.restype = SZ
    L.qmm_workspace_bytes_attn_decode.argtypes = [I64] * 6
    L.qmm_attn_decode.restype = ctypes.c_int
    L.qmm_attn_decode.argtypes = [HP, HP, HP, I64, I64, P, I64, I64, HP, HP, I64, ctypes.c_int, I64, I64, I64, F32, HP,
                                  P, P, SZ, P]
    CP = ctypes.POINTER(Cache)
    L.qmm_kv_page_bytes.restype = SZ
    L.qmm_kv_page_bytes.argtypes = [ctypes.c_int, I64, I64, I64]
    L.qmm_kv_append.restype = ctypes.c_int
    L.qmm_kv_append.argtypes = [HP, HP, HP, ctypes.c_int, I64, I64, I64, I64, P, P, F32, P, P, I64, ctypes.c_int, CP, P,
                                HP, HP, HP, ctypes.c_int, P]
    L.qmm_kv_read.restype = ctypes.c_int
    L.qmm_kv_read.argtypes = [CP, P, I64, I64, P, I64, I64, I64, I64, HP, HP, ctypes.c_int, P]
    L.qmm_workspace_bytes_attn_decode_kv.restype = SZ
    L.qmm_workspace_bytes_attn_decode_kv.argtypes = [I64] * 5
    L.qmm_attn_decode_kv.restype = ctypes.c_int
    L.qmm_attn_decode_kv.argtypes = [HP, CP, P, I64, I64, P, I64, I64, ctypes.c_int, I64, I64, I64, F32, HP, P, P, SZ, P]
    L.qmm_take_attn_error.restype = ctypes.c_int
    L.qmm_take_attn_error.argtypes = [P, P]
    _lib = L
    return L


def _check(rc, what):
    if rc != 0:
        raise QMMError(rc, what)


def _qtype(t) -> int:
    return TYPES[t] if isinstance(t, str) else int(t)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise QMMError(1, f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise QMMError(3, f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise QMMError(1, f"{name} must be contiguous")
    return t


def qmm_status_string(code: int) -> str:
    return lib().qmm_status_string(int(code)).decode()


def qmm_q8_1_bytes(m: int, k: int) -> int:
    return lib().qmm_q8_1_bytes(m, k)


def qmm_row_bytes(qtype, k: int) -> int:
    return lib().qmm_row_bytes(_qtype(qtype), k)


def qmm_workspace_bytes(qtype, n: int, k: int, m: int, n_experts: int = 0, top_k: int = 0) -> int:
    return lib().qmm_workspace_bytes(_qtype(qtype), n, k, m, n_experts, top_k)


def qmm_quantize_q8_1(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [m, k] CUDA tensor -> uint8 [m, k/32*36] q8_1 blocks."""
    _dev(x, "x", torch.float32)
    m, k = x.shape
    if out is None:
        out = torch.empty((m, (k // 32) * 36), dtype=torch.uint8, device=x.device)
    _dev(out, "out", torch.uint8)
    if out.numel() < qmm_q8_1_bytes(m, k):
        raise QMMError(1, "out too small")
    _check(lib().qmm_quantize_q8_1(_ptr(x), m, k, _ptr(out), _stream(stream)), "qmm_quantize_q8_1")
    return out


def qmm_mul_mat(W: torch.Tensor, qtype, n: int, k: int, xq: torch.Tensor, m: int, y: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[m, n] fp32 = x * dequant(W)^T from q8_1 activations xq."""
    _dev(W, "W")
    _dev(xq, "xq")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=W.device)
    _dev(y, "y", torch.float32)
    need = qmm_workspace_bytes(qtype, n, k, m)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=W.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().qmm_mul_mat(_ptr(W), _qtype(qtype), n, k, _ptr(xq), m, _ptr(y), _ptr(workspace), ws_bytes,
                             _stream(stream)), "qmm_mul_mat")
    return y


def qmm_aligned_row_bytes(qtype, k: int) -> int:
    return int(lib().qmm_aligned_row_bytes(_qtype(qtype), k))


def qmm_repack_aligned(W: torch.Tensor, qtype, n: int, k: int, W_aligned: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """W with its rows padded to whole 16-byte units: uint8 [n, qmm_aligned_row_bytes]."""
    _dev(W, "W")
    if W_aligned is None:
        W_aligned = torch.empty((n, qmm_aligned_row_bytes(qtype, k)), dtype=torch.uint8, device=W.device)
    _dev(W_aligned, "W_aligned")
    _check(lib().qmm_repack_aligned(_ptr(W), _qtype(qtype), n, k, _ptr(W_aligned), _stream(stream)),
           "qmm_repack_aligned")
    return W_aligned


def qmm_workspace_bytes_aligned(qtype, n: int, k: int, m: int) -> int:
    return int(lib().qmm_workspace_bytes_aligned(_qtype(qtype), n, k, m))


def qmm_mul_mat_aligned(W_aligned: torch.Tensor, qtype, n: int, k: int, xq: torch.Tensor, m: int,
                        y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """qmm_mul_mat on the padded rows of qmm_repack_aligned."""
    _dev(W_aligned, "W_aligned")
    _dev(xq, "xq")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=W_aligned.device)
    _dev(y, "y", torch.float32)
    need = qmm_workspace_bytes_aligned(qtype, n, k, m)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=W_aligned.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().qmm_mul_mat_aligned(_ptr(W_aligned), _qtype(qtype), n, k, _ptr(xq), m, _ptr(y), _ptr(workspace),
                                     ws_bytes, _stream(stream)), "qmm_mul_mat_aligned")
    return y


def qmm_workspace_bytes_glu(qtype, n: int, k: int, m: int) -> int:
    return lib().qmm_workspace_bytes_glu(_qtype(qtype), n, k, m)


def qmm_mul_mat_glu(W_gate: torch.Tensor, W_up: torch.Tensor, qtype, n: int, k: int, xq: torch.Tensor, m: int,
                    y: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[m, n] fp32 = silu(x * dequant(W_gate)^T) * (x * dequant(W_up)^T) from q8_1 activations."""
    _dev(W_gate, "W_gate")
    _dev(W_up, "W_up")
    _dev(xq, "xq")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=W_gate.device)
    _dev(y, "y", torch.float32)
    need = qmm_workspace_bytes_glu(qtype, n, k, m)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=W_gate.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().qmm_mul_mat_glu(_ptr(W_gate), _ptr(W_up), _qtype(qtype), n, k, _ptr(xq), m, _ptr(y),
                                 _ptr(workspace) if workspace is not None else None, ws_bytes, _stream(stream)),
           "qmm_mul_mat_glu")
    return y


def qmm_repack_glu(W_gate: torch.Tensor, W_up: torch.Tensor, qtype, n: int, k: int,
                   W_gu: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Interleaved copy of a gate/up pair: row 2j = gate row j, row 2j+1 = up row j."""
    _dev(W_gate, "W_gate")
    _dev(W_up, "W_up")
    if W_gu is None:
        W_gu = torch.empty(2 * W_gate.numel(), dtype=torch.uint8, device=W_gate.device)
    _dev(W_gu, "W_gu")
    _check(lib().qmm_repack_glu(_ptr(W_gate), _ptr(W_up), _qtype(qtype), n, k, _ptr(W_gu), _stream(stream)),
           "qmm_repack_glu")
    return W_gu


def qmm_mul_mat_glu_packed(W_gu: torch.Tensor, qtype, n: int, k: int, xq: torch.Tensor, m: int,
                           y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """qmm_mul_mat_glu on the interleaved tensor of qmm_repack_glu."""
    _dev(W_gu, "W_gu")
    _dev(xq, "xq")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=W_gu.device)
    _dev(y, "y", torch.float32)
    need = qmm_workspace_bytes_glu(qtype, n, k, m)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=W_gu.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().qmm_mul_mat_glu_packed(_ptr(W_gu), _qtype(qtype), n, k, _ptr(xq), m, _ptr(y),
                                        _ptr(workspace) if workspace is not None else None, ws_bytes,
                                        _stream(stream)), "qmm_mul_mat_glu_packed")
    return y


def qmm_workspace_bytes_f32_host(qtype, n: int, k: int, m: int) -> int:
    return int(lib().qmm_workspace_bytes_f32_host(_qtype(qtype), n, k, m))


def qmm_mul_mat_f32_host(W: torch.Tensor, qtype, n: int, k: int, x_host: torch.Tensor, m: int, y_host: torch.Tensor,
                         workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """qmm_mul_mat_f32 with x and y in host memory (pinned for asynchronous copies):
    the copies and the product are enqueued on the stream by one C call."""
    _dev(W, "W")
    _dev(workspace, "workspace", torch.uint8)
    for t_, name in ((x_host, "x_host"), (y_host, "y_host")):
        if t_.is_cuda or t_.dtype != torch.float32 or not t_.is_contiguous():
            raise QMMError(1, f"{name} must be a contiguous fp32 host tensor")
    _check(lib().qmm_mul_mat_f32_host(_ptr(W), _qtype(qtype), n, k, _ptr(x_host), m, _ptr(y_host), _ptr(workspace),
                                      workspace.numel(), _stream(stream)), "qmm_mul_mat_f32_host")
    return y_host


def qmm_workspace_bytes_f32(qtype, n: int, k: int, m: int) -> int:
    return int(lib().qmm_workspace_bytes_f32(_qtype(qtype), n, k, m))


def qmm_mul_mat_f32(W: torch.Tensor, qtype, n: int, k: int, x: torch.Tensor, m: int, y: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[m, n] fp32 = x * dequant(W)^T from fp32 activations x, quantized to q8_1 inside
    the call (one launch for m == 1, which needs no workspace; a workspace is made here
    for m > 1 when none is given)."""
    _dev(W, "W")
    _dev(x, "x", torch.float32)
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=W.device)
    _dev(y, "y", torch.float32)
    if workspace is None and m > 1:
        workspace = torch.empty(qmm_workspace_bytes_f32(qtype, n, k, m), dtype=torch.uint8, device=W.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().qmm_mul_mat_f32(_ptr(W), _qtype(qtype), n, k, _ptr(x), m, _ptr(y), _ptr(workspace), ws_bytes,
                                 _stream(stream)), "qmm_mul_mat_f32")
    return y


def _mul_mat_id(fn, name, W, qtype, n_experts, n, k, xq, ids, top_k, n_tokens, y, workspace, stream):
    _dev(W, "W")
    _dev(xq, "xq")
    _dev(ids, "ids", torch.int32)
    if y is None:
        y = torch.empty((n_tokens, top_k, n), dtype=torch.float32, device=W.device)
    _dev(y, "y", torch.float32)
    if workspace is None:
        workspace = torch.empty(qmm_workspace_bytes(qtype, n, k, n_tokens, n_experts, top_k), dtype=torch.uint8,
                                device=W.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(fn(_ptr(W), _qtype(qtype), n_experts, n, k, _ptr(xq), _ptr(ids), top_k, n_tokens, _ptr(y),
              _ptr(workspace), ws_bytes, _stream(stream)), name)
    return y


def qmm_mul_mat_id(W: torch.Tensor, qtype, n_experts: int, n: int, k: int, xq: torch.Tensor, ids: torch.Tensor,
                   top_k: int, n_tokens: int, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """y[n_tokens, top_k, n] fp32 with y[t, s] = x[t] * dequant(W[ids[t, s]])^T."""
    return _mul_mat_id(lib().qmm_mul_mat_id, "qmm_mul_mat_id", W, qtype, n_experts, n, k, xq, ids, top_k, n_tokens,
                       y, workspace, stream)


def qmm_mul_mat_id_slot(W: torch.Tensor, qtype, n_experts: int, n: int, k: int, xq: torch.Tensor, ids: torch.Tensor,
                        top_k: int, n_tokens: int, y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """y[n_tokens, top_k, n] fp32 with y[t, s] = x[t, s] * dequant(W[ids[t, s]])^T: xq holds
    one q8_1 row per (token, slot) pair, row t*top_k + s."""
    return _mul_mat_id(lib().qmm_mul_mat_id_slot, "qmm_mul_mat_id_slot", W, qtype, n_experts, n, k, xq, ids, top_k,
                       n_tokens, y, workspace, stream)


def qmm_workspace_bytes_id_glu(qtype, n: int, k: int, n_tokens: int, n_experts: int, top_k: int) -> int:
    return lib().qmm_workspace_bytes_id_glu(_qtype(qtype), n, k, n_tokens, n_experts, top_k)


def qmm_mul_mat_id_glu(W_gate: torch.Tensor, W_up: torch.Tensor, qtype, n_experts: int, n: int, k: int,
                       xq: torch.Tensor, ids: torch.Tensor, top_k: int, n_tokens: int, y: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[n_tokens, top_k, n] fp32 with y[t, s] = silu(x[t] Wg[e]^T) * (x[t] Wu[e]^T), e = ids[t, s]."""
    _dev(W_gate, "W_gate")
    _dev(W_up, "W_up")
    _dev(xq, "xq")
    _dev(ids, "ids", torch.int32)
    if y is None:
        y = torch.empty((n_tokens, top_k, n), dtype=torch.float32, device=W_gate.device)
    _dev(y, "y", torch.float32)
    if workspace is None:
        workspace = torch.empty(max(qmm_workspace_bytes_id_glu(qtype, n, k, n_tokens, n_experts, top_k), 256),
                                dtype=torch.uint8, device=W_gate.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().qmm_mul_mat_id_glu(_ptr(W_gate), _ptr(W_up), _qtype(qtype), n_experts, n, k, _ptr(xq), _ptr(ids),
                                    top_k, n_tokens, _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)),
           "qmm_mul_mat_id_glu")
    return y


def qmm_mul_mat_id_noalloc(W: torch.Tensor, qtype, n_experts: int, n: int, k: int, xq: torch.Tensor,
                           ids: torch.Tensor, top_k: int, n_tokens: int, y: torch.Tensor, stream=None) -> torch.Tensor:
    """qmm_mul_mat_id with the library's fixed device scratch instead of a workspace;
    y must be given (the call allocates nothing)."""
    _dev(W, "W")
    _dev(xq, "xq")
    _dev(ids, "ids", torch.int32)
    _dev(y, "y", torch.float32)
    _check(lib().qmm_mul_mat_id_noalloc(_ptr(W), _qtype(qtype), n_experts, n, k, _ptr(xq), _ptr(ids), top_k,
                                        n_tokens, _ptr(y), _stream(stream)), "qmm_mul_mat_id_noalloc")
    return y


def qmm_noalloc_scratch_bytes() -> int:
    return lib().qmm_noalloc_scratch_bytes()


def qmm_read_device_status(workspace: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32(-1)
    _check(lib().qmm_read_device_status(_ptr(workspace), ctypes.byref(v), _stream(stream)), "qmm_read_device_status")
    return v.value


def qmm_get_device_status(workspace: torch.Tensor, stream=None) -> int:
    """The status word of the last mul_mat_id on this workspace (synchronises the stream)."""
    return int(lib().qmm_get_device_status(_ptr(workspace), _stream(stream)))


class _Views(threading.local):
    """Room for the qmm_heads of one call, of this thread: filled and read within the call."""

    def __init__(self):
        self.words = (ctypes.c_int64 * 18)()
        first = ctypes.addressof(self.words)
        self.at = tuple(ctypes.cast(first + 24 * i, ctypes.POINTER(Heads)) for i in range(6))


_views = _Views()
_pack4, _pack6 = (struct.Struct(f"{3 * n}q").pack_into for n in (4, 6))


def _view(t: torch.Tensor, name: str, shape, dtype):
    """(data, token stride, head stride) of a CUDA tensor whose last three dimensions are
    [tokens, heads, head_dim], after checking its type and shape."""
    if not t.is_cuda:
        raise QMMError(1, f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise QMMError(3, f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise QMMError(2, f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise QMMError(1, f"{name}: the elements of a head must be contiguous")
    return t.data_ptr(), st[-3], st[-2]


def _small(t, name, dtype, numel):
    """A contiguous CUDA tensor of `numel` elements (or None), as a pointer."""
    if t is None:
        return None
    if not t.is_cuda or t.dtype is not dtype or not t.is_contiguous():
        _dev(t, name, dtype)
    if t.numel() != numel:
        raise QMMError(2, f"{name} must have {numel} elements, got {t.numel()}")
    return t.data_ptr()


_status_words = {}


def _scratch(need, workspace, like):
    """(workspace, pointer, bytes).  Where a call needs no more than its status word and the caller
    gave no workspace, one block for each device takes it."""
    if workspace is not None:
        _dev(workspace, "workspace")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need > 256:
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        return workspace, workspace.data_ptr(), need
    device = like.get_device()
    block = _status_words.get(device)
    if block is None:
        block = _status_words[device] = torch.empty(256, dtype=torch.uint8, device=like.device)
    return block, block.data_ptr(), 256


def _current():
    """The handle of the current stream."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _on_stream(stream, call, *given):
    """call() with `stream` as the current one, so that what it allocates comes from that stream's memory
    and not from blocks that the caller's stream may still use.  Tensors that it returns and the caller
    did not give are kept until both streams are done with them."""
    caller = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        result = call()
    for t in result if isinstance(result, tuple) else (result,):
        if t is not None and all(t is not g for g in given):
            t.record_stream(caller)
    return result


def qmm_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor | None, positions: torch.Tensor | None,
                     inv_freq: torch.Tensor | None, w_q: torch.Tensor | None = None, w_k: torch.Tensor | None = None,
                     eps: float = 1e-6, interleaved: bool = False, out_dtype=torch.bfloat16,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     v_out: torch.Tensor | None = None, stream=None):
    """RMS norm and rotation of the heads of q [m, heads, d] and k [m, kv_heads, d], rounded to
    out_dtype together with v; returns (q_out, k_out, v_out).  inv_freq: fp32 [rotary_dim / 2]
    or None for no rotation.  Views of a fused projection's rows are taken as they are, and
    outputs may be views of a cache."""
    if stream is not None:
        return _on_stream(stream, functools.partial(qmm_qk_norm_rope, q, k, v, positions, inv_freq, w_q, w_k, eps,
                                                    interleaved, out_dtype, q_out, k_out, v_out), q_out, k_out, v_out)
    if q.dim() != 3 or k.dim() != 3:
        raise QMMError(2, "q and k must be [tokens, heads, head_dim]")
    shape, dtype = q.shape, q.dtype
    m, hq, d = shape
    hk = k.shape[1]
    if dtype not in FLOATS or out_dtype not in FLOATS:
        raise QMMError(3, "q must be fp32, fp16 or bf16")
    kv = (m, hk, d)
    if q_out is None:
        q_out = torch.empty_like(q, dtype=out_dtype, memory_format=torch.contiguous_format)
    if k_out is None:
        k_out = torch.empty_like(k, dtype=out_dtype, memory_format=torch.contiguous_format)
    if v is not None and v_out is None:
        v_out = torch.empty_like(v, dtype=out_dtype, memory_format=torch.contiguous_format)
    words, at = _views.words, _views.at
    if v is None:
        _pack4(words, 0, *_view(q, "q", shape, dtype), *_view(k, "k", kv, dtype),
               *_view(q_out, "q_out", shape, out_dtype), *_view(k_out, "k_out", kv, out_dtype))
        q_, k_, v_, qo, ko, vo = at[0], at[1], None, at[2], at[3], None
    else:
        _pack6(words, 0, *_view(q, "q", shape, dtype), *_view(k, "k", kv, dtype), *_view(v, "v", kv, dtype),
               *_view(q_out, "q_out", shape, out_dtype), *_view(k_out, "k_out", kv, out_dtype),
               *_view(v_out, "v_out", kv, out_dtype))
        q_, k_, v_, qo, ko, vo = at
    half = 0 if inv_freq is None else inv_freq.numel()
    _check(lib().qmm_qk_norm_rope(q_, k_, v_, FLOATS[dtype], m, hq, hk, d, _small(w_q, "w_q", torch.float32, d),
                                  _small(w_k, "w_k", torch.float32, d), eps,
                                  _small(positions, "positions", torch.int32, m),
                                  _small(inv_freq, "inv_freq", torch.float32, half), 2 * half, interleaved, qo, ko, vo,
                                  FLOATS[out_dtype], _current()), "qmm_qk_norm_rope")
    return q_out, k_out, v_out


def qmm_workspace_bytes_attn_prompt(tokens_q: int, tokens_k: int, n_seqs: int, heads_q: int, heads_kv: int,
                                    head_dim: int) -> int:
    return lib().qmm_workspace_bytes_attn_prompt(tokens_q, tokens_k, n_seqs, heads_q, heads_kv, head_dim)


def qmm_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                    cu_k: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention over packed sequences: q [tokens_q, heads, d], k and v [tokens_k, kv_heads, d] in fp16
    or bf16, cu_q and cu_k int32 [n_seqs + 1] row bounds (cu_k None: the same as cu_q).
    Without a workspace a device error shows in qmm_take_attn_error alone."""
    if stream is not None:
        return _on_stream(stream, functools.partial(qmm_attn_prompt, q, k, v, cu_q, cu_k, causal, scale, out, lse,
                                                    workspace), out)
    if q.dim() != 3 or k.dim() != 3:
        raise QMMError(2, "q and k must be [tokens, heads, head_dim]")
    shape, dtype = q.shape, q.dtype
    tq, hq, d = shape
    tk, hk = k.shape[0], k.shape[1]
    if dtype not in FLOATS:
        raise QMMError(3, "q must be fp16 or bf16")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    kv = (tk, hk, d)
    _pack4(_views.words, 0, *_view(q, "q", shape, dtype), *_view(k, "k", kv, dtype), *_view(v, "v", kv, dtype),
           *_view(out, "out", shape, dtype))
    q_, k_, v_, o_ = _views.at[:4]
    n = cu_q.numel() - 1
    bounds_q = _small(cu_q, "cu_q", torch.int32, n + 1)
    bounds_k = bounds_q if cu_k is None else _small(cu_k, "cu_k", torch.int32, n + 1)
    L = lib()
    ws, ws_ptr, ws_bytes = _scratch(L.qmm_workspace_bytes_attn_prompt(tq, tk, n, hq, hk, d), workspace, q)
    _check(L.qmm_attn_prompt(q_, k_, v_, FLOATS[dtype], tq, tk, hq, hk, d, bounds_q, bounds_k, n, causal,
                             d ** -0.5 if scale is None else scale, o_,
                             None if lse is None else _small(lse, "lse", torch.float32, tq * hq), ws_ptr, ws_bytes,
                             _current()), "qmm_attn_prompt")
    return out


def qmm_workspace_bytes_attn_decode(batch: int, room: int, prefix_len: int, heads_q: int, heads_kv: int,
                                    head_dim: int) -> int:
    return lib().qmm_workspace_bytes_attn_decode(batch, room, prefix_len, heads_q, heads_kv, head_dim)


_NO_VIEW = (0, 0, 0)


def qmm_attn_decode(q: torch.Tensor, k: torch.Tensor | None, v: torch.Tensor | None, lens: torch.Tensor | None,
                    prefix_k: torch.Tensor | None = None, prefix_v: torch.Tensor | None = None,
                    scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One query token for each request, q [batch, heads, d], over prefix_k and prefix_v [prefix_len, kv_heads, d]
    that all requests share and the caches k and v [batch, room, kv_heads, d] with lens int32 [batch].
    Without a workspace a device error shows in qmm_take_attn_error alone."""
    if stream is not None:
        return _on_stream(stream, functools.partial(qmm_attn_decode, q, k, v, lens, prefix_k, prefix_v, scale, out, lse,
                                                    workspace), out)
    if q.dim() != 3 or (k is None and prefix_k is None):
        raise QMMError(2, "q must be [batch, heads, head_dim], with caches or a prefix")
    shape, dtype = q.shape, q.dtype
    b, hq, d = shape
    if dtype not in FLOATS:
        raise QMMError(3, "q must be fp16 or bf16")
    if (k is None) != (v is None) or (prefix_k is None) != (prefix_v is None):
        raise QMMError(1, "k and v, and prefix_k and prefix_v, go together")
    room = p = kb = vb = 0
    kh = vh = pk = pv = _NO_VIEW
    if k is not None:
        if k.dim() != 4:
            raise QMMError(2, "k must be [batch, room, kv_heads, head_dim]")
        room, hk = k.shape[1], k.shape[2]
        cache = (b, room, hk, d)
        kh, vh = _view(k, "k", cache, dtype), _view(v, "v", cache, dtype)
        kb, vb = k.stride(0), v.stride(0)
    if prefix_k is not None:
        if prefix_k.dim() != 3:
            raise QMMError(2, "prefix_k must be [prefix_len, kv_heads, head_dim]")
        p = prefix_k.shape[0]
        if k is None:
            hk = prefix_k.shape[1]
        pk, pv = _view(prefix_k, "prefix_k", (p, hk, d), dtype), _view(prefix_v, "prefix_v", (p, hk, d), dtype)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    _pack6(_views.words, 0, *_view(q, "q", shape, dtype), *kh, *vh, *pk, *pv, *_view(out, "out", shape, dtype))
    q_, k_, v_, pk_, pv_, o_ = _views.at
    L = lib()
    ws, ws_ptr, ws_bytes = _scratch(L.qmm_workspace_bytes_attn_decode(b, room, p, hq, hk, d), workspace, q)
    _check(L.qmm_attn_decode(q_, k_, v_, kb, vb, _small(lens, "lens", torch.int32, b), b, room, pk_, pv_, p,
                             FLOATS[dtype], hq, hk, d, d ** -0.5 if scale is None else scale, o_,
                             None if lse is None else _small(lse, "lse", torch.float32, b * hq), ws_ptr, ws_bytes,
                             _current()), "qmm_attn_decode")
    return out


def qmm_kv_page_bytes(qtype, page_size: int, heads_kv: int, head_dim: int) -> int:
    return lib().qmm_kv_page_bytes(_qtype(qtype), page_size, heads_kv, head_dim)


class KVPages:
    """A paged key/value cache in q4_0 or q8_0 over the uint8 CUDA tensor pages [n_pages, page_bytes] (its rows
    may be apart: the pages of one layer of several), described once for the calls that write and read it."""

    def __init__(self, pages: torch.Tensor, qtype, page_size: int, heads_kv: int, head_dim: int):
        need = qmm_kv_page_bytes(qtype, page_size, heads_kv, head_dim)
        if need == 0:
            raise QMMError(2, "a cache is q4_0 or q8_0, of pages of 16, 32, 64, 128 or 256 tokens and heads of 32, 64, 96 or 128")
        if not pages.is_cuda:
            raise QMMError(1, "pages must be a CUDA tensor")
        if pages.dtype is not torch.uint8:
            raise QMMError(3, f"pages must be torch.uint8, got {pages.dtype}")
        if pages.dim() != 2 or pages.shape[1] != need or pages.stride(1) != 1:
            raise QMMError(2, f"pages must be [n_pages, {need}] with contiguous rows")
        self.pages, self.qtype, self.page_size, self.heads_kv, self.head_dim = pages, qtype, page_size, heads_kv, head_dim
        self.device = pages.get_device()
        self._c = Cache(pages.data_ptr(), pages.shape[0], pages.stride(0), page_size, _qtype(qtype))
        self._at = ctypes.pointer(self._c)

    @classmethod
    def empty(cls, n_pages: int, qtype, page_size: int, heads_kv: int, head_dim: int, device="cuda"):
        """A cache of new pages, whose content is unspecified."""
        shape = (n_pages, qmm_kv_page_bytes(qtype, page_size, heads_kv, head_dim))
        return cls(torch.empty(shape, dtype=torch.uint8, device=device), qtype, page_size, heads_kv, head_dim)


def _current_device(cache):
    """The cache's device, which has to be the current one."""
    if torch._C._cuda_getDevice() != cache.device:
        raise QMMError(1, f"the cache is on cuda:{cache.device}, which is not the current device")
    return cache.device


def _view_on(device, t: torch.Tensor, name: str, shape, dtype):
    """_view of a tensor that has to be on `device`."""
    if t.get_device() != device:
        raise QMMError(1, f"{name} must be on cuda:{device}, with the cache")
    if t.dtype is not dtype or t.shape != shape:
        return _view(t, name, shape, dtype)
    st = t.stride()
    if st[2] != 1 and shape[2] > 1:
        raise QMMError(1, f"{name}: the elements of a head must be contiguous")
    return t.data_ptr(), st[0], st[1]


def _small_on(device, t, name, dtype, numel):
    """_small of a tensor that has to be on `device`."""
    if t is None:
        return None
    if t.get_device() != device:
        raise QMMError(1, f"{name} must be on cuda:{device}, with the cache")
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() != numel:
        return _small(t, name, dtype, numel)
    return t.data_ptr()


def _made(like, dtype, heads, d):
    """A new contiguous tensor of like's shape [tokens, heads, d], and its view."""
    out = torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
    return out, (out.data_ptr(), heads * d, d)


def qmm_kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None,
                  inv_freq: torch.Tensor | None, cache: KVPages, slots: torch.Tensor, w_q: torch.Tensor | None = None,
                  w_k: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                  out_dtype=torch.bfloat16, values: bool = False, q_out: torch.Tensor | None = None,
                  k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """qmm_qk_norm_rope with the keys and values written to the cache's slots (int32 [m]: page * page_size +
    place, -1 for none); returns (q_out, k_out, v_out).  k_out and v_out, what the cache now stands for in
    out_dtype, are made when `values` is set or either is given, and are None otherwise."""
    if stream is not None:
        return _on_stream(stream, functools.partial(qmm_kv_append, q, k, v, positions, inv_freq, cache, slots, w_q, w_k,
                                                    eps, interleaved, out_dtype, values, q_out, k_out, v_out),
                          q_out, k_out, v_out)
    if k.dim() != 3 or (q is not None and q.dim() != 3):
        raise QMMError(2, "q and k must be [tokens, heads, head_dim]")
    kv, dtype = k.shape, k.dtype
    m, hk, d = kv
    if dtype not in FLOATS or out_dtype not in FLOATS:
        raise QMMError(3, "k must be fp32, fp16 or bf16")
    if hk != cache.heads_kv or d != cache.head_dim:
        raise QMMError(2, f"the cache holds {cache.heads_kv} heads of {cache.head_dim}, k has {hk} of {d}")
    dev = _current_device(cache)
    kw, vw = _view_on(dev, k, "k", kv, dtype), _view_on(dev, v, "v", kv, dtype)
    hq = 0
    qw = qow = kow = vow = _NO_VIEW
    if q is not None:
        hq = q.shape[1]
        shape = (m, hq, d)
        qw = _view_on(dev, q, "q", shape, dtype)
        if q_out is None:
            q_out, qow = _made(q, out_dtype, hq, d)
        else:
            qow = _view_on(dev, q_out, "q_out", shape, out_dtype)
    elif q_out is not None:
        raise QMMError(1, "q_out without q")
    both = values or k_out is not None or v_out is not None
    if both:
        if k_out is None:
            k_out, kow = _made(k, out_dtype, hk, d)
        else:
            kow = _view_on(dev, k_out, "k_out", kv, out_dtype)
        if v_out is None:
            v_out, vow = _made(v, out_dtype, hk, d)
        else:
            vow = _view_on(dev, v_out, "v_out", kv, out_dtype)
    _pack6(_views.words, 0, *qw, *kw, *vw, *qow, *kow, *vow)
    q_, k_, v_, qo, ko, vo = _views.at
    half = 0 if inv_freq is None else inv_freq.numel()
    _check(lib().qmm_kv_append(None if q is None else q_, k_, v_, FLOATS[dtype], m, hq, hk, d,
                               _small_on(dev, w_q, "w_q", torch.float32, d), _small_on(dev, w_k, "w_k", torch.float32, d),
                               eps, _small_on(dev, positions, "positions", torch.int32, m),
                               _small_on(dev, inv_freq, "inv_freq", torch.float32, half), 2 * half, interleaved,
                               cache._at, _small_on(dev, slots, "slots", torch.int32, m), None if q is None else qo,
                               ko if both else None, vo if both else None, FLOATS[out_dtype], _current()),
           "qmm_kv_append")
    return q_out, k_out, v_out


def _table(device, table, rows):
    """(pointer, width, stride) of int32 pages [rows, width]."""
    if table.get_device() != device or table.dtype is not torch.int32:
        raise QMMError(1, "the table of pages must be an int32 CUDA tensor, with the cache")
    if table.dim() != 2 or table.shape[0] != rows or (table.stride(1) != 1 and table.shape[1] > 1):
        raise QMMError(2, f"the table of pages must be [{rows}, pages] with contiguous rows")
    return table.data_ptr(), table.shape[1], table.stride(0)


def qmm_kv_read(cache: KVPages, table: torch.Tensor, cu_k: torch.Tensor, tokens: int, out_dtype=torch.bfloat16,
                k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """The sequences of table int32 [n_seqs, pages] as packed rows k and v [tokens, kv_heads, d] in 16 bits, sequence
    s at rows cu_k[s] to cu_k[s + 1] (int32 [n_seqs + 1]): what qmm_attn_prompt takes."""
    if stream is not None:
        return _on_stream(stream, functools.partial(qmm_kv_read, cache, table, cu_k, tokens, out_dtype, k_out, v_out),
                          k_out, v_out)
    if out_dtype not in FLOATS:
        raise QMMError(3, "out_dtype must be fp16 or bf16")
    dev, hk, d = _current_device(cache), cache.heads_kv, cache.head_dim
    shape = (tokens, hk, d)
    if k_out is None:
        k_out = torch.empty(shape, dtype=out_dtype, device=cache.pages.device)
        kow = (k_out.data_ptr(), hk * d, d)
    else:
        kow = _view_on(dev, k_out, "k_out", shape, out_dtype)
    if v_out is None:
        v_out = torch.empty(shape, dtype=out_dtype, device=cache.pages.device)
        vow = (v_out.data_ptr(), hk * d, d)
    else:
        vow = _view_on(dev, v_out, "v_out", shape, out_dtype)
    n = cu_k.numel() - 1
    _pack4(_views.words, 0, *kow, *vow, *_NO_VIEW, *_NO_VIEW)
    at = _views.at
    _check(lib().qmm_kv_read(cache._at, *_table(dev, table, n), _small_on(dev, cu_k, "cu_k", torch.int32, n + 1), n, tokens,
                             hk, d, at[0], at[1], FLOATS[out_dtype], _current()), "qmm_kv_read")
    return k_out, v_out


def qmm_workspace_bytes_attn_decode_kv(batch: int, max_len: int, heads_q: int, heads_kv: int, head_dim: int) -> int:
    return lib().qmm_workspace_bytes_attn_decode_kv(batch, max_len, heads_q, heads_kv, head_dim)


@functools.lru_cache(maxsize=4096)
def _decode_kv_bytes(device, *sizes):
    return lib().qmm_workspace_bytes_attn_decode_kv(*sizes)


def qmm_attn_decode_kv(q: torch.Tensor, cache: KVPages, table: torch.Tensor, lens: torch.Tensor,
                       max_len: int | None = None, scale: float | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One query token for each request, q [batch, heads, d] in fp16 or bf16, over the first lens (int32 [batch]) tokens
    of its pages, table int32 [batch, pages].  max_len bounds lens (None: all that the table holds); a bound
    close to the lengths is the faster one.  Errors show in qmm_take_attn_error."""
    if stream is not None:
        return _on_stream(stream, functools.partial(qmm_attn_decode_kv, q, cache, table, lens, max_len, scale, out, lse,
                                                    workspace), out)
    if q.dim() != 3:
        raise QMMError(2, "q must be [batch, heads, head_dim]")
    shape, dtype = q.shape, q.dtype
    b, hq, d = shape
    if dtype not in FLOATS:
        raise QMMError(3, "q must be fp16 or bf16")
    if d != cache.head_dim:
        raise QMMError(2, f"the cache holds heads of {cache.head_dim}, q has {d}")
    dev, hk = _current_device(cache), cache.heads_kv
    qw = _view_on(dev, q, "q", shape, dtype)
    if out is None:
        out, ow = _made(q, dtype, hq, d)
    else:
        ow = _view_on(dev, out, "out", shape, dtype)
    _pack4(_views.words, 0, *qw, *ow, *_NO_VIEW, *_NO_VIEW)
    at = _views.at
    table_ptr, width, stride = _table(dev, table, b)
    if max_len is None:
        max_len = width * cache.page_size
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        _dev(workspace, "workspace")
        if workspace.get_device() != dev:
            raise QMMError(1, f"workspace must be on cuda:{dev}, with the cache")
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        ws_bytes = _decode_kv_bytes(dev, b, max_len, hq, hk, d)
        if ws_bytes:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
            ws_ptr = workspace.data_ptr()
    _check(lib().qmm_attn_decode_kv(at[0], cache._at, table_ptr, width, stride, _small_on(dev, lens, "lens", torch.int32, b),
                                    b, max_len, FLOATS[dtype], hq, hk, d, d ** -0.5 if scale is None else scale, at[1],
                                    _small_on(dev, lse, "lse", torch.float32, b * hq), ws_ptr, ws_bytes, _current()),
           "qmm_attn_decode_kv")
    return out


def qmm_take_attn_error(stream=None) -> int:
    """8 (QMM_ERR_DEVICE) if any attention or cache call on the current device has given up a wait since the last
    time this was asked, with or without a workspace of the caller's, 7 (QMM_ERR_IDS) if one met a page outside
    its cache, else 0 (synchronises the stream)."""
    v = ctypes.c_int32(0)
    _check(lib().qmm_take_attn_error(ctypes.byref(v), _stream(stream)), "qmm_take_attn_error")
    return v.value


def qmm_tile_efficiency_percent(ntiles: int, nsm: int) -> int:
    return lib().qmm_tile_efficiency_percent(ntiles, nsm)


def qmm_gemv_ring_stages(t, n: int, k: int, ncols: int, smem_bytes: int) -> int:
    return lib().qmm_gemv_ring_stages(_qtype(t), n, k, ncols, smem_bytes)


def qmm_plan_gemm(qtype, n: int, k: int, m: int, nsm: int, stream_k_mode: int = 0) -> GemmPlan:
    p = GemmPlan()
    _check(lib().qmm_plan_gemm(_qtype(qtype), n, k, m, nsm, stream_k_mode, ctypes.byref(p)), "qmm_plan_gemm")
    return p


def qmm_plan_cta_range(plan: GemmPlan, cta: int):
    b, e = ctypes.c_int64(), ctypes.c_int64()
    lib().qmm_plan_cta_range(ctypes.byref(plan), cta, ctypes.byref(b), ctypes.byref(e))
    return b.value, e.value


def qmm_set_force_path(path: int) -> None:
    lib().qmm_set_force_path(int(path))


def qmm_set_stream_k_mode(mode: int) -> None:
    lib().qmm_set_stream_k_mode(int(mode))


def qmm_set_test_fault(mode: int) -> None:
    lib().qmm_set_test_fault(int(mode))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libqmm.so in-tree (nvcc, sm_103a)."""
    from ._build import build as _b
    global _lib
    path = _b(force=force, verbose=verbose)
    _lib = None
    return path
