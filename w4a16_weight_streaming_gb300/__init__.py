"""Python binding of libw4a16 (the W4A16 weight-streaming GEMM for GB300, sm_103a).

Argument marshalling only: every step of the GEMM runs in the CUDA kernels of
``libw4a16.so`` (built in-tree by ``_build.build()``), reached through the C ABI declared in
``include/w4a16.h``. PyTorch provides device memory and streams. There is no fallback: if the
library is missing or fails to load, importing this package raises.

Function names mirror the C entry points (``w4a16_repack``, ``w4a16_gemm`` ...), plus two
conveniences (``repack``, ``gemm``) that allocate the outputs with torch.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

from . import _build

LIB_PATH = _build.LIB_PATH
DEBUG_LIB_PATH = _build.DEBUG_LIB_PATH

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED_SHAPE = 2
ERR_MISALIGNED = 3
ERR_CUDA = 4
ERR_DEVICE_TIMEOUT = 5
ERR_BOUNDS = 6

PATH_AUTO = 0
PATH_GEMV = 1
PATH_TC = 2

# kernels of w4a16_kv4_attention_ex
KV4_AUTO = 0
KV4_DECODE_WIDE = 1
KV4_DECODE = 2
KV4_PROMPT = 3
KV4_PROMPT_PAIRS = 4

# every symbol include/w4a16.h declares
EXPORTED = [
    "w4a16_version", "w4a16_status_string", "w4a16_repacked_qweight_bytes", "w4a16_repacked_scales_bytes",
    "w4a16_repack", "w4a16_unrepack", "w4a16_gemm", "w4a16_gemm_ex", "w4a16_plan_for", "w4a16_last_dispatch",
    "w4a16_device_status", "w4a16_set_wait_timeout_ns", "w4a16_selftest_wait_timeout", "w4a16_gemm_host",
    "w4a16_silu_mul", "w4a16_debug_bounds", "w4a16_repacked_nvfp4_scales_bytes", "w4a16_repack_nvfp4",
    "w4a16_unrepack_nvfp4", "w4a16_gemm_nvfp4", "w4a16_gemm_nvfp4_ex", "w4a16_plan_for_nvfp4",
    "w4a16_quantize_x_int8", "w4a16_gemm_w4a8", "w4a16_gemm_w4a8_ex", "w4a16_plan_for_w4a8",
    "w4a16_quantize_gemm_w4a8", "w4a16_kv4_cache_bytes", "w4a16_kv4_append", "w4a16_kv4_load",
    "w4a16_kv4_attention_workspace_bytes", "w4a16_kv4_attention", "w4a16_kv4_attention_ex",
    "w4a16_kv4_attention_kernel", "w4a16_kv4_selftest_wait_timeout", "w4a16_kv4_selftest_withhold",
    "w4a16_sample",
    "w4a16_logprobs", "w4a16_block_norm", "w4a16_moe_workspace_bytes", "w4a16_moe",
]


class Plan(ctypes.Structure):
    """Mirror of ``w4a16_plan``; zero fields mean automatic."""

    _fields_ = [("path", ctypes.c_int), ("split_k", ctypes.c_int), ("m_tile", ctypes.c_int),
                ("k_chunk", ctypes.c_int), ("stages", ctypes.c_int), ("tmem_stages", ctypes.c_int),
                ("mma_issuers", ctypes.c_int), ("clusters", ctypes.c_int),
                ("dequant_warps", ctypes.c_int), ("tail_split", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class KV4Desc(ctypes.Structure):
    """Mirror of ``w4a16_kv4_cache``: the pages' address and the cache's shape."""

    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_tokens", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class MoEDesc(ctypes.Structure):
    """Mirror of ``w4a16_moe_experts``."""

    _fields_ = [("gate_up_q", ctypes.c_void_p), ("gate_up_s", ctypes.c_void_p), ("down_q", ctypes.c_void_p),
                ("down_s", ctypes.c_void_p), ("gate_up_scale", ctypes.c_void_p), ("down_scale", ctypes.c_void_p),
                ("experts", ctypes.c_int), ("hidden", ctypes.c_int), ("inner", ctypes.c_int), ("group", ctypes.c_int),
                ("nvfp4", ctypes.c_int)]


class W4A16Error(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)}")


def _load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} is not built ({path}); run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.w4a16_version.restype = I
    lib.w4a16_debug_bounds.restype = I
    lib.w4a16_status_string.restype = ctypes.c_char_p
    lib.w4a16_status_string.argtypes = [I]
    for n in ("w4a16_repacked_qweight_bytes", "w4a16_repacked_scales_bytes"):
        getattr(lib, n).restype = S
        getattr(lib, n).argtypes = [I, I, I]
    for n in ("w4a16_repack", "w4a16_unrepack"):
        getattr(lib, n).restype = I
        getattr(lib, n).argtypes = [P, P, P, P, I, I, I, P]
    lib.w4a16_gemm.restype = I
    lib.w4a16_gemm.argtypes = [P, P, P, P, I, I, I, I, P]
    lib.w4a16_gemm_ex.restype = I
    lib.w4a16_gemm_ex.argtypes = [P, P, P, P, I, I, I, I, ctypes.POINTER(Plan), P]
    lib.w4a16_gemm_host.restype = I
    lib.w4a16_gemm_host.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
    lib.w4a16_silu_mul.restype = I
    lib.w4a16_silu_mul.argtypes = [P, P, I, I, P]
    lib.w4a16_plan_for.restype = I
    lib.w4a16_plan_for.argtypes = [I, I, I, I, ctypes.POINTER(Plan)]
    lib.w4a16_last_dispatch.restype = I
    lib.w4a16_last_dispatch.argtypes = [ctypes.c_char_p, S]
    lib.w4a16_device_status.restype = I
    lib.w4a16_device_status.argtypes = [P]
    lib.w4a16_set_wait_timeout_ns.restype = I
    lib.w4a16_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.w4a16_selftest_wait_timeout.restype = I
    lib.w4a16_selftest_wait_timeout.argtypes = [I, P]
    F = ctypes.c_float
    lib.w4a16_repacked_nvfp4_scales_bytes.restype = S
    lib.w4a16_repacked_nvfp4_scales_bytes.argtypes = [I, I]
    for n in ("w4a16_repack_nvfp4", "w4a16_unrepack_nvfp4"):
        getattr(lib, n).restype = I
        getattr(lib, n).argtypes = [P, P, P, P, I, I, P]
    lib.w4a16_gemm_nvfp4.restype = I
    lib.w4a16_gemm_nvfp4.argtypes = [P, P, P, F, P, I, I, I, P]
    lib.w4a16_gemm_nvfp4_ex.restype = I
    lib.w4a16_gemm_nvfp4_ex.argtypes = [P, P, P, F, P, I, I, I, ctypes.POINTER(Plan), P]
    lib.w4a16_plan_for_nvfp4.restype = I
    lib.w4a16_plan_for_nvfp4.argtypes = [I, I, I, ctypes.POINTER(Plan)]
    lib.w4a16_quantize_x_int8.restype = I
    lib.w4a16_quantize_x_int8.argtypes = [P, P, P, P, I, I, P]
    lib.w4a16_gemm_w4a8.restype = I
    lib.w4a16_gemm_w4a8.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
    lib.w4a16_gemm_w4a8_ex.restype = I
    lib.w4a16_gemm_w4a8_ex.argtypes = [P, P, P, P, P, P, I, I, I, I, ctypes.POINTER(Plan), P]
    lib.w4a16_quantize_gemm_w4a8.restype = I
    lib.w4a16_quantize_gemm_w4a8.argtypes = [P, P, P, P, P, P, P, I, I, I, I, ctypes.POINTER(Plan), P]
    lib.w4a16_plan_for_w4a8.restype = I
    lib.w4a16_plan_for_w4a8.argtypes = [I, I, I, I, ctypes.POINTER(Plan)]
    L, C = ctypes.c_int64, ctypes.POINTER(KV4Desc)
    lib.w4a16_kv4_cache_bytes.restype = S
    lib.w4a16_kv4_cache_bytes.argtypes = [I, I, I, I]
    lib.w4a16_kv4_append.restype = I
    lib.w4a16_kv4_append.argtypes = [P, L, I, P, C, P, P, P, I, I, I, P, P, F, I, P]
    lib.w4a16_kv4_load.restype = I
    lib.w4a16_kv4_load.argtypes = [C, P, P, P, I, P]
    lib.w4a16_kv4_attention_workspace_bytes.restype = S
    lib.w4a16_kv4_attention_workspace_bytes.argtypes = [I]
    lib.w4a16_kv4_attention.restype = I
    lib.w4a16_kv4_attention.argtypes = [P, L, I, C, P, I, P, P, I, I, I, I, F, P, P, P, S, P]
    lib.w4a16_kv4_attention_ex.restype = I
    lib.w4a16_kv4_attention_ex.argtypes = [P, L, I, C, P, I, P, P, I, I, I, I, F, P, P, P, S, I, P]
    lib.w4a16_kv4_attention_kernel.restype = I
    lib.w4a16_kv4_attention_kernel.argtypes = [I, C, I, I, I, I]
    lib.w4a16_kv4_selftest_wait_timeout.restype = I
    lib.w4a16_kv4_selftest_wait_timeout.argtypes = [I, P]
    lib.w4a16_kv4_selftest_withhold.restype = I
    lib.w4a16_kv4_selftest_withhold.argtypes = [I]
    lib.w4a16_sample.restype = I
    lib.w4a16_sample.argtypes = [P, L, I, I, P, P, P, P, P, P, P, P]
    lib.w4a16_logprobs.restype = I
    lib.w4a16_logprobs.argtypes = [P, L, I, I, P, I, I, P, P, P, P, P, P, P]
    lib.w4a16_block_norm.restype = I
    lib.w4a16_block_norm.argtypes = [P, L, I, P, L, P, P, L, I, F, P, F, F, P, P, I, I, P]
    lib.w4a16_moe_workspace_bytes.restype = S
    lib.w4a16_moe_workspace_bytes.argtypes = [I, I, I]
    lib.w4a16_moe.restype = I
    lib.w4a16_moe.argtypes = [P, L, ctypes.POINTER(MoEDesc), P, P, I, I, I, F, P, P, P, I, P, S, P]
    return lib


lib = _load()


def load_debug_bounds() -> ctypes.CDLL:
    """The debug-bounds build (libw4a16_debug.so) as a second, independent handle with the same C
    entry points: every kernel checks its indices and reports W4A16_ERR_BOUNDS instead of accessing
    out of range."""
    return _load(DEBUG_LIB_PATH)


# ------------------------------------------------------------------------------ raw C ABI
def status_string(code: int) -> str:
    return lib.w4a16_status_string(int(code)).decode()


def w4a16_version() -> int:
    return lib.w4a16_version()


def w4a16_repacked_qweight_bytes(N: int, K: int, group: int) -> int:
    return lib.w4a16_repacked_qweight_bytes(N, K, group)


def w4a16_repacked_scales_bytes(N: int, K: int, group: int) -> int:
    return lib.w4a16_repacked_scales_bytes(N, K, group)


def w4a16_repack(qweight: int, scales: int, qweight_r: int, scales_r: int, N: int, K: int, group: int,
                 stream: int | None) -> int:
    return lib.w4a16_repack(qweight, scales, qweight_r, scales_r, N, K, group, stream)


def w4a16_unrepack(qweight_r: int, scales_r: int, qweight: int, scales: int, N: int, K: int, group: int,
                   stream: int | None) -> int:
    return lib.w4a16_unrepack(qweight_r, scales_r, qweight, scales, N, K, group, stream)


def w4a16_gemm(x: int, qweight_r: int, scales_r: int, y: int, M: int, N: int, K: int, group: int,
               stream: int | None) -> int:
    return lib.w4a16_gemm(x, qweight_r, scales_r, y, M, N, K, group, stream)


def w4a16_gemm_ex(x: int, qweight_r: int, scales_r: int, y: int, M: int, N: int, K: int, group: int,
                  plan: Plan | None, stream: int | None) -> int:
    return lib.w4a16_gemm_ex(x, qweight_r, scales_r, y, M, N, K, group,
                             ctypes.byref(plan) if plan is not None else None, stream)


def w4a16_gemm_host(x_host: int, x_dev: int, qweight_r: int, scales_r: int, y_dev: int, y_host: int, M: int, N: int,
                    K: int, group: int, stream: int | None) -> int:
    return lib.w4a16_gemm_host(x_host, x_dev, qweight_r, scales_r, y_dev, y_host, M, N, K, group, stream)


def w4a16_silu_mul(gu: int, act: int, M: int, I: int, stream: int | None) -> int:
    return lib.w4a16_silu_mul(gu, act, M, I, stream)


def w4a16_repacked_nvfp4_scales_bytes(N: int, K: int) -> int:
    return lib.w4a16_repacked_nvfp4_scales_bytes(N, K)


def w4a16_repack_nvfp4(qweight: int, scales8: int, qweight_r: int, scales_r: int, N: int, K: int,
                       stream: int | None) -> int:
    return lib.w4a16_repack_nvfp4(qweight, scales8, qweight_r, scales_r, N, K, stream)


def w4a16_unrepack_nvfp4(qweight_r: int, scales_r: int, qweight: int, scales8: int, N: int, K: int,
                         stream: int | None) -> int:
    return lib.w4a16_unrepack_nvfp4(qweight_r, scales_r, qweight, scales8, N, K, stream)


def w4a16_gemm_nvfp4(x: int, qweight_r: int, scales_r: int, tensor_scale: float, y: int, M: int, N: int, K: int,
                     stream: int | None) -> int:
    return lib.w4a16_gemm_nvfp4(x, qweight_r, scales_r, tensor_scale, y, M, N, K, stream)


def w4a16_gemm_nvfp4_ex(x: int, qweight_r: int, scales_r: int, tensor_scale: float, y: int, M: int, N: int, K: int,
                        plan: Plan | None, stream: int | None) -> int:
    return lib.w4a16_gemm_nvfp4_ex(x, qweight_r, scales_r, tensor_scale, y, M, N, K,
                                   ctypes.byref(plan) if plan is not None else None, stream)


def w4a16_plan_for_nvfp4(M: int, N: int, K: int) -> Plan:
    p = Plan()
    rc = lib.w4a16_plan_for_nvfp4(M, N, K, ctypes.byref(p))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_plan_for_nvfp4")
    return p


def w4a16_plan_for(M: int, N: int, K: int, group: int) -> Plan:
    p = Plan()
    rc = lib.w4a16_plan_for(M, N, K, group, ctypes.byref(p))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_plan_for")
    return p


def w4a16_last_dispatch() -> str:
    buf = ctypes.create_string_buffer(512)
    lib.w4a16_last_dispatch(buf, len(buf))
    return buf.value.decode()


def w4a16_device_status(stream: int | None = None) -> int:
    return lib.w4a16_device_status(stream)


def w4a16_set_wait_timeout_ns(ns: int) -> int:
    return lib.w4a16_set_wait_timeout_ns(int(ns))


def w4a16_selftest_wait_timeout(mode: int, stream: int | None = None) -> int:
    """Raw C ABI: `stream` is a cudaStream_t handle (None = the legacy default stream)."""
    return lib.w4a16_selftest_wait_timeout(int(mode), stream)


# ------------------------------------------------------------------------------ torch conveniences
def _stream_handle(stream: torch.cuda.Stream | None) -> int:
    # the current stream's handle without a Stream object around it (0.3 against 2.9 us on the host)
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _check(rc: int, where: str):
    if rc != OK:
        raise W4A16Error(rc, where)


def repack(qweight: torch.Tensor, scales: torch.Tensor, group: int = 128, stream=None):
    """Device layout from canonical device tensors (int32 [K/8, N], float16/int16 [K/G, N])."""
    K, N = qweight.shape[0] * 8, qweight.shape[1]
    qw_r = torch.empty(w4a16_repacked_qweight_bytes(N, K, group) // 4, dtype=torch.int32, device=qweight.device)
    sc_r = torch.empty(max(w4a16_repacked_scales_bytes(N, K, group) // 2, 1), dtype=torch.int16,
                       device=qweight.device)
    _check(w4a16_repack(qweight.data_ptr(), scales.data_ptr(), qw_r.data_ptr(), sc_r.data_ptr(), N, K, group,
                        _stream_handle(stream)), "w4a16_repack")
    return qw_r, sc_r


def w4a16_quantize_x_int8(x: int, xq: int, xq_f16: int | None, sx: int, M: int, K: int, stream: int | None) -> int:
    return lib.w4a16_quantize_x_int8(x, xq, xq_f16, sx, M, K, stream)


def w4a16_gemm_w4a8(xq: int, xq_f16: int | None, sx: int, qweight_r: int, scales_r: int, y: int, M: int, N: int,
                    K: int, group: int, stream: int | None) -> int:
    return lib.w4a16_gemm_w4a8(xq, xq_f16, sx, qweight_r, scales_r, y, M, N, K, group, stream)


def w4a16_gemm_w4a8_ex(xq: int, xq_f16: int | None, sx: int, qweight_r: int, scales_r: int, y: int, M: int, N: int,
                       K: int, group: int, plan: Plan | None, stream: int | None) -> int:
    return lib.w4a16_gemm_w4a8_ex(xq, xq_f16, sx, qweight_r, scales_r, y, M, N, K, group,
                                  ctypes.byref(plan) if plan is not None else None, stream)


def w4a16_quantize_gemm_w4a8(x: int, xq: int, xq_f16: int | None, sx: int, qweight_r: int, scales_r: int, y: int,
                             M: int, N: int, K: int, group: int, plan: Plan | None, stream: int | None) -> int:
    return lib.w4a16_quantize_gemm_w4a8(x, xq, xq_f16, sx, qweight_r, scales_r, y, M, N, K, group,
                                        ctypes.byref(plan) if plan is not None else None, stream)


def w4a16_plan_for_w4a8(M: int, N: int, K: int, group: int = 128) -> Plan:
    p = Plan()
    rc = lib.w4a16_plan_for_w4a8(M, N, K, group, ctypes.byref(p))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_plan_for_w4a8")
    return p


def gemm_host(x_host: torch.Tensor, x_dev: torch.Tensor, qweight_r: torch.Tensor, scales_r: torch.Tensor,
              y_dev: torch.Tensor, y_host: torch.Tensor, N: int, K: int, group: int = 128, stream=None) -> None:
    """w4a16_gemm_host on tensors: x_host / y_host fp16 on the CPU (pinned), x_dev / y_dev on cuda.
    Queues the three operations on `stream`; y_host is valid after that stream is synchronised."""
    M = x_host.shape[0]
    _check(w4a16_gemm_host(x_host.data_ptr(), x_dev.data_ptr(), qweight_r.data_ptr(), scales_r.data_ptr(),
                           y_dev.data_ptr(), y_host.data_ptr(), M, N, K, group, _stream_handle(stream)),
           "w4a16_gemm_host")


def unrepack(qweight_r: torch.Tensor, scales_r: torch.Tensor, N: int, K: int, group: int = 128, stream=None):
    qw = torch.empty((K // 8, N), dtype=torch.int32, device=qweight_r.device)
    sc = torch.empty((K // group, N), dtype=torch.int16, device=qweight_r.device)
    _check(w4a16_unrepack(qweight_r.data_ptr(), scales_r.data_ptr(), qw.data_ptr(), sc.data_ptr(), N, K, group,
                          _stream_handle(stream)), "w4a16_unrepack")
    return qw, sc


def silu_mul(gu: torch.Tensor, act: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """act[M, I] = silu(gu[:, :I]) * gu[:, I:] (float16, CUDA) through w4a16_silu_mul."""
    M, I = gu.shape[0], gu.shape[1] // 2
    if act is None:
        act = torch.empty((M, I), dtype=torch.float16, device=gu.device)
    _check(w4a16_silu_mul(gu.data_ptr(), act.data_ptr(), M, I, _stream_handle(stream)), "w4a16_silu_mul")
    return act


def gemm(x: torch.Tensor, qweight_r: torch.Tensor, scales_r: torch.Tensor, N: int, K: int, group: int = 128,
         y: torch.Tensor | None = None, plan: Plan | dict | None = None, stream=None) -> torch.Tensor:
    """y[M, N] (float16) = x[M, K] (float16, CUDA) . dequant(W) through w4a16_gemm / w4a16_gemm_ex."""
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if isinstance(plan, dict):
        plan = Plan(**plan)
    _check(w4a16_gemm_ex(x.data_ptr(), qweight_r.data_ptr(), scales_r.data_ptr(), y.data_ptr(), M, N, K, group, plan,
                         _stream_handle(stream)), "w4a16_gemm")
    return y


# ------------------------------------------------------------------------------ NVFP4 weights
def repack_nvfp4(qweight: torch.Tensor, scales8: torch.Tensor, stream=None):
    """Device layout from canonical NVFP4 device tensors (int32 [K/8, N] of E2M1 codes, uint8
    [K/16, N] of E4M3 patterns): (qweight_r int32, scales_r int16 of fp16 bits)."""
    K, N = qweight.shape[0] * 8, qweight.shape[1]
    qw_r = torch.empty(N * K // 8, dtype=torch.int32, device=qweight.device)
    sc_r = torch.empty(max(w4a16_repacked_nvfp4_scales_bytes(N, K) // 2, 1), dtype=torch.int16, device=qweight.device)
    _check(w4a16_repack_nvfp4(qweight.data_ptr(), scales8.data_ptr(), qw_r.data_ptr(), sc_r.data_ptr(), N, K,
                              _stream_handle(stream)), "w4a16_repack_nvfp4")
    return qw_r, sc_r


def unrepack_nvfp4(qweight_r: torch.Tensor, scales_r: torch.Tensor, N: int, K: int, stream=None):
    qw = torch.empty((K // 8, N), dtype=torch.int32, device=qweight_r.device)
    s8 = torch.empty((K // 16, N), dtype=torch.uint8, device=qweight_r.device)
    _check(w4a16_unrepack_nvfp4(qweight_r.data_ptr(), scales_r.data_ptr(), qw.data_ptr(), s8.data_ptr(), N, K,
                                _stream_handle(stream)), "w4a16_unrepack_nvfp4")
    return qw, s8


def gemm_nvfp4(x: torch.Tensor, qweight_r: torch.Tensor, scales_r: torch.Tensor, tensor_scale: float, N: int, K: int,
               y: torch.Tensor | None = None, plan: Plan | dict | None = None, stream=None) -> torch.Tensor:
    """y[M, N] (float16) = x[M, K] (float16, CUDA) . dequant(W) for repacked NVFP4 weights."""
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if isinstance(plan, dict):
        plan = Plan(**plan)
    _check(w4a16_gemm_nvfp4_ex(x.data_ptr(), qweight_r.data_ptr(), scales_r.data_ptr(), float(tensor_scale),
                               y.data_ptr(), M, N, K, plan, _stream_handle(stream)), "w4a16_gemm_nvfp4")
    return y


# ------------------------------------------------------------------------------ W4A8 (int8 activations)
def quantize_x_int8(x: torch.Tensor, with_f16: bool = True, out=None, stream=None):
    """Per-token symmetric int8 quantisation of x (float16 [M, K], CUDA) through w4a16_quantize_x_int8:
    (xq int8 [M, K], xq_f16 float16 [M, K] holding the same integers or None, sx float32 [M])."""
    M, K = x.shape
    if out is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        xh = torch.empty((M, K), dtype=torch.float16, device=x.device) if with_f16 else None
        sx = torch.empty(M, dtype=torch.float32, device=x.device)
    else:
        xq, xh, sx = out
    _check(w4a16_quantize_x_int8(x.data_ptr(), xq.data_ptr(), xh.data_ptr() if xh is not None else None,
                                 sx.data_ptr(), M, K, _stream_handle(stream)), "w4a16_quantize_x_int8")
    return xq, xh, sx


def gemm_w4a8(xq: torch.Tensor, xq_f16: torch.Tensor | None, sx: torch.Tensor, qweight_r: torch.Tensor,
              scales_r: torch.Tensor, N: int, K: int, group: int = 128, y: torch.Tensor | None = None,
              plan: Plan | dict | None = None, stream=None) -> torch.Tensor:
    """y[M, N] (float16) for int8 activations (from quantize_x_int8) and repacked int4 weights."""
    M = xq.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=xq.device)
    if isinstance(plan, dict):
        plan = Plan(**plan)
    _check(w4a16_gemm_w4a8_ex(xq.data_ptr(), xq_f16.data_ptr() if xq_f16 is not None else None, sx.data_ptr(),
                              qweight_r.data_ptr(), scales_r.data_ptr(), y.data_ptr(), M, N, K, group, plan,
                              _stream_handle(stream)), "w4a16_gemm_w4a8")
    return y


def quantize_gemm_w4a8(x: torch.Tensor, qweight_r: torch.Tensor, scales_r: torch.Tensor, N: int, K: int,
                       group: int = 128, out=None, y: torch.Tensor | None = None, plan: Plan | dict | None = None,
                       with_f16: bool = True, stream=None):
    """(y, (xq, xq_f16, sx)): quantise x (float16 [M, K], CUDA) and multiply in one call
    (w4a16_quantize_gemm_w4a8); the quantised activations are returned for other GEMMs of the same x."""
    M = x.shape[0]
    if out is None:
        out = (torch.empty((M, K), dtype=torch.int8, device=x.device),
               torch.empty((M, K), dtype=torch.float16, device=x.device) if with_f16 else None,
               torch.empty(M, dtype=torch.float32, device=x.device))
    xq, xh, sx = out
    if y is None:
        y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    if isinstance(plan, dict):
        plan = Plan(**plan)
    _check(w4a16_quantize_gemm_w4a8(x.data_ptr(), xq.data_ptr(), xh.data_ptr() if xh is not None else None,
                                    sx.data_ptr(), qweight_r.data_ptr(), scales_r.data_ptr(), y.data_ptr(), M, N, K,
                                    group, plan, _stream_handle(stream)), "w4a16_quantize_gemm_w4a8")
    return y, out


# ------------------------------------------------------------------------------ 4-bit paged key/value cache
def w4a16_kv4_cache_bytes(num_pages: int, page_tokens: int, kv_heads: int, head_dim: int) -> int:
    return lib.w4a16_kv4_cache_bytes(num_pages, page_tokens, kv_heads, head_dim)


def w4a16_kv4_append(qkv: int, qkv_stride: int, heads: int, q_out: int | None, cache: KV4Desc, slots: int,
                     positions: int | None, rope: int | None, rope_positions: int, rot: int, adjacent: int,
                     q_norm: int | None, k_norm: int | None, eps: float, M: int, stream: int | None) -> int:
    return lib.w4a16_kv4_append(qkv, qkv_stride, heads, q_out, ctypes.byref(cache), slots, positions, rope,
                                rope_positions, rot, adjacent, q_norm, k_norm, eps, M, stream)


def w4a16_kv4_load(cache: KV4Desc, slots: int, k: int, v: int, n: int, stream: int | None) -> int:
    return lib.w4a16_kv4_load(ctypes.byref(cache), slots, k, v, n, stream)


def w4a16_kv4_attention_workspace_bytes(head_dim: int) -> int:
    return lib.w4a16_kv4_attention_workspace_bytes(head_dim)


def w4a16_kv4_attention(q: int, q_stride: int, heads: int, cache: KV4Desc, block_table: int, max_pages: int,
                        kv_len: int, q_start: int, B: int, M: int, max_q_len: int, causal: int, scale: float,
                        out: int, lse: int | None, workspace: int, workspace_bytes: int, stream: int | None) -> int:
    return lib.w4a16_kv4_attention(q, q_stride, heads, ctypes.byref(cache), block_table, max_pages, kv_len, q_start,
                                   B, M, max_q_len, causal, scale, out, lse, workspace, workspace_bytes, stream)


def w4a16_kv4_attention_ex(q: int, q_stride: int, heads: int, cache: KV4Desc, block_table: int, max_pages: int,
                           kv_len: int, q_start: int, B: int, M: int, max_q_len: int, causal: int, scale: float,
                           out: int, lse: int | None, workspace: int, workspace_bytes: int, kernel: int,
                           stream: int | None) -> int:
    return lib.w4a16_kv4_attention_ex(q, q_stride, heads, ctypes.byref(cache), block_table, max_pages, kv_len, q_start,
                                      B, M, max_q_len, causal, scale, out, lse, workspace, workspace_bytes, kernel, stream)


def w4a16_kv4_attention_kernel(heads: int, cache: KV4Desc, max_pages: int, B: int, M: int, max_q_len: int) -> int:
    return lib.w4a16_kv4_attention_kernel(heads, ctypes.byref(cache), max_pages, B, M, max_q_len)


def w4a16_kv4_selftest_wait_timeout(mode: int, stream: int | None = None) -> int:
    return lib.w4a16_kv4_selftest_wait_timeout(int(mode), stream)


def w4a16_kv4_selftest_withhold(copy: int) -> int:
    """Of this build: INVALID_ARG but in the handle of load_debug_bounds()."""
    return lib.w4a16_kv4_selftest_withhold(int(copy))


def w4a16_sample(logits: int, stride: int, M: int, V: int, temperature: int | None, top_k: int | None,
                 top_p: int | None, min_p: int | None, u: int, tokens: int, probs: int | None,
                 stream: int | None) -> int:
    return lib.w4a16_sample(logits, stride, M, V, temperature, top_k, top_p, min_p, u, tokens, probs, stream)


def w4a16_logprobs(logits: int, stride: int, M: int, V: int, tokens: int | None, given: int, top: int,
                   temperature: int | None, logprob: int | None, rank: int | None, entropy: int | None,
                   top_tokens: int | None, top_logprob: int | None, stream: int | None) -> int:
    return lib.w4a16_logprobs(logits, stride, M, V, tokens, given, top, temperature, logprob, rank, entropy, top_tokens,
                              top_logprob, stream)


def w4a16_block_norm(h: int, h_stride: int, h_f32: int, y: int | None, y_stride: int, post_weight: int | None,
                     gate: int | None, gate_stride: int, gate_per_row: int, scale: float, weight: int | None, offset: float,
                     eps: float, h_out: int | None, x: int | None, M: int, H: int, stream: int | None) -> int:
    return lib.w4a16_block_norm(h, h_stride, h_f32, y, y_stride, post_weight, gate, gate_stride, gate_per_row, scale, weight,
                                offset, eps, h_out, x, M, H, stream)


def w4a16_moe_workspace_bytes(experts: int, hidden: int, inner: int) -> int:
    return lib.w4a16_moe_workspace_bytes(experts, hidden, inner)


def w4a16_moe(x: int, x_stride: int, experts: MoEDesc, router: int, bias: int | None, top_k: int, scoring: int,
              renormalize: int, scale: float, y: int, ids: int | None, weights: int | None, tokens: int, workspace: int,
              workspace_bytes: int, stream: int | None) -> int:
    return lib.w4a16_moe(x, x_stride, ctypes.byref(experts), router, bias, top_k, scoring, renormalize, scale, y, ids, weights,
                         tokens, workspace, workspace_bytes, stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return t.data_ptr() if t is not None else None


def _refuse(where: str, what: str):
    raise ValueError(f"{where}: {what}")


def _vec(t: torch.Tensor | None, dtype: torch.dtype, n: int) -> bool:
    """None, or a contiguous CUDA vector of n elements of `dtype`."""
    return t is None or (t.dtype is dtype and t.is_cuda and t.numel() == n and t.dim() == 1 and t.is_contiguous())


def _dense(t: torch.Tensor | None, dtype: torch.dtype, shape: tuple) -> bool:
    return t is None or (t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous())


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """An output in the memory pool of the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class KV4Cache:
    """Keys and values in 4 bits (0.5625 bytes an element), in pages of `page_tokens` tokens. A token's
    slot is page * page_tokens + its offset in the page; which pages a sequence has is the caller's."""

    def __init__(self, num_pages: int, page_tokens: int, kv_heads: int, head_dim: int, device="cuda"):
        n = w4a16_kv4_cache_bytes(num_pages, page_tokens, kv_heads, head_dim)
        if n == 0:
            raise W4A16Error(ERR_UNSUPPORTED_SHAPE, "KV4Cache")
        self.num_pages, self.page_tokens, self.kv_heads, self.head_dim = num_pages, page_tokens, kv_heads, head_dim
        self.pages = torch.empty(n, dtype=torch.uint8, device=device)
        self.desc = KV4Desc(self.pages.data_ptr(), num_pages, page_tokens, kv_heads, head_dim)
        self.ref = ctypes.byref(self.desc)


def kv4_append(qkv: torch.Tensor, cache: KV4Cache, slots: torch.Tensor, heads: int, positions=None, rope=None,
               adjacent: bool = False, q_norm=None, k_norm=None, eps: float = 1e-6, q: torch.Tensor | None = None,
               stream=None) -> torch.Tensor | None:
    """Norms and rotation of the heads of qkv [M, (heads + 2 kv_heads) head_dim] (float16), keys and values
    stored at `slots` (int32 [M], negative: not stored); returns the queries [M, heads, head_dim] (None for
    heads = 0). rope float32 [positions, rot]: rot/2 cosines, rot/2 sines; positions int32 [M]."""
    half, D = torch.float16, cache.head_dim
    if not (qkv.dtype is half and qkv.is_cuda and qkv.dim() == 2 and qkv.shape[1] == (heads + 2 * cache.kv_heads) * D
            and qkv.stride(1) == 1):
        _refuse("kv4_append", "qkv must be a CUDA float16 tensor [M, (heads + 2 kv_heads) head_dim], dense in a row")
    M = qkv.shape[0]
    if not (_vec(slots, torch.int32, M) and _vec(positions, torch.int32, M)):
        _refuse("kv4_append", "slots and positions must be CUDA int32 vectors of M elements")
    rope_p = norm_q = norm_k = q_p = None
    rows = rot = 0
    if rope is not None:
        if not (rope.dtype is torch.float32 and rope.is_cuda and rope.dim() == 2 and rope.is_contiguous()):
            _refuse("kv4_append", "rope must be a contiguous CUDA float32 tensor [positions, rot]")
        rows, rot = rope.shape
        rope_p = rope.data_ptr()
    if q_norm is not None or k_norm is not None:
        if not (_vec(q_norm, half, D) and _vec(k_norm, half, D)):
            _refuse("kv4_append", "q_norm and k_norm must be CUDA float16 vectors of head_dim elements")
        norm_q, norm_k = _ptr(q_norm), _ptr(k_norm)
    if heads > 0:
        if q is None:
            q = _new((M, heads, D), half, qkv.device, stream)
        elif not _dense(q, half, (M, heads, D)):
            _refuse("kv4_append", "q must be a contiguous CUDA float16 tensor [M, heads, head_dim]")
        q_p = q.data_ptr()
    rc = lib.w4a16_kv4_append(qkv.data_ptr(), qkv.stride(0), heads, q_p, cache.ref, slots.data_ptr(), _ptr(positions),
                              rope_p, rows, rot, int(adjacent), norm_q, norm_k, eps, M, _stream_handle(stream))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_kv4_append")
    return q if heads > 0 else None


def kv4_load(cache: KV4Cache, slots: torch.Tensor, out=None, stream=None):
    """The stored values at `slots` (int32 [n]): keys and values, float16 [n, kv_heads, head_dim] each."""
    n = slots.shape[0]
    shape = (n, cache.kv_heads, cache.head_dim)
    if not _vec(slots, torch.int32, n):
        _refuse("kv4_load", "slots must be a CUDA int32 vector")
    if out is None:
        k, v = _new(shape, torch.float16, slots.device, stream), _new(shape, torch.float16, slots.device, stream)
    else:
        k, v = out
        if not (_dense(k, torch.float16, shape) and _dense(v, torch.float16, shape)):
            _refuse("kv4_load", "out must be two contiguous CUDA float16 tensors [n, kv_heads, head_dim]")
    rc = lib.w4a16_kv4_load(cache.ref, slots.data_ptr(), k.data_ptr(), v.data_ptr(), n, _stream_handle(stream))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_kv4_load")
    return k, v


def kv4_attention_workspace(cache: KV4Cache) -> torch.Tensor:
    """Device memory for kv4_attention calls on `cache` (or on any cache of its head size) that follow one
    another on one stream; calls that may overlap need one each."""
    return torch.zeros(w4a16_kv4_attention_workspace_bytes(cache.head_dim), dtype=torch.uint8,
                       device=cache.pages.device)


def kv4_attention(q: torch.Tensor, cache: KV4Cache, block_table: torch.Tensor, kv_len: torch.Tensor,
                  q_start: torch.Tensor, max_q_len: int, workspace: torch.Tensor, scale: float | None = None,
                  causal: bool = True, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  stream=None, kernel: int = KV4_AUTO) -> torch.Tensor:
    """Attention of q [M, heads, head_dim] (float16) over the cached tokens of B sequences: block_table
    int32 [B, pages], kv_len int32 [B], q_start int32 [B + 1] (sequence b's rows of q). Queries are the last
    tokens of their sequence (causal) or see all of them. scale: 1 / sqrt(head_dim) when None. kernel: KV4_DECODE
    for exact codes and weights whatever the rows, else chosen by max_q_len, M, B and the block table's width."""
    half, i32, D = torch.float16, torch.int32, cache.head_dim
    if not (q.dtype is half and q.is_cuda and q.dim() == 3 and q.shape[2] == D and q.stride()[1:] == (D, 1)):
        _refuse("kv4_attention", "q must be a CUDA float16 tensor [M, heads, head_dim], dense in a row")
    M, heads = q.shape[0], q.shape[1]
    B = kv_len.shape[0]
    if not (_vec(kv_len, i32, B) and _vec(q_start, i32, B + 1)):
        _refuse("kv4_attention", "kv_len and q_start must be CUDA int32 vectors of B and B + 1 elements")
    if not (block_table.dtype is i32 and block_table.is_cuda and block_table.dim() == 2 and block_table.shape[0] == B
            and block_table.is_contiguous()):
        _refuse("kv4_attention", "block_table must be a contiguous CUDA int32 tensor [B, pages]")
    if not (workspace.dtype is torch.uint8 and workspace.is_cuda and workspace.is_contiguous()):
        _refuse("kv4_attention", "workspace must come from kv4_attention_workspace")
    if not _dense(lse, torch.float32, (M, heads)):
        _refuse("kv4_attention", "lse must be a contiguous CUDA float32 tensor [M, heads]")
    if out is None:
        out = _new((M, heads, D), half, q.device, stream)
    elif not _dense(out, half, (M, heads, D)):
        _refuse("kv4_attention", "out must be a contiguous CUDA float16 tensor [M, heads, head_dim]")
    rc = lib.w4a16_kv4_attention_ex(q.data_ptr(), q.stride(0), heads, cache.ref, block_table.data_ptr(),
                                    block_table.shape[1], kv_len.data_ptr(), q_start.data_ptr(), B, M, max_q_len,
                                    int(causal), D ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(lse),
                                    workspace.data_ptr(), workspace.numel(), kernel, _stream_handle(stream))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_kv4_attention")
    return out


# ------------------------------------------------------------------------------ sampling
def sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None, out=None,
           stream=None):
    """One token per row of logits [M, V] (float16, rows of any stride) by the uniform numbers u [M]:
    (tokens int32 [M], probs float32 [M]). temperature, top_p, min_p float32 [M], top_k int32 [M], or None."""
    f = torch.float32
    if not (logits.dtype is torch.float16 and logits.is_cuda and logits.dim() == 2 and logits.stride(1) == 1):
        _refuse("sample", "logits must be a CUDA float16 tensor [M, V], dense in a row")
    M, V = logits.shape
    if not (_vec(u, f, M) and _vec(temperature, f, M) and _vec(top_k, torch.int32, M) and _vec(top_p, f, M)
            and _vec(min_p, f, M)):
        _refuse("sample", "u, temperature, top_p, min_p must be CUDA float32 vectors, top_k an int32 one, of M elements")
    if out is None:
        tokens, probs = _new(M, torch.int32, logits.device, stream), _new(M, f, logits.device, stream)
    else:
        tokens, probs = out
        if not (_vec(tokens, torch.int32, M) and _vec(probs, f, M)):
            _refuse("sample", "out must be a CUDA int32 and a float32 vector of M elements")
    rc = lib.w4a16_sample(logits.data_ptr(), logits.stride(0), M, V, _ptr(temperature), _ptr(top_k), _ptr(top_p),
                          _ptr(min_p), u.data_ptr(), tokens.data_ptr(), _ptr(probs), _stream_handle(stream))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_sample")
    return tokens, probs


class LogProbs(NamedTuple):
    """What `logprobs` gives; None for what was not asked for."""

    logprob: torch.Tensor | None       # float32, like `tokens`
    rank: torch.Tensor | None          # int32, like `tokens`
    entropy: torch.Tensor              # float32 [M]
    top_tokens: torch.Tensor | None    # int32 [M, top]
    top_logprob: torch.Tensor | None   # float32 [M, top]


def logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0, temperature=None, out: LogProbs | None = None,
             stream=None) -> LogProbs:
    """Of every row of logits [M, V] (float16, rows of any stride): log probabilities and ranks (from 1) of `tokens`
    (int32 [M] or [M, up to 8]; a negative one: 0 and rank 0), the entropy, the first `top` (up to 32) tokens in the
    order of `sample`. temperature float32 [M], or None for 1."""
    f, i32 = torch.float32, torch.int32
    if not (logits.dtype is torch.float16 and logits.is_cuda and logits.dim() == 2 and logits.stride(1) == 1):
        _refuse("logprobs", "logits must be a CUDA float16 tensor [M, V], dense in a row")
    M, V = logits.shape
    shape, given = None, 0
    if tokens is not None:
        if not (tokens.dtype is i32 and tokens.is_cuda and tokens.dim() in (1, 2) and tokens.shape[0] == M and tokens.is_contiguous()):
            _refuse("logprobs", "tokens must be a contiguous CUDA int32 tensor [M] or [M, n]")
        shape, given = tuple(tokens.shape), 1 if tokens.dim() == 1 else tokens.shape[1]
        if given == 0:
            _refuse("logprobs", "tokens [M, n] must have an n above 0")
    if not _vec(temperature, f, M):
        _refuse("logprobs", "temperature must be a CUDA float32 vector of M elements")
    if top < 0:
        _refuse("logprobs", "top must not be negative")
    logprob = rank = top_tokens = top_logprob = None
    if out is None:
        dev = logits.device
        if stream is None:
            if shape is not None:
                logprob, rank = torch.empty(shape, dtype=f, device=dev), torch.empty_like(tokens)
            entropy = torch.empty(M, dtype=f, device=dev)
            if top:
                top_tokens, top_logprob = torch.empty((M, top), dtype=i32, device=dev), torch.empty((M, top), dtype=f, device=dev)
        else:
            if shape is not None:
                logprob, rank = _new(shape, f, dev, stream), _new(shape, i32, dev, stream)
            entropy = _new(M, f, dev, stream)
            if top:
                top_tokens, top_logprob = _new((M, top), i32, dev, stream), _new((M, top), f, dev, stream)
        out = LogProbs(logprob, rank, entropy, top_tokens, top_logprob)
    elif not ((out.logprob is None or shape) and (out.rank is None or shape) and _dense(out.logprob, f, shape)
              and _dense(out.rank, i32, shape) and _vec(out.entropy, f, M) and _dense(out.top_tokens, i32, (M, top))
              and _dense(out.top_logprob, f, (M, top)) and (top > 0) == (out.top_tokens is not None) == (out.top_logprob is not None)):
        _refuse("logprobs", "out must be LogProbs of contiguous CUDA tensors of the result's shapes")
    else:
        logprob, rank, entropy, top_tokens, top_logprob = out
    rc = lib.w4a16_logprobs(logits.data_ptr(), logits.stride(0), M, V, _ptr(tokens), given, top, _ptr(temperature),
                            _ptr(logprob), _ptr(rank), _ptr(entropy), _ptr(top_tokens), _ptr(top_logprob), _stream_handle(stream))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_logprobs")
    return out


# ------------------------------------------------------------------------------ around a block
def block_norm(h: torch.Tensor, y: torch.Tensor | None = None, weight=None, post_weight=None, gate=None, scale: float = 1.0,
               eps: float = 1e-6, offset: float = 0.0, out=None, stream=None):
    """(h', x): h' = h + scale * gate * z on the residual stream h [M, H] (float16 or float32), z the block's output y
    (float16) or, with post_weight, its norm; x (float16) the norm of h'. Norms multiply by offset + weight (float16 [H];
    weight None: by 1). gate (float16): [H], [M, H] or [M, 1]. Without y: x is the norm of h, and h' is h. out: the pair to
    write, where h' may be h itself and x None; an h' of None is not written."""
    half, f32 = torch.float16, h.dtype is torch.float32
    if not ((f32 or h.dtype is half) and h.is_cuda and h.dim() == 2 and h.stride(1) == 1):
        _refuse("block_norm", "h must be a CUDA float16 or float32 tensor [M, H], dense in a row")
    shape = M, H = h.shape
    h_stride = h.stride(0)
    y_p = w_p = post_p = gate_p = None
    y_stride = gate_stride = per_row = 0
    if y is not None:
        if not (y.dtype is half and y.is_cuda and y.shape == shape and y.stride(1) == 1):
            _refuse("block_norm", "y must be a CUDA float16 tensor of h's shape, dense in a row")
        y_p, y_stride = y.data_ptr(), y.stride(0)
    elif post_weight is not None or gate is not None:
        _refuse("block_norm", "post_weight and gate need y")
    if not (_vec(weight, half, H) and _vec(post_weight, half, H)):
        _refuse("block_norm", "weight and post_weight must be contiguous CUDA float16 vectors of H elements")
    if weight is not None:
        w_p = weight.data_ptr()
    if post_weight is not None:
        post_p = post_weight.data_ptr()
    if gate is not None:
        wide = gate.dim() == 2 and gate.shape[0] == M and gate.shape[1] in (1, H)
        if not (gate.dtype is half and gate.is_cuda and (wide or gate.shape == (H,)) and (gate.shape[-1] == 1 or gate.stride(-1) == 1)):
            _refuse("block_norm", "gate must be a CUDA float16 tensor [H], [M, H] or [M, 1], dense in a row")
        gate_p = gate.data_ptr()
        gate_stride = gate.stride(0) if wide else 0
        per_row = int(wide and gate.shape[1] == 1)
    if out is not None:
        h_out, x = out
        if not (_dense(h_out, h.dtype, shape) and _dense(x, half, shape)):
            _refuse("block_norm", "out must be contiguous CUDA tensors [M, H]: one of h's type, one float16")
    elif stream is None:
        h_out = h if y is None else torch.empty_like(h)
        x = torch.empty_like(h, dtype=half) if f32 else torch.empty_like(h)
    else:
        h_out = h if y is None else _new(shape, h.dtype, h.device, stream)
        x = _new(shape, half, h.device, stream)
    rc = lib.w4a16_block_norm(h.data_ptr(), h_stride, f32, y_p, y_stride, post_p, gate_p, gate_stride, per_row, scale, w_p, offset, eps,
                              None if h_out is None or h_out is h and y is None else h_out.data_ptr(),
                              None if x is None else x.data_ptr(), M, H, _stream_handle(stream))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_block_norm")
    return h_out, x


# ------------------------------------------------------------------------------ experts
class Experts:
    """The matrices of a mixture-of-experts layer in the device layout, repacked once: gate_up int4 [E, hidden / 8,
    2 inner] (gate columns first) and down [E, inner / 8, hidden] with their scales float16 [E, rows / group, columns].
    With gate_up_scale and down_scale (float32 [E], the tensor scales) the codes are NVFP4 and the scales
    uint8 [E, rows / 16, columns]."""

    def __init__(self, gate_up: torch.Tensor, gate_up_scales: torch.Tensor, down: torch.Tensor, down_scales: torch.Tensor,
                 group: int = 128, gate_up_scale: torch.Tensor | None = None, down_scale: torch.Tensor | None = None, stream=None):
        if group <= 0 or not all(t.is_cuda and t.dim() == 3 and t.is_contiguous() for t in (gate_up, gate_up_scales, down, down_scales)):
            _refuse("Experts", "gate_up, down and their scales must be contiguous CUDA tensors [E, rows, columns]")
        nvfp4 = gate_up_scale is not None
        E = gate_up.shape[0]
        self.experts, self.hidden, self.inner = E, gate_up.shape[1] * 8, gate_up.shape[2] // 2
        rows = 16 if nvfp4 else group
        half = (torch.uint8,) if nvfp4 else (torch.float16, torch.int16)
        if not (gate_up.dtype is torch.int32 and down.dtype is torch.int32 and gate_up_scales.dtype in half and down_scales.dtype in half
                and gate_up.shape[2] == 2 * self.inner and tuple(down.shape) == (E, self.inner // 8, self.hidden)
                and tuple(gate_up_scales.shape) == (E, self.hidden // rows, 2 * self.inner)
                and tuple(down_scales.shape) == (E, self.inner // rows, self.hidden)):
            _refuse("Experts", "codes must be int32 [E, rows / 8, columns], scales [E, rows / group, columns], of one hidden and inner size")
        if nvfp4 != (down_scale is not None) or not (_vec(gate_up_scale, torch.float32, E) and _vec(down_scale, torch.float32, E)):
            _refuse("Experts", "gate_up_scale and down_scale must be CUDA float32 vectors of E elements, or both None")
        if w4a16_moe_workspace_bytes(E, self.hidden, self.inner) == 0:
            raise W4A16Error(ERR_UNSUPPORTED_SHAPE, "Experts")

        def in_turns(t):  # 16 columns of gate, the same 16 of up, and on
            return t.unflatten(-1, (2, -1, 16)).transpose(-3, -2).flatten(-3).contiguous()

        def packed(codes, scales, turns):
            K, N = codes.shape[1] * 8, codes.shape[2]
            q = torch.empty((E, K // 8 * N), dtype=torch.int32, device=codes.device)
            s = torch.empty((E, K // rows * N), dtype=torch.int16, device=codes.device)
            call = lib.w4a16_repack_nvfp4 if nvfp4 else lib.w4a16_repack
            shape = (N, K) if nvfp4 else (N, K, group)
            for e in range(E):
                a, b = (in_turns(codes[e]), in_turns(scales[e])) if turns else (codes[e], scales[e])
                _check(call(a.data_ptr(), b.data_ptr(), q[e].data_ptr(), s[e].data_ptr(), *shape, _stream_handle(stream)), "Experts")
            return q, s

        self.group, self.nvfp4 = rows, nvfp4
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(gate_up.device)):
            self.gate_up, self.down = packed(gate_up, gate_up_scales, True), packed(down, down_scales, False)
        self.scales = (gate_up_scale, down_scale)
        self.desc = MoEDesc(*(t.data_ptr() for t in self.gate_up + self.down), _ptr(gate_up_scale), _ptr(down_scale), E,
                            self.hidden, self.inner, rows, int(nvfp4))
        self.ref = ctypes.byref(self.desc)


def moe_workspace(experts: Experts) -> torch.Tensor:
    """Device memory for moe calls on `experts` (or others of their shape) that follow one another on one stream;
    calls that may overlap need one each."""
    return torch.zeros(w4a16_moe_workspace_bytes(experts.experts, experts.hidden, experts.inner), dtype=torch.uint8,
                       device=experts.gate_up[0].device)


def moe(x: torch.Tensor, experts: Experts, router: torch.Tensor, top_k: int, workspace: torch.Tensor,
        bias: torch.Tensor | None = None, sigmoid: bool = False, renormalize: bool = True, scale: float = 1.0, out=None, stream=None):
    """(y, ids, weights) of a mixture-of-experts layer on x [T, hidden] (float16, up to 64 tokens): y float16 [T, hidden],
    the chosen experts int32 [T, top_k] in order and their weights float32 [T, top_k]. router float16 [E, hidden]; scores by
    softmax or sigmoid, bias float32 [E] for the choice only (sigmoid); renormalize: the chosen ones' scores add up to 1
    before `scale`. out: the three tensors to write (ids and weights may be None)."""
    half, E, H = torch.float16, experts.experts, experts.hidden
    if not (x.dtype is half and x.is_cuda and x.dim() == 2 and x.shape[1] == H and x.stride(1) == 1):
        _refuse("moe", "x must be a CUDA float16 tensor [T, hidden], dense in a row")
    if not _dense(router, half, (E, H)) or router is None:
        _refuse("moe", "router must be a contiguous CUDA float16 tensor [E, hidden]")
    if not _vec(bias, torch.float32, E):
        _refuse("moe", "bias must be a CUDA float32 vector of E elements")
    if not (workspace.dtype is torch.uint8 and workspace.is_cuda and workspace.is_contiguous()):
        _refuse("moe", "workspace must come from moe_workspace")
    if not 1 <= top_k <= E:
        _refuse("moe", "top_k must be from 1 to the number of experts")
    T = x.shape[0]
    if out is None:
        dev = x.device
        if stream is None:
            y, ids = torch.empty_like(x), torch.empty((T, top_k), dtype=torch.int32, device=dev)
            weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        else:
            y, ids, weights = _new((T, H), half, dev, stream), _new((T, top_k), torch.int32, dev, stream), _new((T, top_k), torch.float32, dev, stream)
    else:
        y, ids, weights = out
        if y is None or not (_dense(y, half, (T, H)) and _dense(ids, torch.int32, (T, top_k)) and _dense(weights, torch.float32, (T, top_k))):
            _refuse("moe", "out must be contiguous CUDA tensors: float16 [T, hidden], int32 and float32 [T, top_k]")
    rc = lib.w4a16_moe(x.data_ptr(), x.stride(0), experts.ref, router.data_ptr(), _ptr(bias), top_k, int(sigmoid), int(renormalize),
                       scale, y.data_ptr(), _ptr(ids), _ptr(weights), T, workspace.data_ptr(), workspace.numel(),
                       _stream_handle(stream))
    if rc != OK:
        raise W4A16Error(rc, "w4a16_moe")
    return y, ids, weights
