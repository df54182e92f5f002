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
