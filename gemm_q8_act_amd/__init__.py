"""gemm_q8_act_amd -- Python binding of libnvq, the MI355X (gfx950) library for
NVFP4, Q4_1, Q4_K and IQ4_XS x Q8_0 quantized matrix products.

This module only marshals arguments: every step of the computation runs in the
HIP kernels of ``libnvq.so`` behind the C ABI declared in ``include/nvq.h``.  The
functions keep the C names.  Device buffers are torch tensors (torch is used for
device memory and streams only); their data pointers and the current HIP stream
are passed straight through.  There is no fallback: if the library is missing
every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_DIR, "libnvq.so")

NVQ_OK = 0
NVQ_FMT_NVFP4 = 0
NVQ_FMT_Q4_1 = 1
NVQ_FMT_Q4_K = 2
NVQ_FMT_IQ4_XS = 3
NVQ_FMT_Q5_K = 4
NVQ_FMT_Q6_K = 5
NVQ_PATH_GEMV = 0
NVQ_PATH_GEMM = 1
NVQ_PATH_GEMV_DOT4 = 2
NVQ_GEMV_MAX_M = 15
NVQ_TYPE_F32 = 0
NVQ_TYPE_F16 = 1
NVQ_TYPE_BF16 = 2
NVQ_KV_Q8_0 = 0
NVQ_KV_F16 = 1
NVQ_KV_BF16 = 2
NVQ_ROPE_HALVES = 0
NVQ_ROPE_NEIGHBOURS = 1

# Every symbol include/nvq.h and include/nvq_probe.h declare.
EXPORTS = (
    "nvq_nvfp4_weight_bytes", "nvq_q4_1_weight_bytes", "nvq_q4_k_weight_bytes", "nvq_iq4_xs_weight_bytes",
    "nvq_gemm_workspace_bytes",
    "nvq_pack_nvfp4", "nvq_pack_q4_1", "nvq_pack_q4_k", "nvq_pack_iq4_xs", "nvq_quantize_act_q8_0", "nvq_gemv_nvfp4",
    "nvq_gemv_nvfp4_fused", "nvq_gemv_nvfp4_dot4",
    "nvq_gemv_nvfp4_routed", "nvq_gemm_nvfp4", "nvq_gemm_nvfp4_noalloc", "nvq_gemv_q4_1", "nvq_gemm_q4_1",
    "nvq_gemv_q4_k", "nvq_gemm_q4_k", "nvq_gemv_iq4_xs", "nvq_gemm_iq4_xs", "nvq_debug_isums",
    "nvq_debug_isums_iq4_xs",
    "nvq_q5_k_weight_bytes", "nvq_q6_k_weight_bytes", "nvq_pack_q5_k", "nvq_pack_q6_k",
    "nvq_gemv_q5_k", "nvq_gemm_q5_k", "nvq_gemv_q6_k", "nvq_gemm_q6_k",
    "nvq_kv_write", "nvq_kv_read", "nvq_attn_decode_workspace_bytes", "nvq_attn_decode", "nvq_attn_prompt",
    "nvq_rope_table", "nvq_qk_norm_rope", "nvq_rope_kv_write", "nvq_attn_decode_window",
    "nvq_attn_chunk_workspace_bytes", "nvq_attn_chunk",
    "nvq_status_str", "nvq_last_error",
    "nvq_probe_read", "nvq_probe_gemv_loads", "nvq_probe_mfma",
)


class NvqError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {status_str(status)} ({status}): {detail}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libnvq.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libnvq.so not built at {LIB_PATH}; run gemm_q8_act_amd.build.build()")
        # torch first: it loads its own HIP runtime (soname libamdhip64.so.7), which
        # libnvq's dependency then resolves to, so the process has one runtime and the
        # library sees torch's devices, memory and streams.  Loaded the other way round,
        # torch would bring a second runtime and libnvq's would find no device.
        import torch  # noqa: F401

        L = ctypes.CDLL(LIB_PATH)
        P, I64, SZ, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        sigs = {
            "nvq_nvfp4_weight_bytes": (SZ, [I64, I64]),
            "nvq_q4_1_weight_bytes": (SZ, [I64, I64]),
            "nvq_q4_k_weight_bytes": (SZ, [I64, I64]),
            "nvq_iq4_xs_weight_bytes": (SZ, [I64, I64]),
            "nvq_gemm_workspace_bytes": (SZ, [ctypes.c_int, I64, I64, I64]),
            "nvq_pack_nvfp4": (ctypes.c_int, [P, P, I64, I64, P]),
            "nvq_pack_q4_1": (ctypes.c_int, [P, P, P, I64, I64, P]),
            "nvq_pack_q4_k": (ctypes.c_int, [P, P, P, P, P, I64, I64, P]),
            "nvq_pack_iq4_xs": (ctypes.c_int, [P, P, P, I64, I64, P]),
            "nvq_quantize_act_q8_0": (ctypes.c_int, [P, I64, I64, P, P, P, P]),
            "nvq_gemv_nvfp4": (ctypes.c_int, [P, F, P, P, I64, I64, I64, P, P]),
            "nvq_gemv_nvfp4_fused": (ctypes.c_int, [P, F, P, I64, I64, P, P, P, P]),
            "nvq_gemv_nvfp4_dot4": (ctypes.c_int, [P, F, P, P, I64, I64, I64, P, P]),
            "nvq_gemv_nvfp4_routed": (ctypes.c_int, [P, P, P, I64, I64, P, P, I64, I64, I64, P, P]),
            "nvq_gemm_nvfp4": (ctypes.c_int, [P, F, P, P, I64, I64, I64, P, P, SZ, P]),
            "nvq_gemm_nvfp4_noalloc": (ctypes.c_int, [P, F, P, P, I64, I64, I64, P, P]),
            "nvq_gemv_q4_1": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P]),
            "nvq_gemm_q4_1": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P, SZ, P]),
            "nvq_gemv_q4_k": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P]),
            "nvq_gemm_q4_k": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P, SZ, P]),
            "nvq_gemv_iq4_xs": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P]),
            "nvq_gemm_iq4_xs": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P, SZ, P]),
            "nvq_debug_isums_iq4_xs": (ctypes.c_int, [P, ctypes.c_int, P, P, I64, I64, I64, P, P]),
            "nvq_debug_isums": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, P, P, I64, I64, I64, P, P]),
            "nvq_status_str": (ctypes.c_char_p, [ctypes.c_int]),
            "nvq_last_error": (ctypes.c_char_p, []),
            "nvq_q5_k_weight_bytes": (SZ, [I64, I64]),
            "nvq_q6_k_weight_bytes": (SZ, [I64, I64]),
            "nvq_pack_q5_k": (ctypes.c_int, [P, P, P, P, P, I64, I64, P]),
            "nvq_pack_q6_k": (ctypes.c_int, [P, P, P, I64, I64, P]),
            "nvq_gemv_q5_k": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P]),
            "nvq_gemm_q5_k": (ctypes.c_int, [P, P, P, P, I64, I64, I64, P, P, SZ, P]),
            "nvq_gemv_q6_k": (ctypes.c_int, [P, P, P, I64, I64, I64, P, P]),
            "nvq_gemm_q6_k": (ctypes.c_int, [P, P, P, I64, I64, I64, P, P, SZ, P]),
            "nvq_kv_write": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, P, I64, I64, P, I64, I64, P, I64, I64, I64,
                                            P, P, P, P, I64, I64, P]),
            "nvq_kv_read": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, P, I64, I64, P, I64, I64, P, I64, I64, I64,
                                           P, P, P, P, I64, I64, P]),
            "nvq_attn_decode_workspace_bytes": (SZ, [I64, I64, I64, I64, I64, I64]),
            "nvq_attn_decode": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, P, I64, I64, I64, I64, I64, I64, P, P, P, P,
                                               I64, I64, P, I64, P, F, P, P, SZ, P]),
            "nvq_attn_decode_window": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, P, I64, I64, I64, I64, I64, I64, P, P, P, P,
                                                      I64, I64, P, I64, P, F, I64, I64, P, P, SZ, P]),
            "nvq_attn_chunk_workspace_bytes": (SZ, [ctypes.c_int, I64, I64, I64, I64, I64, I64, I64, I64, I64]),
            "nvq_attn_chunk": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, P, P, I64, I64, I64, I64, I64, P, P, P, P, I64, I64, P, I64, P, P, F, I64, I64,
                                              P, P, SZ, P]),
            "nvq_attn_prompt": (ctypes.c_int, [ctypes.c_int, P, P, P, P, P, P, P, I64, I64, I64, I64, I64, I64, F,
                                               ctypes.c_int, P]),
            "nvq_rope_table": (ctypes.c_int, [P, I64, I64, P]),
            "nvq_qk_norm_rope": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, P, I64, I64, P, I64, I64, I64, I64, I64, I64, P, P, F, P, I64, I64,
                                                ctypes.c_int, P, ctypes.c_int, P, P, I64, I64, P, I64, I64, P]),
            "nvq_rope_kv_write": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, P, I64, I64, P, I64, I64, P, I64, I64, I64, I64, I64, I64,
                                                 P, P, F, P, I64, I64, ctypes.c_int, P, ctypes.c_int, P, P, P, I64, I64, P, P, P, P, I64, I64, P]),
            "nvq_probe_read": (ctypes.c_int, [P, SZ, ctypes.c_int, P, P]),
            "nvq_probe_gemv_loads": (ctypes.c_int, [P, I64, I64, ctypes.c_int, ctypes.c_int, ctypes.c_int, P, P]),
            "nvq_probe_mfma": (ctypes.c_int, [ctypes.c_int, I64, ctypes.c_int, P, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_str(s: int) -> str:
    return lib().nvq_status_str(int(s)).decode()


def last_error() -> str:
    return lib().nvq_last_error().decode()


def _check(status: int, where: str) -> None:
    if status != NVQ_OK:
        raise NvqError(status, where, last_error())


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(t):
    """Device address of a torch tensor (or None)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libnvq must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, *tensors):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch

    dev = next((t.device for t in tensors if t is not None and t.is_cuda), None)
    if dev is None:
        return None
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, dtype, shape, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _workspace(nbytes, stream, like):
    """Scratch of one call, asked for with the call's stream current: torch's allocator hands memory out again in the
    order of the stream that it was asked for on, so a block that work waiting on another stream has just
    let go of is not it."""
    if not nbytes:
        return None
    import torch

    if stream is None or int(stream) == torch.cuda.current_stream(like.device).cuda_stream:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=like.device) if int(stream) else torch.cuda.default_stream(like.device)):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


# ---------------------------------------------------------------------------
# sizes and packers (host)
# ---------------------------------------------------------------------------

def nvq_nvfp4_weight_bytes(N: int, K: int) -> int:
    return int(lib().nvq_nvfp4_weight_bytes(N, K))


def nvq_q4_1_weight_bytes(N: int, K: int) -> int:
    return int(lib().nvq_q4_1_weight_bytes(N, K))


def nvq_q4_k_weight_bytes(N: int, K: int) -> int:
    return int(lib().nvq_q4_k_weight_bytes(N, K))


def nvq_iq4_xs_weight_bytes(N: int, K: int) -> int:
    return int(lib().nvq_iq4_xs_weight_bytes(N, K))


def nvq_gemm_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(lib().nvq_gemm_workspace_bytes(fmt, M, N, K))


def nvq_pack_nvfp4(codes: np.ndarray, ue4m3: np.ndarray) -> np.ndarray:
    """codes uint8 [N, K] (0..15), ue4m3 uint8 [N, K/16] -> packed uint8 buffer."""
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    ue4m3 = np.ascontiguousarray(ue4m3, dtype=np.uint8)
    N, K = codes.shape
    if ue4m3.shape != (N, K // 16):
        raise ValueError("ue4m3 must be [N, K/16]")
    nbytes = nvq_nvfp4_weight_bytes(N, K)
    out = np.empty(max(nbytes, 1), np.uint8)
    _check(lib().nvq_pack_nvfp4(codes.ctypes.data_as(ctypes.c_void_p), ue4m3.ctypes.data_as(ctypes.c_void_p),
                                N, K, out.ctypes.data_as(ctypes.c_void_p)), "nvq_pack_nvfp4")
    return out[:nbytes]


def nvq_pack_q4_1(q: np.ndarray, d_f16: np.ndarray, m_f16: np.ndarray) -> np.ndarray:
    """q uint8 [N, K] (0..15), d_f16 / m_f16 uint16 [N, K/32] -> packed uint8 buffer."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    d_f16 = np.ascontiguousarray(d_f16, dtype=np.uint16)
    m_f16 = np.ascontiguousarray(m_f16, dtype=np.uint16)
    N, K = q.shape
    if d_f16.shape != (N, K // 32) or m_f16.shape != (N, K // 32):
        raise ValueError("d_f16 and m_f16 must be [N, K/32]")
    nbytes = nvq_q4_1_weight_bytes(N, K)
    out = np.empty(max(nbytes, 1), np.uint8)
    _check(lib().nvq_pack_q4_1(q.ctypes.data_as(ctypes.c_void_p), d_f16.ctypes.data_as(ctypes.c_void_p),
                               m_f16.ctypes.data_as(ctypes.c_void_p), N, K,
                               out.ctypes.data_as(ctypes.c_void_p)), "nvq_pack_q4_1")
    return out[:nbytes]


# ---------------------------------------------------------------------------
# device entry points (torch tensors on the GPU)
# ---------------------------------------------------------------------------

def nvq_quantize_act_q8_0(x, q, d_f16, bsum16=None, stream=None) -> None:
    """x float32 [M, K] -> q int8 [M, K], d_f16 int16/uint16 bits [M, K/32], bsum16 int16 [M, K/16]."""
    import torch

    M, K = x.shape
    _need(x, torch.float32, (M, K), "x")
    _need(q, torch.int8, (M, K), "q")
    if d_f16 is None or tuple(d_f16.shape) != (M, K // 32) or d_f16.element_size() != 2:
        raise ValueError("d_f16 must be a 2-byte tensor [M, K/32]")
    if bsum16 is not None:
        _need(bsum16, torch.int16, (M, K // 16), "bsum16")
    _check(lib().nvq_quantize_act_q8_0(_ptr(x), M, K, _ptr(q), _ptr(d_f16), _ptr(bsum16),
                                       _stream(stream, x)), "nvq_quantize_act_q8_0")


def _weights(w, nbytes, name):
    import torch

    if w is None or w.dtype != torch.uint8 or w.numel() < nbytes:
        raise ValueError(f"{name}: packed uint8 weight buffer of >= {nbytes} bytes required")


def _acts(q, d_f16):
    import torch

    M, K = q.shape
    _need(q, torch.int8, (M, K), "q")
    if d_f16 is None or tuple(d_f16.shape) != (M, K // 32) or d_f16.element_size() != 2:
        raise ValueError("d_f16 must be a 2-byte tensor [M, K/32]")
    return M, K


def nvq_gemv_nvfp4(w, w_scale: float, q, d_f16, y, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_nvfp4_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_nvfp4(_ptr(w), float(w_scale), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y),
                                _stream(stream, y)), "nvq_gemv_nvfp4")


def nvq_gemv_nvfp4_fused(w, w_scale: float, x, y, q_out=None, d_out=None, stream=None) -> None:
    """One token: x float32 [1, K] (or [K]) -> y float32 [1, N] (or [N]), Q8_0
    quantization inside the GEMV launch; q_out int8 [.., K] / d_out 2-byte [.., K/32]
    optionally receive the codes and scales."""
    import torch

    K = x.shape[-1]
    N = y.shape[-1]
    if x.numel() != K or y.numel() != N:
        raise ValueError("nvq_gemv_nvfp4_fused takes one token: x [K] or [1, K], y [N] or [1, N]")
    _need(x, torch.float32, tuple(x.shape), "x")
    _need(y, torch.float32, tuple(y.shape), "y")
    if (q_out is None) != (d_out is None):
        raise ValueError("q_out and d_out are given together or not at all")
    if q_out is not None:
        if q_out.dtype != torch.int8 or q_out.numel() != K:
            raise ValueError("q_out: int8 tensor of K elements required")
        if d_out.element_size() != 2 or d_out.numel() != K // 32:
            raise ValueError("d_out: 2-byte tensor of K/32 elements required")
    _weights(w, nvq_nvfp4_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_nvfp4_fused(_ptr(w), float(w_scale), _ptr(x), N, K, _ptr(y), _ptr(q_out), _ptr(d_out),
                                      _stream(stream, y)), "nvq_gemv_nvfp4_fused")


def nvq_gemv_nvfp4_routed(w, w_scales, ids, q, d_f16, y, stream=None) -> None:
    """w: uint8, n_experts packed [N][K] matrices back to back; w_scales float32
    [n_experts]; ids int32 [M, n_active]; q, d_f16 [M, K]; y float32 [M, n_active, N]."""
    import torch

    M, K = _acts(q, d_f16)
    E = w_scales.shape[0]
    _need(w_scales, torch.float32, (E,), "w_scales")
    A = ids.shape[1] if ids is not None and ids.dim() == 2 else -1
    _need(ids, torch.int32, (M, A), "ids")
    N = y.shape[2]
    _need(y, torch.float32, (M, A, N), "y")
    _weights(w, E * nvq_nvfp4_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_nvfp4_routed(_ptr(w), _ptr(w_scales), _ptr(ids), E, A, _ptr(q), _ptr(d_f16), M, N, K,
                                       _ptr(y), _stream(stream, y)), "nvq_gemv_nvfp4_routed")


def nvq_gemv_nvfp4_dot4(w, w_scale: float, q, d_f16, y, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_nvfp4_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_nvfp4_dot4(_ptr(w), float(w_scale), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y),
                                     _stream(stream, y)), "nvq_gemv_nvfp4_dot4")


def nvq_gemm_nvfp4(w, w_scale: float, q, d_f16, y, workspace=None, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_nvfp4_weight_bytes(N, K), "w")
    if workspace is None:  # the split-K partial tiles; torch's caching allocator makes this cheap
        workspace = _workspace(lib().nvq_gemm_workspace_bytes(NVQ_FMT_NVFP4, M, N, K), stream, y)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().nvq_gemm_nvfp4(_ptr(w), float(w_scale), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y),
                                _ptr(workspace), ws_bytes, _stream(stream, y)), "nvq_gemm_nvfp4")


def nvq_gemm_nvfp4_noalloc(w, w_scale: float, q, d_f16, y, stream=None) -> None:
    """nvq_gemm_nvfp4 with its K-split partials in the library's static per-GPU scratch
    (nothing allocated; calls on one GPU must not overlap in time)."""
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_nvfp4_weight_bytes(N, K), "w")
    _check(lib().nvq_gemm_nvfp4_noalloc(_ptr(w), float(w_scale), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y),
                                        _stream(stream, y)), "nvq_gemm_nvfp4_noalloc")


def nvq_gemv_q4_1(w, q, d_f16, bsum16, y, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _need(bsum16, torch.int16, (M, K // 16), "bsum16")
    _weights(w, nvq_q4_1_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_q4_1(_ptr(w), _ptr(q), _ptr(d_f16), _ptr(bsum16), M, N, K, _ptr(y),
                               _stream(stream, y)), "nvq_gemv_q4_1")


def nvq_gemm_q4_1(w, q, d_f16, bsum16, y, workspace=None, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _need(bsum16, torch.int16, (M, K // 16), "bsum16")
    _weights(w, nvq_q4_1_weight_bytes(N, K), "w")
    if workspace is None:
        workspace = _workspace(lib().nvq_gemm_workspace_bytes(NVQ_FMT_Q4_1, M, N, K), stream, y)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().nvq_gemm_q4_1(_ptr(w), _ptr(q), _ptr(d_f16), _ptr(bsum16), M, N, K, _ptr(y),
                               _ptr(workspace), ws_bytes, _stream(stream, y)), "nvq_gemm_q4_1")


def nvq_pack_q4_k(q: np.ndarray, sc: np.ndarray, mn: np.ndarray, d_f16: np.ndarray,
                  dmin_f16: np.ndarray) -> np.ndarray:
    """q uint8 [N, K] (0..15), sc / mn uint8 [N, K/32] (0..63), d_f16 / dmin_f16 uint16
    [N, K/256] -> packed uint8 buffer."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    sc = np.ascontiguousarray(sc, dtype=np.uint8)
    mn = np.ascontiguousarray(mn, dtype=np.uint8)
    d_f16 = np.ascontiguousarray(d_f16, dtype=np.uint16)
    dmin_f16 = np.ascontiguousarray(dmin_f16, dtype=np.uint16)
    N, K = q.shape
    if sc.shape != (N, K // 32) or mn.shape != (N, K // 32):
        raise ValueError("sc and mn must be [N, K/32]")
    if d_f16.shape != (N, K // 256) or dmin_f16.shape != (N, K // 256):
        raise ValueError("d_f16 and dmin_f16 must be [N, K/256]")
    nbytes = nvq_q4_k_weight_bytes(N, K)
    out = np.empty(max(nbytes, 1), np.uint8)
    _check(lib().nvq_pack_q4_k(*(a.ctypes.data_as(ctypes.c_void_p) for a in (q, sc, mn, d_f16, dmin_f16)), N, K,
                               out.ctypes.data_as(ctypes.c_void_p)), "nvq_pack_q4_k")
    return out[:nbytes]


def nvq_gemv_q4_k(w, q, d_f16, bsum16, y, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _need(bsum16, torch.int16, (M, K // 16), "bsum16")
    _weights(w, nvq_q4_k_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_q4_k(_ptr(w), _ptr(q), _ptr(d_f16), _ptr(bsum16), M, N, K, _ptr(y),
                               _stream(stream, y)), "nvq_gemv_q4_k")


def nvq_gemm_q4_k(w, q, d_f16, bsum16, y, workspace=None, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _need(bsum16, torch.int16, (M, K // 16), "bsum16")
    _weights(w, nvq_q4_k_weight_bytes(N, K), "w")
    if workspace is None:
        workspace = _workspace(lib().nvq_gemm_workspace_bytes(NVQ_FMT_Q4_K, M, N, K), stream, y)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().nvq_gemm_q4_k(_ptr(w), _ptr(q), _ptr(d_f16), _ptr(bsum16), M, N, K, _ptr(y),
                               _ptr(workspace), ws_bytes, _stream(stream, y)), "nvq_gemm_q4_k")


def nvq_q5_k_weight_bytes(N: int, K: int) -> int:
    return int(lib().nvq_q5_k_weight_bytes(N, K))


def nvq_q6_k_weight_bytes(N: int, K: int) -> int:
    return int(lib().nvq_q6_k_weight_bytes(N, K))


def nvq_pack_q5_k(q: np.ndarray, sc: np.ndarray, mn: np.ndarray, d_f16: np.ndarray,
                  dmin_f16: np.ndarray) -> np.ndarray:
    """q uint8 [N, K] (0..31), sc / mn uint8 [N, K/32] (0..63), d_f16 / dmin_f16 uint16
    [N, K/256] -> packed uint8 buffer."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    sc = np.ascontiguousarray(sc, dtype=np.uint8)
    mn = np.ascontiguousarray(mn, dtype=np.uint8)
    d_f16 = np.ascontiguousarray(d_f16, dtype=np.uint16)
    dmin_f16 = np.ascontiguousarray(dmin_f16, dtype=np.uint16)
    N, K = q.shape
    if sc.shape != (N, K // 32) or mn.shape != (N, K // 32):
        raise ValueError("sc and mn must be [N, K/32]")
    if d_f16.shape != (N, K // 256) or dmin_f16.shape != (N, K // 256):
        raise ValueError("d_f16 and dmin_f16 must be [N, K/256]")
    nbytes = nvq_q5_k_weight_bytes(N, K)
    out = np.empty(max(nbytes, 1), np.uint8)
    _check(lib().nvq_pack_q5_k(*(a.ctypes.data_as(ctypes.c_void_p) for a in (q, sc, mn, d_f16, dmin_f16)), N, K,
                               out.ctypes.data_as(ctypes.c_void_p)), "nvq_pack_q5_k")
    return out[:nbytes]


def nvq_pack_q6_k(q: np.ndarray, sc: np.ndarray, d_f16: np.ndarray) -> np.ndarray:
    """q uint8 [N, K] (0..63), sc int8 [N, K/16], d_f16 uint16 [N, K/256] -> packed uint8
    buffer."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    sc = np.ascontiguousarray(sc, dtype=np.int8)
    d_f16 = np.ascontiguousarray(d_f16, dtype=np.uint16)
    N, K = q.shape
    if sc.shape != (N, K // 16) or d_f16.shape != (N, K // 256):
        raise ValueError("sc must be [N, K/16] and d_f16 [N, K/256]")
    nbytes = nvq_q6_k_weight_bytes(N, K)
    out = np.empty(max(nbytes, 1), np.uint8)
    _check(lib().nvq_pack_q6_k(*(a.ctypes.data_as(ctypes.c_void_p) for a in (q, sc, d_f16)), N, K,
                               out.ctypes.data_as(ctypes.c_void_p)), "nvq_pack_q6_k")
    return out[:nbytes]


def nvq_gemv_q5_k(w, q, d_f16, bsum16, y, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _need(bsum16, torch.int16, (M, K // 16), "bsum16")
    _weights(w, nvq_q5_k_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_q5_k(_ptr(w), _ptr(q), _ptr(d_f16), _ptr(bsum16), M, N, K, _ptr(y),
                               _stream(stream, y)), "nvq_gemv_q5_k")


def nvq_gemm_q5_k(w, q, d_f16, bsum16, y, workspace=None, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _need(bsum16, torch.int16, (M, K // 16), "bsum16")
    _weights(w, nvq_q5_k_weight_bytes(N, K), "w")
    if workspace is None:
        workspace = _workspace(lib().nvq_gemm_workspace_bytes(NVQ_FMT_Q5_K, M, N, K), stream, y)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().nvq_gemm_q5_k(_ptr(w), _ptr(q), _ptr(d_f16), _ptr(bsum16), M, N, K, _ptr(y),
                               _ptr(workspace), ws_bytes, _stream(stream, y)), "nvq_gemm_q5_k")


def nvq_gemv_q6_k(w, q, d_f16, y, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_q6_k_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_q6_k(_ptr(w), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y), _stream(stream, y)),
           "nvq_gemv_q6_k")


def nvq_gemm_q6_k(w, q, d_f16, y, workspace=None, stream=None) -> None:
    import torch

    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_q6_k_weight_bytes(N, K), "w")
    if workspace is None:
        workspace = _workspace(lib().nvq_gemm_workspace_bytes(NVQ_FMT_Q6_K, M, N, K), stream, y)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().nvq_gemm_q6_k(_ptr(w), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y), _ptr(workspace), ws_bytes,
                               _stream(stream, y)), "nvq_gemm_q6_k")


def nvq_pack_iq4_xs(q: np.ndarray, ls: np.ndarray, d_f16: np.ndarray) -> np.ndarray:
    """q uint8 [N, K] (0..15), ls uint8 [N, K/32] (0..63), d_f16 uint16 [N, K/256] ->
    packed uint8 buffer (the value table is passed to the products)."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    ls = np.ascontiguousarray(ls, dtype=np.uint8)
    d_f16 = np.ascontiguousarray(d_f16, dtype=np.uint16)
    N, K = q.shape
    if ls.shape != (N, K // 32) or d_f16.shape != (N, K // 256):
        raise ValueError("ls must be [N, K/32] and d_f16 [N, K/256]")
    nbytes = nvq_iq4_xs_weight_bytes(N, K)
    out = np.empty(max(nbytes, 1), np.uint8)
    _check(lib().nvq_pack_iq4_xs(*(a.ctypes.data_as(ctypes.c_void_p) for a in (q, ls, d_f16)), N, K,
                                 out.ctypes.data_as(ctypes.c_void_p)), "nvq_pack_iq4_xs")
    return out[:nbytes]


def _table(table) -> np.ndarray:
    t = np.ascontiguousarray(table, dtype=np.int8)
    if t.shape != (16,):
        raise ValueError("table must hold 16 int8 values")
    return t


def nvq_gemv_iq4_xs(w, table, q, d_f16, y, stream=None) -> None:
    import torch

    t = _table(table)
    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_iq4_xs_weight_bytes(N, K), "w")
    _check(lib().nvq_gemv_iq4_xs(_ptr(w), t.ctypes.data_as(ctypes.c_void_p), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y),
                                 _stream(stream, y)), "nvq_gemv_iq4_xs")


def nvq_gemm_iq4_xs(w, table, q, d_f16, y, workspace=None, stream=None) -> None:
    import torch

    t = _table(table)
    M, K = _acts(q, d_f16)
    N = y.shape[1]
    _need(y, torch.float32, (M, N), "y")
    _weights(w, nvq_iq4_xs_weight_bytes(N, K), "w")
    if workspace is None:
        workspace = _workspace(lib().nvq_gemm_workspace_bytes(NVQ_FMT_IQ4_XS, M, N, K), stream, y)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().nvq_gemm_iq4_xs(_ptr(w), t.ctypes.data_as(ctypes.c_void_p), _ptr(q), _ptr(d_f16), M, N, K, _ptr(y),
                                 _ptr(workspace), ws_bytes, _stream(stream, y)), "nvq_gemm_iq4_xs")


def nvq_debug_isums_iq4_xs(table, path: int, w, q, N: int, isums, stream=None) -> None:
    """isums int32 [M, N, K/16]: sum of table[code] * q per 16, from the dispatched kernel."""
    import torch

    t = _table(table)
    M, K = q.shape
    _need(q, torch.int8, (M, K), "q")
    _need(isums, torch.int32, (M, N, K // 16), "isums")
    _weights(w, nvq_iq4_xs_weight_bytes(N, K), "w")
    _check(lib().nvq_debug_isums_iq4_xs(t.ctypes.data_as(ctypes.c_void_p), int(path), _ptr(w), _ptr(q), M, N, K,
                                        _ptr(isums), _stream(stream, q)), "nvq_debug_isums_iq4_xs")


def nvq_debug_isums(fmt: int, path: int, w, q, N: int, isums, stream=None) -> None:
    """isums int32 [M, N, K/16]: integer per-16 sums from the chosen production path."""
    import torch

    M, K = q.shape
    _need(q, torch.int8, (M, K), "q")
    _need(isums, torch.int32, (M, N, K // 16), "isums")
    nbytes = {NVQ_FMT_NVFP4: nvq_nvfp4_weight_bytes, NVQ_FMT_Q4_1: nvq_q4_1_weight_bytes,
              NVQ_FMT_Q4_K: nvq_q4_k_weight_bytes}.get(fmt, nvq_q4_1_weight_bytes)(N, K)
    _weights(w, nbytes, "w")
    _check(lib().nvq_debug_isums(int(fmt), int(path), _ptr(w), _ptr(q), M, N, K, _ptr(isums),
                                 _stream(stream, q)), "nvq_debug_isums")


# ---------------------------------------------------------------------------
# paged key-value cache and attention
# ---------------------------------------------------------------------------

# A decode step makes these calls with a few microseconds of work each.  Each one first asks
# everything it needs to know of its tensors in one expression; only if something is wrong does
# a second look (_wrong_*) find out what, and raise.
_torch = None            # set with the tables
_row_types: dict = {}    # torch dtype -> NVQ_TYPE_*
_cache_types: dict = {}  # torch dtype -> NVQ_KV_*


def _attn_lib():
    """The library, loaded if it was not; the entries take _lib by itself once _torch says that both are there, so
    that is set last."""
    global _torch
    import torch

    L = lib()
    _row_types.update({torch.float32: NVQ_TYPE_F32, torch.float16: NVQ_TYPE_F16, torch.bfloat16: NVQ_TYPE_BF16})
    _cache_types.update({torch.int8: NVQ_KV_Q8_0, torch.float16: NVQ_KV_F16, torch.bfloat16: NVQ_KV_BF16})
    _torch = torch
    return L


def _wrong_rows(t, dtype, shape, name):
    if t is None or t.dim() != 3 or t.dtype not in _row_types:
        raise ValueError(f"{name}: a float32, float16 or bfloat16 tensor [rows, heads, D] is required")
    _need(t, dtype, shape, name)
    if t.stride(2) != 1:
        raise ValueError(f"{name}: a row's channels must be contiguous")


def _wrong_dense(t, dtype, shape, name):
    _need(t, dtype, shape, name)
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors passed to libnvq must be contiguous")


def _wrong_cache(k_cache, v_cache, k_d, v_d):
    if k_cache is None or k_cache.dim() != 4 or k_cache.dtype not in _cache_types:
        raise ValueError("k_cache: an int8 (Q8_0), float16 or bfloat16 tensor [n_pages, heads, page, D] is required")
    _wrong_dense(k_cache, k_cache.dtype, k_cache.shape, "k_cache")
    _wrong_dense(v_cache, k_cache.dtype, k_cache.shape, "v_cache")
    d_shape = (*k_cache.shape[:3], k_cache.shape[3] // 32)
    for t, name in ((k_d, "k_d"), (v_d, "v_d")):
        if k_cache.dtype != _torch.int8:
            if t is not None:
                raise ValueError(f"{name}: a 16-bit cache has no scales")
        elif t is None or t.shape != d_shape or t.element_size() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2-byte tensor [n_pages, heads, page, D/32]")


def _wrong_device(*tensors):
    """Pointers of another GPU must not reach a launch on the current one's stream."""
    here = _torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"tensor on {t.device}, expected the current device cuda:{here}")


def _cache_fine(fmt, shape, k_cache, v_cache, k_d, v_d):
    """Whether a cache [n_pages, heads, page, D] and its scales fit together (all contiguous)."""
    if not (v_cache.dtype is k_cache.dtype and v_cache.shape == shape and k_cache.is_contiguous() and v_cache.is_contiguous()):
        return False
    if fmt:
        return k_d is None and v_d is None
    d_shape = (shape[0], shape[1], shape[2], shape[3] // 32)
    return (k_d.shape == d_shape and v_d.shape == d_shape and k_d.element_size() == 2 and v_d.element_size() == 2
            and k_d.is_contiguous() and v_d.is_contiguous())


def _kv_copy(fn, name, k, v, slots, k_cache, v_cache, k_d, v_d, stream):
    here = -1
    try:
        fmt, shape, rows, dtype = _cache_types[k_cache.dtype], k_cache.shape, k.shape, k.dtype
        n_pages, heads, page, D = shape
        T = rows[0]
        ks, vs, code = k.stride(), v.stride(), _row_types[dtype]
        fine = (_cache_fine(fmt, shape, k_cache, v_cache, k_d, v_d) and rows == (T, heads, D) and v.shape == rows and v.dtype is dtype
                and ks[2] == 1 and vs[2] == 1 and slots.dtype is _torch.int64 and slots.shape == rows[:1] and slots.is_contiguous())
        if fine:
            here = _torch.cuda.current_device()
            fine = (k.get_device() == here and v.get_device() == here and slots.get_device() == here and k_cache.get_device() == here
                    and v_cache.get_device() == here and (fmt or k_d.get_device() == here and v_d.get_device() == here))
    except (AttributeError, KeyError, ValueError, IndexError):
        fine = False
    if not fine:
        _wrong_cache(k_cache, v_cache, k_d, v_d)
        T, (_, heads, _, D) = k.shape[0] if k is not None and k.dim() == 3 else -1, k_cache.shape
        _wrong_rows(k, k.dtype if k is not None else None, (T, heads, D), "k")
        _wrong_rows(v, k.dtype, (T, heads, D), "v")
        _wrong_dense(slots, _torch.int64, (T,), "slots")
        _wrong_device(k, v, slots, k_cache, v_cache, k_d, v_d)
        raise ValueError("k, v, slots and the cache do not fit together")
    st = fn(fmt, code, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slots.data_ptr(), T, heads, D, k_cache.data_ptr(), v_cache.data_ptr(),
            None if fmt else k_d.data_ptr(), None if fmt else v_d.data_ptr(), n_pages, page,
            _torch._C._cuda_getCurrentRawStream(here) if stream is None else int(stream))
    if st:
        _check(st, name)


def nvq_kv_write(k, v, slots, k_cache, v_cache, k_d=None, v_d=None, stream=None) -> None:
    """Rows k, v [T, Hkv, D] (float32, float16 or bfloat16; token and head strides free) into a paged cache
    [n_pages, Hkv, page, D] at slots int64 [T] (page number * page + place; negative: none).  An int8 cache is
    Q8_0 and takes the binary16 scales k_d, v_d [n_pages, Hkv, page, D/32]; a 16-bit one takes none."""
    L = _lib if _torch is not None else _attn_lib()
    _kv_copy(L.nvq_kv_write, "nvq_kv_write", k, v, slots, k_cache, v_cache, k_d, v_d, stream)


def nvq_kv_read(k_cache, v_cache, slots, k, v, k_d=None, v_d=None, stream=None) -> None:
    """The cache rows at slots int64 [T] into k, v [T, Hkv, D] (arguments as nvq_kv_write's)."""
    L = _lib if _torch is not None else _attn_lib()
    _kv_copy(L.nvq_kv_read, "nvq_kv_read", k, v, slots, k_cache, v_cache, k_d, v_d, stream)


def nvq_rope_table(P: int, R: int, base: float = 10000.0, inv_freq=None) -> np.ndarray:
    """The position rotation's table, float32 [P, R] on the host: of base^(-2 c / R), or of inv_freq [R/2]."""
    if inv_freq is None:
        if R < 1 or not base > 0:
            raise ValueError("nvq_rope_table: R and base must be positive")
        inv_freq = float(base) ** (-np.arange(R // 2) * 2.0 / R)
    inv_freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if inv_freq.shape != (R // 2,):
        raise ValueError("inv_freq must be [R/2]")
    out = np.empty((max(P, 0), max(R, 0)), np.float32)
    _check(lib().nvq_rope_table(inv_freq.ctypes.data_as(ctypes.c_void_p), P, R, out.ctypes.data_as(ctypes.c_void_p)), "nvq_rope_table")
    return out


@functools.lru_cache(maxsize=64)
def _sections(sections):
    return (ctypes.c_int32 * len(sections))(*sections)


_no_strides = (0, 0, 1)


def _weight_fine(w, D):
    return w is None or w.dtype is _torch.float32 and w.shape == (D,) and w.is_contiguous()


def _rope_fine(table, positions, sections, T, q_weight, k_weight, D):
    """Whether the table, the positions and the weights fit a call of T tokens; positions is [T] or [axes, T]."""
    shape = positions.shape
    axes = shape[0] if len(shape) == 2 else 1
    return (shape[-1] == T and (len(shape) == 2 or len(shape) == 1) and positions.dtype is _torch.int32 and positions.is_contiguous()
            and table.dtype is _torch.float32 and table.dim() == 2 and table.is_contiguous()
            and (axes == 1 if sections is None else len(sections) == axes and (axes > 1 or 2 * sections[0] == table.shape[1]))
            and _weight_fine(q_weight, D) and _weight_fine(k_weight, D))


def _rope_here(table, positions, q_weight, k_weight, here):
    return (table.get_device() == here and positions.get_device() == here and (q_weight is None or q_weight.get_device() == here)
            and (k_weight is None or k_weight.get_device() == here))


def _wrong_rope(table, positions, sections, T, q_weight, k_weight, D):
    if table is None or table.dim() != 2:
        raise ValueError("table: float32 [positions, R] is required")
    _wrong_dense(table, _torch.float32, table.shape, "table")
    if positions is None or positions.dim() not in (1, 2):
        raise ValueError("positions: int32 [T] or [axes, T] is required")
    _wrong_dense(positions, _torch.int32, (*positions.shape[:-1], T), "positions")
    axes = positions.shape[0] if positions.dim() == 2 else 1
    if (axes != 1) if sections is None else len(sections) != axes:
        raise ValueError("sections: a number of pairs for each axis of positions is required")
    if sections is not None and axes == 1 and 2 * sections[0] != table.shape[1]:
        raise ValueError(f"sections: one axis turns all {table.shape[1] // 2} pairs")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _wrong_dense(w, _torch.float32, (D,), name)


def nvq_qk_norm_rope(q, k, table, positions, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, pairs=NVQ_ROPE_HALVES, sections=None,
                     stream=None) -> None:
    """Query and key heads [T, H, D] (strides free), normed (weights float32 [D]; None: not) and turned by the rows
    of table float32 [P, R] at positions int32 [T], into q_out and k_out (strides free, one type, perhaps
    another than q's).  q with q_out, or k with k_out, may be None.  Several axes: positions [axes, T], sections: pairs
    of each."""
    L = _lib if _torch is not None else _attn_lib()
    here = -1
    try:
        x, o = (k, k_out) if q is None else (q, q_out)
        T, _, D = x.shape
        dtype, out_dtype = x.dtype, o.dtype
        code, out_code = _row_types[dtype], _row_types[out_dtype]
        qs, qo, Hq, ks, ko, Hkv = _no_strides, _no_strides, 1, _no_strides, _no_strides, 1
        fine = _rope_fine(table, positions, sections, T, q_weight, k_weight, D)
        if q is not None:
            shape, qs, qo = q.shape, q.stride(), q_out.stride()
            Hq = shape[1]
            fine = (fine and shape == (T, Hq, D) and q.dtype is dtype and q_out.dtype is out_dtype and q_out.shape == shape and qs[2] == 1 and qo[2] == 1)
        else:
            fine = fine and q_out is None
        if k is not None:
            shape, ks, ko = k.shape, k.stride(), k_out.stride()
            Hkv = shape[1]
            fine = (fine and shape == (T, Hkv, D) and k.dtype is dtype and k_out.dtype is out_dtype and k_out.shape == shape and ks[2] == 1 and ko[2] == 1)
        else:
            fine = fine and k_out is None
        if fine:
            here = _torch.cuda.current_device()
            fine = ((q is None or q.get_device() == here and q_out.get_device() == here) and (k is None or k.get_device() == here and k_out.get_device() == here)
                    and _rope_here(table, positions, q_weight, k_weight, here))
    except (AttributeError, KeyError, ValueError, IndexError, TypeError):
        fine = False
    if not fine:
        if q is None and k is None or (q is None) != (q_out is None) or (k is None) != (k_out is None):
            raise ValueError("q with q_out, k with k_out, or both are required")
        x, o = (k, k_out) if q is None else (q, q_out)
        _wrong_rows(x, x.dtype, x.shape, "k" if q is None else "q")
        T, D = x.shape[0], x.shape[2]
        for y, out, name in ((q, q_out, "q"), (k, k_out, "k")):
            if y is not None:
                _wrong_rows(y, x.dtype, (T, y.shape[1] if y.dim() == 3 else -1, D), name)
                _wrong_rows(out, o.dtype, y.shape, name + "_out")
        _wrong_rope(table, positions, sections, T, q_weight, k_weight, D)
        _wrong_device(q, k, table, positions, q_out, k_out, q_weight, k_weight)
        raise ValueError("q, k, their outputs, table, positions and weights do not fit together")
    st = L.nvq_qk_norm_rope(code, out_code, None if q is None else q.data_ptr(), qs[0], qs[1], None if k is None else k.data_ptr(), ks[0], ks[1], T, Hq,
                            Hkv, D, None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(), eps,
                            table.data_ptr(), table.shape[0], table.shape[1], pairs, positions.data_ptr(), 1 if sections is None else len(sections),
                            None if sections is None or len(sections) == 1 else _sections(tuple(sections)), None if q is None else q_out.data_ptr(),
                            qo[0], qo[1], None if k is None else k_out.data_ptr(), ko[0], ko[1],
                            _torch._C._cuda_getCurrentRawStream(here) if stream is None else int(stream))
    if st:
        _check(st, "nvq_qk_norm_rope")


def nvq_rope_kv_write(q, k, v, table, positions, slots, q_out, k_cache, v_cache, k_d=None, v_d=None, q_weight=None, k_weight=None, eps=1e-6,
                      pairs=NVQ_ROPE_HALVES, sections=None, stream=None) -> None:
    """What a layer does with its QKV product, in one launch: keys [T, Hkv, D], normed and turned as nvq_qk_norm_rope's, and
    values into a paged cache at slots as nvq_kv_write's; queries [T, Hq, D], normed and turned, into q_out (both
    may be None)."""
    L = _lib if _torch is not None else _attn_lib()
    here = -1
    try:
        fmt, shape, rows, dtype = _cache_types[k_cache.dtype], k_cache.shape, k.shape, k.dtype
        n_pages, heads, page, D = shape
        T = rows[0]
        ks, vs, code, out_code = k.stride(), v.stride(), _row_types[dtype], 0
        qs, qo, Hq = _no_strides, _no_strides, 1
        fine = (_cache_fine(fmt, shape, k_cache, v_cache, k_d, v_d) and rows == (T, heads, D) and v.shape == rows and v.dtype is dtype
                and ks[2] == 1 and vs[2] == 1 and slots.dtype is _torch.int64 and slots.shape == rows[:1] and slots.is_contiguous()
                and _rope_fine(table, positions, sections, T, q_weight, k_weight, D))
        if q is not None:
            shape, qs, qo, out_code = q.shape, q.stride(), q_out.stride(), _row_types[q_out.dtype]
            Hq = shape[1]
            fine = (fine and shape == (T, Hq, D) and q.dtype is dtype and q_out.shape == shape and qs[2] == 1 and qo[2] == 1)
        else:
            fine = fine and q_out is None
        if fine:
            here = _torch.cuda.current_device()
            fine = (k.get_device() == here and v.get_device() == here and slots.get_device() == here and k_cache.get_device() == here
                    and v_cache.get_device() == here and (fmt or k_d.get_device() == here and v_d.get_device() == here)
                    and (q is None or q.get_device() == here and q_out.get_device() == here) and _rope_here(table, positions, q_weight, k_weight, here))
    except (AttributeError, KeyError, ValueError, IndexError, TypeError):
        fine = False
    if not fine:
        _wrong_cache(k_cache, v_cache, k_d, v_d)
        T, (_, heads, _, D) = k.shape[0] if k is not None and k.dim() == 3 else -1, k_cache.shape
        _wrong_rows(k, k.dtype if k is not None else None, (T, heads, D), "k")
        _wrong_rows(v, k.dtype, (T, heads, D), "v")
        _wrong_dense(slots, _torch.int64, (T,), "slots")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out are given together or not at all")
        if q is not None:
            _wrong_rows(q, k.dtype, (T, q.shape[1] if q.dim() == 3 else -1, D), "q")
            _wrong_rows(q_out, q_out.dtype, q.shape, "q_out")
        _wrong_rope(table, positions, sections, T, q_weight, k_weight, D)
        _wrong_device(q, k, v, table, positions, slots, q_out, k_cache, v_cache, k_d, v_d, q_weight, k_weight)
        raise ValueError("q, k, v, q_out, table, positions, slots, weights and the cache do not fit together")
    st = L.nvq_rope_kv_write(fmt, code, out_code, None if q is None else q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                             T, Hq, heads, D, None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(), eps,
                             table.data_ptr(), table.shape[0], table.shape[1], pairs, positions.data_ptr(), 1 if sections is None else len(sections),
                             None if sections is None or len(sections) == 1 else _sections(tuple(sections)), slots.data_ptr(),
                             None if q is None else q_out.data_ptr(), qo[0], qo[1], k_cache.data_ptr(), v_cache.data_ptr(),
                             None if fmt else k_d.data_ptr(), None if fmt else v_d.data_ptr(), n_pages, page,
                             _torch._C._cuda_getCurrentRawStream(here) if stream is None else int(stream))
    if st:
        _check(st, "nvq_rope_kv_write")


@functools.lru_cache(maxsize=256)  # a function of its arguments alone; a decode loop asks it each step
def nvq_attn_decode_workspace_bytes(B: int, Hq: int, Hkv: int, D: int, max_pages: int, page: int) -> int:
    return int(lib().nvq_attn_decode_workspace_bytes(B, Hq, Hkv, D, max_pages, page))


def _attn_decode(fn, name, q, k_cache, v_cache, table, lengths, out, k_d, v_d, scale, window, sinks, more, workspace, stream):
    here = -1
    try:
        fmt, shape, rows, dtype = _cache_types[k_cache.dtype], k_cache.shape, q.shape, q.dtype
        n_pages, heads, page, D = shape
        B, Hq, max_pages = rows[0], rows[1], table.shape[1]
        qs, code, i32 = q.stride(), _row_types[dtype], _torch.int32
        fine = (_cache_fine(fmt, shape, k_cache, v_cache, k_d, v_d) and rows == (B, Hq, D) and out.shape == rows and out.dtype is dtype
                and qs[2] == 1 and out.is_contiguous() and table.dtype is i32 and table.shape == (B, max_pages) and table.is_contiguous()
                and lengths.dtype is i32 and lengths.shape == rows[:1] and lengths.is_contiguous())
        if fine:
            here = _torch.cuda.current_device()
            fine = (q.get_device() == here and out.get_device() == here and k_cache.get_device() == here and v_cache.get_device() == here
                    and table.get_device() == here and lengths.get_device() == here
                    and (fmt or k_d.get_device() == here and v_d.get_device() == here)
                    and (workspace is None or workspace.get_device() == here and workspace.is_contiguous()))
    except (AttributeError, KeyError, ValueError, IndexError):
        fine = False
    if not fine:
        _wrong_cache(k_cache, v_cache, k_d, v_d)
        B, Hq = q.shape[:2] if q is not None and q.dim() == 3 else (-1, -1)
        D = k_cache.shape[3]
        _wrong_rows(q, q.dtype if q is not None else None, (B, Hq, D), "q")
        _wrong_dense(out, q.dtype, (B, Hq, D), "out")
        _wrong_dense(table, _torch.int32, (B, table.shape[1] if table is not None and table.dim() == 2 else -1), "table")
        _wrong_dense(lengths, _torch.int32, (B,), "lengths")
        _wrong_device(q, k_cache, v_cache, table, lengths, out, k_d, v_d, workspace)
        raise ValueError("q, out, the cache, table, lengths and workspace do not fit together (all but q contiguous)")
    if workspace is None:
        pages = max_pages if not window else min(max_pages, (window + sinks + 30) // max(page, 1) + 1)  # a longer table's other pages are not read
        workspace = _workspace(nvq_attn_decode_workspace_bytes(B, Hq, heads, D, pages, page), stream, q)
    wp, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = fn(fmt, code, q.data_ptr(), qs[0], qs[1], B, Hq, heads, D, k_cache.data_ptr(), v_cache.data_ptr(),
            None if fmt else k_d.data_ptr(), None if fmt else v_d.data_ptr(), n_pages, page, table.data_ptr(), max_pages,
            lengths.data_ptr(), max(D, 1) ** -0.5 if scale is None else scale, *more, out.data_ptr(), wp, ws_bytes,
            _torch._C._cuda_getCurrentRawStream(here) if stream is None else int(stream))
    if st:
        _check(st, name)


def nvq_attn_decode(q, k_cache, v_cache, table, lengths, out, k_d=None, v_d=None, scale=None, workspace=None,
                    stream=None) -> None:
    """One new token per sequence: q [B, Hq, D] (strides free), the paged cache, table int32 [B, max_pages] and
    lengths int32 [B] -> out [B, Hq, D] of q's type.  scale: 1 / sqrt(D) unless given."""
    L = _lib if _torch is not None else _attn_lib()
    _attn_decode(L.nvq_attn_decode, "nvq_attn_decode", q, k_cache, v_cache, table, lengths, out, k_d, v_d, scale, 0, 0, (), workspace, stream)


def nvq_attn_decode_window(q, k_cache, v_cache, table, lengths, out, k_d=None, v_d=None, window=0, sinks=0, scale=None, workspace=None,
                           stream=None) -> None:
    """nvq_attn_decode over the last `window` keys of each sequence (0: all) and its first `sinks`; the other pages may be
    gone."""
    L = _lib if _torch is not None else _attn_lib()
    _attn_decode(L.nvq_attn_decode_window, "nvq_attn_decode_window", q, k_cache, v_cache, table, lengths, out, k_d, v_d, scale, window, sinks,
                 (window, sinks), workspace, stream)


def nvq_attn_prompt(q, k, v, cu_q, cu_k, out, scale=None, causal=True, stream=None) -> None:
    """Packed prompts: q [Tq, Hq, D], k, v [Tk, Hkv, D] (float16 or bfloat16, strides free), cu_q, cu_k int32 [B+1]
    -> out [Tq, Hq, D] (strides free).  Query i of m sees keys j <= i + n - m of its n (causal), else all.
    scale: 1 / sqrt(D) unless given."""
    L = _lib if _torch is not None else _attn_lib()
    here = -1
    try:
        shape, keys, dtype, i32 = q.shape, k.shape, q.dtype, _torch.int32
        (Tq, Hq, D), (Tk, Hkv, _) = shape, keys
        qs, ks, vs, ps, n = q.stride(), k.stride(), v.stride(), out.stride(), cu_q.shape
        fine = (dtype in _row_types and k.dtype is dtype and v.dtype is dtype and out.dtype is dtype and out.shape == shape and keys[2] == D
                and v.shape == keys and qs[2] == ks[2] == vs[2] == ps[2] == 1 and len(n) == 1 and n[0] > 0 and cu_k.shape == n and cu_q.dtype is i32
                and cu_k.dtype is i32 and cu_q.is_contiguous() and cu_k.is_contiguous())
        if fine:
            here = _torch.cuda.current_device()
            fine = (q.get_device() == here and k.get_device() == here and v.get_device() == here and out.get_device() == here
                    and cu_q.get_device() == here and cu_k.get_device() == here)
    except (AttributeError, KeyError, ValueError, IndexError):
        fine = False
    if not fine:
        shape = tuple(q.shape) if q is not None and q.dim() == 3 else (-1, -1, -1)
        _wrong_rows(q, q.dtype if q is not None else None, shape, "q")
        keys = (*(k.shape[:2] if k is not None and k.dim() == 3 else (-1, -1)), shape[2])
        for t, s, name in ((k, keys, "k"), (v, keys, "v"), (out, shape, "out")):
            _wrong_rows(t, q.dtype, s, name)
        if cu_q is None or cu_q.dim() != 1 or cu_q.shape[0] < 1:
            raise ValueError("cu_q: int32 [B + 1] is required")
        _wrong_dense(cu_q, _torch.int32, cu_q.shape, "cu_q")
        _wrong_dense(cu_k, _torch.int32, cu_q.shape, "cu_k")
        _wrong_device(q, k, v, cu_q, cu_k, out)
        raise ValueError("q, k, v, out, cu_q and cu_k do not fit together")
    strides = _Strides(qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], ps[0], ps[1])
    st = L.nvq_attn_prompt(_row_types[dtype], q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), strides, cu_q.data_ptr(), cu_k.data_ptr(),
                           n[0] - 1, Tq, Tk, Hq, Hkv, D, max(D, 1) ** -0.5 if scale is None else scale, 1 if causal else 0,
                           _torch._C._cuda_getCurrentRawStream(here) if stream is None else int(stream))
    if st:
        _check(st, "nvq_attn_prompt")


_Strides = ctypes.c_int64 * 8
_Strides4 = ctypes.c_int64 * 4


@functools.lru_cache(maxsize=256)
def nvq_attn_chunk_workspace_bytes(fmt: int, B: int, Tq: int, Hq: int, Hkv: int, D: int, max_pages: int, page: int, window: int = 0, sinks: int = 0) -> int:
    return int(lib().nvq_attn_chunk_workspace_bytes(fmt, B, Tq, Hq, Hkv, D, max_pages, page, window, sinks))


def nvq_attn_chunk(q, k_cache, v_cache, table, cu_q, lengths, out, k_d=None, v_d=None, window=0, sinks=0, scale=None, workspace=None,
                   stream=None) -> None:
    """New tokens over the paged cache that holds them: q [Tq, Hq, D] (float16 or bfloat16, a 16-bit cache's type; strides free)
    packed by cu_q int32 [B+1], table int32 [B, max_pages], lengths int32 [B] (keys, the new tokens' among them) -> out
    [Tq, Hq, D] (strides free).  Query i of m sees keys j <= p = i + n - m of its n; with a window those of j > p - window or
    j < sinks.  scale: 1 / sqrt(D) unless given."""
    L = _lib if _torch is not None else _attn_lib()
    here = -1
    try:
        fmt, shape, rows, dtype = _cache_types[k_cache.dtype], k_cache.shape, q.shape, q.dtype
        n_pages, heads, page, D = shape
        Tq, Hq, _ = rows
        B, max_pages = table.shape
        qs, ps, code, i32 = q.stride(), out.stride(), _row_types[dtype], _torch.int32
        fine = (_cache_fine(fmt, shape, k_cache, v_cache, k_d, v_d) and rows == (Tq, Hq, D) and out.shape == rows and out.dtype is dtype
                and qs[2] == 1 and ps[2] == 1 and table.dtype is i32 and table.is_contiguous() and cu_q.dtype is i32 and cu_q.shape == (B + 1,)
                and cu_q.is_contiguous() and lengths.dtype is i32 and lengths.shape == (B,) and lengths.is_contiguous())
        if fine:
            here = _torch.cuda.current_device()
            fine = (q.get_device() == here and out.get_device() == here and k_cache.get_device() == here and v_cache.get_device() == here
                    and table.get_device() == here and cu_q.get_device() == here and lengths.get_device() == here
                    and (fmt or k_d.get_device() == here and v_d.get_device() == here)
                    and (workspace is None or workspace.get_device() == here and workspace.is_contiguous()))
    except (AttributeError, KeyError, ValueError, IndexError):
        fine = False
    if not fine:
        _wrong_cache(k_cache, v_cache, k_d, v_d)
        shape = (*(q.shape[:2] if q is not None and q.dim() == 3 else (-1, -1)), k_cache.shape[3])
        _wrong_rows(q, q.dtype if q is not None else None, shape, "q")
        _wrong_rows(out, q.dtype, shape, "out")
        if table is None or table.dim() != 2:
            raise ValueError("table: int32 [B, max_pages] is required")
        _wrong_dense(table, _torch.int32, table.shape, "table")
        _wrong_dense(cu_q, _torch.int32, (table.shape[0] + 1,), "cu_q")
        _wrong_dense(lengths, _torch.int32, table.shape[:1], "lengths")
        _wrong_device(q, k_cache, v_cache, table, cu_q, lengths, out, k_d, v_d, workspace)
        raise ValueError("q, out, the cache, table, cu_q, lengths and workspace do not fit together")
    if workspace is None:
        workspace = _workspace(nvq_attn_chunk_workspace_bytes(fmt, B, Tq, Hq, heads, D, max_pages, page, window, sinks), stream, q)
    wp, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = L.nvq_attn_chunk(fmt, code, q.data_ptr(), _Strides4(qs[0], qs[1], ps[0], ps[1]), B, Tq, Hq, heads, D, k_cache.data_ptr(), v_cache.data_ptr(),
                          None if fmt else k_d.data_ptr(), None if fmt else v_d.data_ptr(), n_pages, page, table.data_ptr(), max_pages,
                          cu_q.data_ptr(), lengths.data_ptr(), max(D, 1) ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(), wp, ws_bytes,
                          _torch._C._cuda_getCurrentRawStream(here) if stream is None else int(stream))
    if st:
        _check(st, "nvq_attn_chunk")


# ---------------------------------------------------------------------------
# measurement probes (include/nvq_probe.h): ceilings, not part of the product path
# ---------------------------------------------------------------------------

def nvq_probe_read(src, blocks: int, sink, stream=None) -> None:
    """Stream every byte of the device tensor ``src`` (size a multiple of 16) with
    16-byte non-temporal loads over ``blocks`` blocks of 256 threads; ``sink``: int32
    or uint32 device tensor of >= 4 * blocks elements."""
    nbytes = src.numel() * src.element_size()
    if sink.element_size() != 4 or sink.numel() < 4 * blocks:
        raise ValueError("sink: 4-byte tensor of at least 4 * blocks elements required")
    _check(lib().nvq_probe_read(_ptr(src), nbytes, int(blocks), _ptr(sink), _stream(stream, src)), "nvq_probe_read")


def nvq_probe_gemv_loads(w, N: int, K: int, splits: int, waves: int, batch: int, sink, stream=None) -> None:
    """The weight loads of the single-token decode GEMV over packed NVFP4 ``w`` (N x K)
    and nothing else; ``sink``: 4-byte device tensor of >= waves * ceil(N/16) * splits
    elements."""
    _weights(w, nvq_nvfp4_weight_bytes(N, K), "w")
    if sink.element_size() != 4 or sink.numel() < waves * ((N + 15) // 16) * splits:
        raise ValueError("sink: 4-byte tensor of at least waves * ceil(N/16) * splits elements required")
    _check(lib().nvq_probe_gemv_loads(_ptr(w), int(N), int(K), int(splits), int(waves), int(batch), _ptr(sink),
                                      _stream(stream, w)), "nvq_probe_gemv_loads")


def nvq_probe_mfma(blocks: int, iters: int, random_operands: bool, out, stream=None) -> None:
    """Back-to-back v_mfma_f32_32x32x16_f16 on register operands; ``out``: float32
    device tensor of >= 256 * blocks elements.  Flops per call:
    blocks * 4 * 12 * iters * 32768."""
    import torch

    if out.dtype != torch.float32 or out.numel() < 256 * blocks:
        raise ValueError("out: float32 tensor of at least 256 * blocks elements required")
    _check(lib().nvq_probe_mfma(int(blocks), int(iters), 1 if random_operands else 0, _ptr(out), _stream(stream, out)),
           "nvq_probe_mfma")
