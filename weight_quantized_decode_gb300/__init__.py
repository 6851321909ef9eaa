"""weight_quantized_decode_gb300 -- block-quantised (GGUF Q4_0 / Q8_0) weight x
activation products for single-stream decode on one GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/qmv.h`` (``libqmv.so``,
built in-tree by ``build.py``).  It only marshals arguments: every step of the
computation runs in the library's CUDA kernels.  There is no CPU path; calls
raise if the library is missing or a tensor is not on a CUDA device.

Functions (same names as the C ABI):
    qmv_q4_0(W, x, y=None, stream=None)          -> y fp32 [M, N]
    qmv_q8_0(W, x, y=None, stream=None)          -> y fp32 [M, N]
    qmv_q4_0_swiglu(W_gate, W_up, x, y=None, stream=None) -> silu(gate) * up, fp32 [M, N]
    qmv_q4_0_f32, qmv_q4_0_swiglu_f32            -> the same two with fp32 x
    qmv_q2w(W, x, y=None, stream=None)           -> plain 2-bit weights, y fp32 [M, N]
    qmv_q4_0_q8_1(W, x, y=None, stream=None)     -> Q4_0 against Q8_1-quantised x (integer dots)
    qmv_quantize_q8_1(x, stream=None)            -> (q, d_bits, sumq) of the Q8_1 activations
    qmv_q4_0_q8_1_pre(W, q, d_bits, sumq, ...)   -> the Q8_1 product on activations already quantised
    qmv_moe(W_pool, expert_idx, n_experts, x, N, y=None, stream=None)
    qmm_q4_0_prefill(W, x, y=None, stream=None)  -> y fp32 [M, N]
    qmm_q8_0_prefill(W, x, y=None, stream=None)  -> y fp32 [M, N]
    KvCache(k, v, k_scale=None, v_scale=None), qmv_kv_cache(...) -> a paged key/value cache (fp16 or int8 rows)
    qmv_kv_pages(lens, n_new, free, table, page, tokens, ...) -> KvPages: start, kv_len, slots, pos, request, head
                                                                (with held=...: KvPagesHeld, and held)
    qmv_kv_append(qkv, cache, slots, n_heads, pos, cos, sin, ...) -> rotated q; k, v rows written to the cache
    qmv_tree_attn(q, cache, table, start, kv_len, tree=None, ...) -> attention over the cache, fp16 [T, heads, D]
    qmv_tree_attn_workspace(device=None)         -> the workspace a program keeps for qmv_tree_attn
    qmv_device_status(stream=None)               -> int (QMV_DEV_* bits, cleared)
    qmv_read_probe(buf, out=None, stream=None)   -> checksum tensor (read-only bandwidth probe)
    qmv_set_pdl(enable), qmv_status_str(code), qmv_version()
Raw-pointer forms (``*_ptr``) take integers and are what the benchmark times.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
# QMV_LIB selects another build of the same library (the phase-timeline
# variant of phase_timeline.py); there is no CPU path either way.
LIB_PATH = os.environ.get("QMV_LIB") or os.path.join(_HERE, "libqmv.so")

QMV_OK = 0
QMV_DEV_BAD_EXPERT = 0x1
QMV_DEV_TIMEOUT = 0x2
QMV_DEV_BAD_PAGE = 0x4
QMV_DEV_NO_PAGES = 0x8
QMV_DEV_BAD_LENGTH = 0x10
QMV_KV_F16 = 0
QMV_KV_Q8 = 1
Q4_0_BLOCK_BYTES = 18
Q8_0_BLOCK_BYTES = 34
Q2W_BLOCK_BYTES = 10

_lock = threading.Lock()
_lib = None


class QmvError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {qmv_status_str(code)} ({code})")
        self.code = code


def lib():
    """Load ``libqmv.so`` (raises loudly if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run weight_quantized_decode_gb300/build.py "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64 = ctypes.c_void_p, ctypes.c_int64
        for name in ("qmv_q4_0", "qmv_q8_0", "qmm_q4_0_prefill", "qmm_q8_0_prefill", "qmv_q4_0_f32", "qmv_q2w", "qmv_q4_0_q8_1",
                     "qmv_q8_0_q8_1"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [vp, vp, vp, i64, i64, i64, vp]
        L.qmv_moe.restype = ctypes.c_int
        L.qmv_moe.argtypes = [vp, vp, i64, vp, vp, i64, i64, i64, vp]
        L.qmv_q4_0_swiglu.restype = ctypes.c_int
        L.qmv_q4_0_swiglu.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        L.qmv_q4_0_q8_1_pre.restype = ctypes.c_int
        L.qmv_q4_0_q8_1_pre.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp]
        L.qmv_q8_0_q8_1_pre.restype = ctypes.c_int
        L.qmv_q8_0_q8_1_pre.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        L.qmv_quantize_q8_1.restype = ctypes.c_int
        L.qmv_quantize_q8_1.argtypes = [vp, vp, vp, vp, i64, i64, vp]
        L.qmv_q4_0_swiglu_f32.restype = ctypes.c_int
        L.qmv_q4_0_swiglu_f32.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        L.qmv_device_status.restype = ctypes.c_int
        L.qmv_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int32)]
        L.qmv_read_probe.restype = ctypes.c_int
        L.qmv_read_probe.argtypes = [vp, i64, vp, vp]
        ci = ctypes.c_int
        L.qmv_kv_pages.restype = ci
        L.qmv_kv_pages.argtypes = [vp, vp, vp, i64, vp, vp, i64] + [vp] * 7 + [i64] * 5 + [vp]
        L.qmv_kv_pages_held.restype = ci
        L.qmv_kv_pages_held.argtypes = [vp, vp, vp, i64, vp, vp, i64] + [vp] * 9 + [i64] * 5 + [vp]
        L.qmv_kv_append.restype = ci
        L.qmv_kv_append.argtypes = [vp, i64, ci, vp, vp, vp, vp, i64, i64, ci, vp, vp, vp, vp, vp, ci] + [i64] * 7 + [vp]
        L.qmv_tree_attn_workspace.restype = i64
        L.qmv_tree_attn_workspace.argtypes = []
        L.qmv_tree_attn.restype = ci
        L.qmv_tree_attn.argtypes = [vp, i64, vp, vp, vp, vp, ci, i64, i64, i64, vp, i64, vp, vp, vp, i64, vp, vp, vp,
                                    i64] + [i64] * 5 + [vp]
        L.qmv_set_pdl.restype = None
        L.qmv_set_pdl.argtypes = [ctypes.c_int]
        L.qmv_status_str.restype = ctypes.c_char_p
        L.qmv_status_str.argtypes = [ctypes.c_int]
        L.qmv_version.restype = ctypes.c_char_p
        L.qmv_version.argtypes = []
        _lib = L
        return L


def qmv_status_str(code: int) -> str:
    return lib().qmv_status_str(int(code)).decode()


def qmv_version() -> str:
    return lib().qmv_version().decode()


def qmv_set_pdl(enable: bool) -> None:
    lib().qmv_set_pdl(1 if enable else 0)


# -- raw-pointer entry points ------------------------------------------------------

def _check(fn, code):
    if code != QMV_OK:
        raise QmvError(fn, code)


def qmv_q4_0_swiglu_ptr(W_gate: int, W_up: int, x: int, y: int, N: int, K: int, M: int,
                        stream: int = 0) -> None:
    _check("qmv_q4_0_swiglu", lib().qmv_q4_0_swiglu(W_gate, W_up, x, y, N, K, M, stream))


def qmv_q4_0_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmv_q4_0", lib().qmv_q4_0(W, x, y, N, K, M, stream))


def qmv_q4_0_f32_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmv_q4_0_f32", lib().qmv_q4_0_f32(W, x, y, N, K, M, stream))


def qmv_q4_0_swiglu_f32_ptr(W_gate: int, W_up: int, x: int, y: int, N: int, K: int, M: int,
                            stream: int = 0) -> None:
    _check("qmv_q4_0_swiglu_f32", lib().qmv_q4_0_swiglu_f32(W_gate, W_up, x, y, N, K, M, stream))


def qmv_q8_0_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmv_q8_0", lib().qmv_q8_0(W, x, y, N, K, M, stream))


def qmv_q4_0_q8_1_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmv_q4_0_q8_1", lib().qmv_q4_0_q8_1(W, x, y, N, K, M, stream))


def qmv_q4_0_q8_1_pre_ptr(W: int, q: int, d_bits: int, sumq: int, y: int, N: int, K: int, M: int,
                          stream: int = 0) -> None:
    _check("qmv_q4_0_q8_1_pre", lib().qmv_q4_0_q8_1_pre(W, q, d_bits, sumq, y, N, K, M, stream))


def qmv_q8_0_q8_1_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmv_q8_0_q8_1", lib().qmv_q8_0_q8_1(W, x, y, N, K, M, stream))


def qmv_q8_0_q8_1_pre_ptr(W: int, q: int, d_bits: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmv_q8_0_q8_1_pre", lib().qmv_q8_0_q8_1_pre(W, q, d_bits, y, N, K, M, stream))


def qmv_quantize_q8_1_ptr(x: int, q: int, d_bits: int, sumq: int, M: int, K: int, stream: int = 0) -> None:
    _check("qmv_quantize_q8_1", lib().qmv_quantize_q8_1(x, q, d_bits, sumq, M, K, stream))


def qmv_q2w_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmv_q2w", lib().qmv_q2w(W, x, y, N, K, M, stream))


def qmv_moe_ptr(W_pool: int, idx: int, n_experts: int, x: int, y: int, N: int, K: int, M: int,
                stream: int = 0) -> None:
    _check("qmv_moe", lib().qmv_moe(W_pool, idx, n_experts, x, y, N, K, M, stream))


def qmm_q4_0_prefill_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmm_q4_0_prefill", lib().qmm_q4_0_prefill(W, x, y, N, K, M, stream))


def qmm_q8_0_prefill_ptr(W: int, x: int, y: int, N: int, K: int, M: int, stream: int = 0) -> None:
    _check("qmm_q8_0_prefill", lib().qmm_q8_0_prefill(W, x, y, N, K, M, stream))


def qmv_read_probe_ptr(buf: int, nbytes: int, out: int, stream: int = 0) -> None:
    _check("qmv_read_probe", lib().qmv_read_probe(buf, nbytes, out, stream))


# -- torch-tensor entry points ---------------------------------------------------------

_torch_module = _int32_type = None


def _torch():
    global _torch_module, _int32_type
    if _torch_module is None:
        import torch
        _torch_module, _int32_type = torch, torch.int32
    return _torch_module


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _on_device(fn, *tensors):
    """All tensors on one CUDA device; returns a context that makes it current.
    The library launches on the current device and takes its status word and
    SM count from it, so a call on another device's tensors must switch first."""
    torch = _torch()
    dev = tensors[0].device
    for t in tensors[1:]:
        if t.device != dev:
            raise ValueError(f"{fn}: all tensors must be on one device ({dev} and {t.device})")
    return torch.cuda.device(dev)


def _check_y(y, M, N, fn):
    torch = _torch()
    if not (y.is_cuda and y.dtype == torch.float32 and y.is_contiguous() and y.numel() == M * N):
        raise ValueError(f"{fn}: y must be a contiguous CUDA float32 tensor of {M}x{N}")


def _prep(W, x, y, block_bytes, fn, x_dtype=None):
    torch = _torch()
    x_dtype = torch.float16 if x_dtype is None else x_dtype
    if not (W.is_cuda and x.is_cuda):
        raise TypeError(f"{fn}: W and x must be CUDA tensors (no CPU path)")
    if W.dtype != torch.uint8:
        raise TypeError(f"{fn}: W must be uint8 GGUF bytes")
    if x.dtype != x_dtype:
        raise TypeError(f"{fn}: x must be {str(x_dtype).replace('torch.', '')}")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if not (W.is_contiguous() and x.is_contiguous()):
        raise ValueError(f"{fn}: W and x must be contiguous")
    M, K = x.shape
    if K % 32:
        raise ValueError(f"{fn}: K={K} is not a multiple of 32")
    row_bytes = (K // 32) * block_bytes
    if row_bytes == 0:
        N = W.shape[0] if W.dim() >= 1 else 0
    else:
        if W.numel() % row_bytes:
            raise ValueError(f"{fn}: W size {W.numel()} is not a whole number of rows of {row_bytes} bytes")
        N = W.numel() // row_bytes
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    else:
        _check_y(y, M, N, fn)
    return W, x, y, N, K, M


def qmv_q4_0(W, x, y=None, stream=None):
    """y[M, N] = x[M, K] @ dequant(W)^T for Q4_0 weights ``W`` (uint8, N rows)."""
    W, x, y, N, K, M = _prep(W, x, y, Q4_0_BLOCK_BYTES, "qmv_q4_0")
    with _on_device("qmv_q4_0", W, x, y):
        qmv_q4_0_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def qmv_q4_0_f32(W, x, y=None, stream=None):
    """qmv_q4_0 with float32 activations, rounded to fp16 inside the kernel."""
    W, x, y, N, K, M = _prep(W, x, y, Q4_0_BLOCK_BYTES, "qmv_q4_0_f32", _torch().float32)
    with _on_device("qmv_q4_0_f32", W, x, y):
        qmv_q4_0_f32_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def _check_up(W_gate, W_up, fn):
    torch = _torch()
    if not (W_up.is_cuda and W_up.dtype == torch.uint8 and W_up.is_contiguous()
            and W_up.numel() == W_gate.numel()):
        raise ValueError(f"{fn}: W_up must be a contiguous CUDA uint8 table shaped like W_gate")


def qmv_q4_0_swiglu(W_gate, W_up, x, y=None, stream=None):
    """y[M, N] = silu(x @ dequant(W_gate)^T) * (x @ dequant(W_up)^T) for two
    Q4_0 tables of N rows each (the MLP's gate + up + SwiGLU in one call)."""
    W_gate, x, y, N, K, M = _prep(W_gate, x, y, Q4_0_BLOCK_BYTES, "qmv_q4_0_swiglu")
    _check_up(W_gate, W_up, "qmv_q4_0_swiglu")
    with _on_device("qmv_q4_0_swiglu", W_gate, W_up, x, y):
        qmv_q4_0_swiglu_ptr(W_gate.data_ptr(), W_up.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M,
                            _stream_handle(stream))
    return y


def qmv_q4_0_swiglu_f32(W_gate, W_up, x, y=None, stream=None):
    """qmv_q4_0_swiglu with float32 activations, rounded to fp16 inside the kernel."""
    W_gate, x, y, N, K, M = _prep(W_gate, x, y, Q4_0_BLOCK_BYTES, "qmv_q4_0_swiglu_f32", _torch().float32)
    _check_up(W_gate, W_up, "qmv_q4_0_swiglu_f32")
    with _on_device("qmv_q4_0_swiglu_f32", W_gate, W_up, x, y):
        qmv_q4_0_swiglu_f32_ptr(W_gate.data_ptr(), W_up.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M,
                                _stream_handle(stream))
    return y


def qmv_q8_0(W, x, y=None, stream=None):
    """y[M, N] = x[M, K] @ dequant(W)^T for Q8_0 weights."""
    W, x, y, N, K, M = _prep(W, x, y, Q8_0_BLOCK_BYTES, "qmv_q8_0")
    with _on_device("qmv_q8_0", W, x, y):
        qmv_q8_0_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def qmv_q4_0_q8_1(W, x, y=None, stream=None):
    """qmv_q4_0 with the activations quantised to Q8_1 in the kernel (integer dots)."""
    W, x, y, N, K, M = _prep(W, x, y, Q4_0_BLOCK_BYTES, "qmv_q4_0_q8_1")
    with _on_device("qmv_q4_0_q8_1", W, x, y):
        qmv_q4_0_q8_1_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def _prep_pre(W, q, d_bits, sumq, y, block_bytes, fn):
    """Checks shared by the calls on activations already in Q8_1 (sumq may be None)."""
    torch = _torch()
    tensors = [W, q, d_bits] + ([sumq] if sumq is not None else [])
    if not all(t.is_cuda for t in tensors):
        raise TypeError(f"{fn}: all tensors must be on a CUDA device (no CPU path)")
    if W.dtype != torch.uint8 or q.dtype != torch.int8 or d_bits.dtype != torch.int16 or \
            (sumq is not None and sumq.dtype != torch.int32):
        raise TypeError(f"{fn}: W uint8, q int8, d_bits int16" + (", sumq int32" if sumq is not None else ""))
    if q.dim() == 1:
        q = q.unsqueeze(0)
    M, K = q.shape
    if K % 32 or d_bits.numel() != M * (K // 32) or (sumq is not None and sumq.numel() != M * (K // 32)):
        raise ValueError(f"{fn}: q [M, K] with K % 32 == 0, d_bits" + (" and sumq" if sumq is not None else "")
                         + " [M, K/32]")
    if not all(t.is_contiguous() for t in tensors):
        raise ValueError(f"{fn}: tensors must be contiguous")
    row_bytes = (K // 32) * block_bytes
    if row_bytes and W.numel() % row_bytes:
        raise ValueError(f"{fn}: W size {W.numel()} is not a whole number of rows of {row_bytes} bytes")
    N = W.numel() // row_bytes if row_bytes else (W.shape[0] if W.dim() >= 1 else 0)
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=q.device)
    else:
        _check_y(y, M, N, fn)
    return q, y, N, K, M


def qmv_q4_0_q8_1_pre(W, q, d_bits, sumq, y=None, stream=None):
    """qmv_q4_0_q8_1 on activations already in Q8_1 (q int8 [M, K], d_bits int16
    [M, K/32], sumq int32 [M, K/32], as qmv_quantize_q8_1 returns them)."""
    q, y, N, K, M = _prep_pre(W, q, d_bits, sumq, y, Q4_0_BLOCK_BYTES, "qmv_q4_0_q8_1_pre")
    with _on_device("qmv_q4_0_q8_1_pre", W, q, d_bits, sumq, y):
        qmv_q4_0_q8_1_pre_ptr(W.data_ptr(), q.data_ptr(), d_bits.data_ptr(), sumq.data_ptr(), y.data_ptr(), N, K,
                              M, _stream_handle(stream))
    return y


def qmv_q8_0_q8_1(W, x, y=None, stream=None):
    """qmv_q8_0 with the activations quantised to Q8_1 in the kernel (signed integer dots)."""
    W, x, y, N, K, M = _prep(W, x, y, Q8_0_BLOCK_BYTES, "qmv_q8_0_q8_1")
    with _on_device("qmv_q8_0_q8_1", W, x, y):
        qmv_q8_0_q8_1_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def qmv_q8_0_q8_1_pre(W, q, d_bits, y=None, stream=None):
    """qmv_q8_0_q8_1 on activations already in Q8_1 (q int8 [M, K], d_bits int16
    [M, K/32]; the code sums qmv_quantize_q8_1 also returns are not needed)."""
    q, y, N, K, M = _prep_pre(W, q, d_bits, None, y, Q8_0_BLOCK_BYTES, "qmv_q8_0_q8_1_pre")
    with _on_device("qmv_q8_0_q8_1_pre", W, q, d_bits, y):
        qmv_q8_0_q8_1_pre_ptr(W.data_ptr(), q.data_ptr(), d_bits.data_ptr(), y.data_ptr(), N, K, M,
                              _stream_handle(stream))
    return y


def qmv_quantize_q8_1(x, stream=None):
    """Q8_1 blocks of fp16 activations [M, K] on the GPU: (q int8 [M, K],
    d_bits int16 [M, K/32] holding the fp16 scales' bits, sumq int32 [M, K/32])."""
    torch = _torch()
    if not x.is_cuda or x.dtype != torch.float16:
        raise TypeError("qmv_quantize_q8_1: x must be a float16 CUDA tensor (no CPU path)")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    x = x.contiguous()
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    d = torch.empty((M, K // 32), dtype=torch.int16, device=x.device)
    s = torch.empty((M, K // 32), dtype=torch.int32, device=x.device)
    with _on_device("qmv_quantize_q8_1", x):
        qmv_quantize_q8_1_ptr(x.data_ptr(), q.data_ptr(), d.data_ptr(), s.data_ptr(), M, K, _stream_handle(stream))
    return q, d, s


def qmv_q2w(W, x, y=None, stream=None):
    """y[M, N] = x[M, K] @ dequant(W)^T for plain 2-bit weights (10-byte blocks)."""
    W, x, y, N, K, M = _prep(W, x, y, Q2W_BLOCK_BYTES, "qmv_q2w")
    with _on_device("qmv_q2w", W, x, y):
        qmv_q2w_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def qmm_q4_0_prefill(W, x, y=None, stream=None):
    """Many-token (prefill) form of qmv_q4_0 on the tensor cores."""
    W, x, y, N, K, M = _prep(W, x, y, Q4_0_BLOCK_BYTES, "qmm_q4_0_prefill")
    with _on_device("qmm_q4_0_prefill", W, x, y):
        qmm_q4_0_prefill_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def qmm_q8_0_prefill(W, x, y=None, stream=None):
    """Many-token (prefill) form of qmv_q8_0 on the tensor cores."""
    W, x, y, N, K, M = _prep(W, x, y, Q8_0_BLOCK_BYTES, "qmm_q8_0_prefill")
    with _on_device("qmm_q8_0_prefill", W, x, y):
        qmm_q8_0_prefill_ptr(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, M, _stream_handle(stream))
    return y


def qmv_moe(W_pool, expert_idx, n_experts, x, N, y=None, stream=None):
    """Slot s: y[s] = x[s] @ dequant(expert expert_idx[s])^T, all slots in one launch."""
    torch = _torch()
    if not (W_pool.is_cuda and x.is_cuda and expert_idx.is_cuda):
        raise TypeError("qmv_moe: W_pool, expert_idx and x must be CUDA tensors (no CPU path)")
    if expert_idx.dtype != torch.int32 or not expert_idx.is_contiguous():
        raise TypeError("qmv_moe: expert_idx must be a contiguous int32 CUDA tensor")
    if W_pool.dtype != torch.uint8 or x.dtype != torch.float16:
        raise TypeError("qmv_moe: W_pool must be uint8, x float16")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if not (W_pool.is_contiguous() and x.is_contiguous()):
        raise ValueError("qmv_moe: W_pool and x must be contiguous")
    M, K = x.shape
    if expert_idx.numel() != M:
        raise ValueError("qmv_moe: one expert index per token")
    need = n_experts * N * (K // 32) * Q4_0_BLOCK_BYTES
    if W_pool.numel() < need:
        raise ValueError(f"qmv_moe: W_pool holds {W_pool.numel()} bytes, needs {need}")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    else:
        _check_y(y, M, N, "qmv_moe")
    with _on_device("qmv_moe", W_pool, expert_idx, x, y):
        qmv_moe_ptr(W_pool.data_ptr(), expert_idx.data_ptr(), int(n_experts), x.data_ptr(), y.data_ptr(),
                    int(N), int(K), int(M), _stream_handle(stream))
    return y


def qmv_read_probe(buf, out=None, stream=None):
    """Stream the bytes of the CUDA tensor ``buf`` (a multiple of 256 bytes) through
    the read-only bandwidth probe; returns the device uint32 checksum tensor ``out``
    (an int32 view: the XOR of the 16 bytes at every 256-byte offset, as 32-bit words)."""
    torch = _torch()
    if not (buf.is_cuda and buf.is_contiguous()):
        raise ValueError("qmv_read_probe: buf must be a contiguous CUDA tensor (no CPU path)")
    if out is None:
        out = torch.empty(1, dtype=torch.int32, device=buf.device)
    with _on_device("qmv_read_probe", buf, out):
        qmv_read_probe_ptr(buf.data_ptr(), buf.numel() * buf.element_size(), out.data_ptr(), _stream_handle(stream))
    return out


def qmv_device_status(stream=None) -> int:
    """Read and clear the device status word (synchronises the stream)."""
    out = ctypes.c_int32(0)
    _check("qmv_device_status", lib().qmv_device_status(_stream_handle(stream), ctypes.byref(out)))
    return int(out.value)


# -- the paged key/value cache ---------------------------------------------------------

class KvCache:
    """A paged key/value cache: k and v [n_pages, kv_heads, page, head_dim], fp16 or int8 (then with one fp32
    scale to a row, k_scale and v_scale [n_pages, kv_heads, page]).  The rows of a page are dense; pages may lie
    apart by any stride the two share (k and v interleaved in one buffer, for instance).  What the object says of its
    tensors is checked once, here: it cannot be given others (make another KvCache, which is cheap)."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "n_pages", "kv_heads", "page", "head_dim", "kind", "device", "index",
                 "page_stride")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        torch = _torch()
        if not (k.is_cuda and v.is_cuda):
            raise TypeError("KvCache: k and v must be CUDA tensors (no CPU path)")
        if k.dtype != v.dtype or k.dtype not in (torch.float16, torch.int8):
            raise TypeError("KvCache: k and v must both be float16 or int8")
        if k.dim() != 4 or k.shape != v.shape or k.device != v.device:
            raise ValueError("KvCache: k and v must be [n_pages, kv_heads, page, head_dim] on one device")
        n_pages, heads, page, dim = k.shape
        # (one head's stride means nothing: a pool [n_pages, page, 1, head_dim] transposed will do)
        dense = all(tuple(t.stride()[2:]) == (dim, 1) and (heads == 1 or t.stride(1) == page * dim) for t in (k, v))
        if not dense or (n_pages > 1 and k.stride(0) != v.stride(0)):
            raise ValueError("KvCache: the rows of a page must be dense, and k and v have one page stride")
        kind = QMV_KV_F16 if k.dtype == torch.float16 else QMV_KV_Q8
        for s in (k_scale, v_scale):
            if (kind == QMV_KV_Q8) != (s is not None):
                raise ValueError("KvCache: an int8 cache has k_scale and v_scale, a float16 cache has none")
            if s is not None and not (s.is_cuda and s.device == k.device and s.dtype == torch.float32
                                      and s.is_contiguous() and tuple(s.shape) == (n_pages, heads, page)):
                raise ValueError("KvCache: scales must be contiguous float32 [n_pages, kv_heads, page] beside k and v")
        values = (k, v, k_scale, v_scale, n_pages, heads, page, dim, kind, k.device, k.get_device(),
                  k.stride(0) if n_pages > 1 else heads * page * dim)
        for name, value in zip(self.__slots__, values):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError(f"KvCache: {name} cannot be set")

    def _ptrs(self):
        """Addresses of k, v and the scales, as they are now."""
        if self.kind == QMV_KV_F16:
            return self.k.data_ptr(), self.v.data_ptr(), 0, 0
        return self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr()


def qmv_kv_cache(n_pages, kv_heads, page, head_dim, dtype=None, device="cuda"):
    """A KvCache of zeros: dtype torch.float16 (default) or torch.int8 (8-bit codes with a scale to a row)."""
    torch = _torch()
    dtype = torch.float16 if dtype is None else dtype
    shape = (n_pages, kv_heads, page, head_dim)
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype != torch.int8:
        return KvCache(k, v)
    return KvCache(k, v, *(torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)))


class KvPages(NamedTuple):
    """The maps of one step (qmv_kv_pages): int32 CUDA tensors."""
    start: object      # [R + 1] offsets of the requests' new tokens
    kv_len: object     # [R] tokens in the cache, the new ones included
    slots: object      # [tokens] cache slot of each new token, -1 for padding
    pos: object        # [tokens] position (depth in the tree, with one)
    request: object    # [tokens] request, -1 for padding
    head: object       # [1] index in the free list after the last page taken


class KvPagesHeld(NamedTuple):
    """KvPages, and what each request holds after the step (qmv_kv_pages with `held`)."""
    start: object
    kv_len: object
    slots: object
    pos: object
    request: object
    head: object
    held: object       # [R] pages of each request, also past its length


# The paged-cache calls take a few microseconds on the GPU, so their checks look at each property of a tensor once
# (get_device: the index, or -1 for a CPU tensor).

def _on(fn, name, t, index):
    got = t.get_device()
    if got != index:
        if got < 0 or index < 0:
            raise TypeError(f"{fn}: {name} must be a CUDA tensor (no CPU path)")
        raise ValueError(f"{fn}: all tensors must be on one device (cuda:{index} and {name} on cuda:{got})")


def _int32(fn, name, t, dim, index):
    if t.get_device() == index and t.dtype is _int32_type and t.dim() == dim and t.is_contiguous() and index >= 0:
        return t.data_ptr()
    _on(fn, name, t, index)
    if index < 0:
        raise TypeError(f"{fn}: {name} must be a CUDA tensor (no CPU path)")
    raise TypeError(f"{fn}: {name} must be a contiguous int32 tensor with {dim} dimension" + ("s" if dim > 1 else ""))


def _tree_args(fn, tree, tokens, index):
    """(address, words) of a tree mask [tokens, words]."""
    ptr = _int32(fn, "tree", tree, 2, index)
    if tree.shape[0] != tokens or (tree.shape[1] == 0 and tokens > 0):
        raise ValueError(f"{fn}: tree must have a row of at least one word for each of the {tokens} tokens")
    return ptr, tree.shape[1]


def _call_on(fn, index, stream, args):
    """Calls library function `fn` with args and the stream's handle, device `index` current.  In the usual case (it
    is current already and its current stream is meant) no Python object is made for either."""
    torch = _torch()
    f = getattr(_lib or lib(), fn)
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            code = f(*args, _stream_handle(stream))
    else:
        code = f(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_handle(stream))
    if code != QMV_OK:
        raise QmvError(fn, code)


def _side_stream(index, stream):
    """The stream of a call as torch has it, where it is not device `index`'s current one; else None.  Memory for the
    call alone is then allocated under it: the allocator gives a freed block to the next tensor of the stream it was
    allocated under, in that stream's order, and any other stream's work could still be using it."""
    if stream is None:
        return None
    torch, handle = _torch(), _stream_handle(stream)
    if handle == torch._C._cuda_getCurrentRawStream(index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle, device=index) if handle else torch.cuda.default_stream(index)


def _output(shape, dtype, device, index, stream):
    """An output of a call on `stream`: memory that nothing before the call on that stream can still be using, and that
    is not given away, once freed, before the current stream's work up to then is done."""
    torch = _torch()
    side = _side_stream(index, stream)
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    reader = torch.cuda.current_stream(index)
    with torch.cuda.stream(side):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(reader)
    return out


def qmv_kv_pages(lens, n_new, free, table, page, tokens, head=None, tree=None, n_pages=None, stream=None, held=None):
    """Page and slot maps of one step, on the GPU.  lens, n_new [R]; free [n], ids of unused pages, taken in order
    from index `head` ([1], default 0) on; table [R, width] is completed in place; tokens: length of the per-token
    outputs (what the new tokens leave over is padding); tree [tokens, words]: positions are depths.  n_pages: size
    of the cache, to refuse wrong page ids (default: any that a slot can hold).  held [R]: pages that each request
    holds, where rejected tokens were taken off its length and their pages stay (default: what its length fills, so a
    program that cuts a length back returns the pages past it to the list).  Returns KvPages, with `held` KvPagesHeld."""
    torch = _torch()
    fn = "qmv_kv_pages"
    at = lens.get_device()
    len_ptr, new_ptr = _int32(fn, "lens", lens, 1, at), _int32(fn, "n_new", n_new, 1, at)
    free_ptr, table_ptr = _int32(fn, "free", free, 1, at), _int32(fn, "table", table, 2, at)
    R, tokens, page = lens.shape[0], int(tokens), int(page)
    if n_new.shape[0] != R or table.shape[0] != R:
        raise ValueError(f"{fn}: lens, n_new and table must have one row to a request")
    if tokens < 0 or page <= 0:
        raise ValueError(f"{fn}: tokens must not be negative, page must be positive")
    head_ptr = 0
    if head is not None:
        head_ptr = _int32(fn, "head", head, 1, at)
        if head.shape[0] != 1:
            raise ValueError(f"{fn}: head must be one number")
    tree_ptr, words = (0, 0) if tree is None else _tree_args(fn, tree, tokens, at)
    held_ptr = 0
    if held is not None:
        held_ptr = _int32(fn, "held", held, 1, at)
        if held.shape[0] != R:
            raise ValueError(f"{fn}: held must have one number to a request")
    size = 2 * R + 2 + 3 * tokens + (0 if held is None else R)
    out = torch.empty(size, dtype=torch.int32, device=lens.device) if stream is None else \
        _output(size, torch.int32, lens.device, at, stream)
    o, n = out.data_ptr(), 4 * tokens
    s = o + 4 * (2 * R + 1)
    if held is None:
        _call_on(fn, at, stream,
                 (len_ptr, new_ptr, free_ptr, free.shape[0], head_ptr, tree_ptr, words, table_ptr, o, o + 4 * (R + 1), s,
                  s + n, s + 2 * n, s + 3 * n, R, table.shape[1], page,
                  (0x7fffffff // page) if n_pages is None else int(n_pages), tokens))
        return KvPages(*out.split_with_sizes((R + 1, R, tokens, tokens, tokens, 1)))
    _call_on("qmv_kv_pages_held", at, stream,
             (len_ptr, new_ptr, free_ptr, free.shape[0], head_ptr, tree_ptr, words, table_ptr, held_ptr, o,
              o + 4 * (R + 1), s, s + n, s + 2 * n, s + 3 * n, s + 3 * n + 4, R, table.shape[1], page,
              (0x7fffffff // page) if n_pages is None else int(n_pages), tokens))
    return KvPagesHeld(*out.split_with_sizes((R + 1, R, tokens, tokens, tokens, 1, R)))


def qmv_kv_append(qkv, cache, slots, n_heads, pos=None, cos=None, sin=None, interleaved=False, q=None, stream=None):
    """Writes the key and value rows of qkv [T, (n_heads + 2 kv_heads) * D] (fp32 or fp16, rows any multiple of four
    values apart) to the cache at slots [T], rotated by rows pos [T] of the tables cos, sin [positions, rot / 2]
    (None: not rotated); returns the rotated queries, fp16 [T, n_heads, D]."""
    torch = _torch()
    fn = "qmv_kv_append"
    at = qkv.get_device()
    if at != cache.index or at < 0:
        _on(fn, "cache", cache.k, at)
        raise TypeError(f"{fn}: qkv must be a CUDA tensor (no CPU path)")
    f32 = qkv.dtype is torch.float32
    if not f32 and qkv.dtype is not torch.float16:
        raise TypeError(f"{fn}: qkv must be float32 or float16")
    hk, D = cache.kv_heads, cache.head_dim
    shape, apart = qkv.shape, qkv.stride()
    if len(shape) != 2 or shape[1] != (n_heads + 2 * hk) * D or (apart[1] != 1 and shape[0]):
        raise ValueError(f"{fn}: qkv must be [T, (n_heads + 2 * {hk}) * {D}] with dense rows")
    T, wide = shape
    slots_ptr = _int32(fn, "slots", slots, 1, at)
    if slots.shape[0] != T:
        raise ValueError(f"{fn}: one slot to a token")
    pos_ptr = cos_ptr = sin_ptr = n_pos = rot = 0
    if (cos is None) != (sin is None) or (cos is not None and pos is None):
        raise ValueError(f"{fn}: a rotation takes pos, cos and sin")
    if cos is not None:
        pos_ptr = _int32(fn, "pos", pos, 1, at)
        if pos.shape[0] != T:
            raise ValueError(f"{fn}: one position to a token")
        if not (cos.get_device() == sin.get_device() == at and cos.dtype is torch.float32 and sin.dtype is torch.float32
                and cos.dim() == 2 and cos.shape == sin.shape and cos.is_contiguous() and sin.is_contiguous()):
            raise ValueError(f"{fn}: cos and sin must be contiguous CUDA float32 [positions, rot / 2]")
        n_pos, rot = cos.shape
        rot *= 2
        cos_ptr, sin_ptr = cos.data_ptr(), sin.data_ptr()
    if q is None:
        q = torch.empty((T, n_heads, D), dtype=torch.float16, device=cache.device) if stream is None else \
            _output((T, n_heads, D), torch.float16, cache.device, at, stream)
    elif not (q.get_device() == at and q.dtype is torch.float16 and q.is_contiguous() and q.numel() == T * n_heads * D):
        raise ValueError(f"{fn}: q must be a contiguous CUDA float16 tensor of {T}x{n_heads}x{D}")
    k, v, ks, vs = cache._ptrs()
    _call_on(fn, at, stream,
             (qkv.data_ptr(), apart[0] if T > 1 else wide, f32, slots_ptr, pos_ptr, cos_ptr, sin_ptr, n_pos, rot,
              bool(interleaved), q.data_ptr(), k, v, ks, vs, cache.kind, T, int(n_heads), hk, D, cache.n_pages,
              cache.page, cache.page_stride))
    return q


def qmv_tree_attn_workspace(device=None):
    """The workspace of qmv_tree_attn: kept by a program from call to call, one for each stream that may run at the
    same time as another."""
    torch = _torch()
    device = torch.device("cuda" if device is None else device)
    with torch.cuda.device(device):
        n = lib().qmv_tree_attn_workspace()
        if n < 0:
            raise QmvError("qmv_tree_attn_workspace", 6)
        return torch.empty(n, dtype=torch.uint8, device=device)


def qmv_tree_attn(q, cache, table, start, kv_len, tree=None, scale=None, out=None, workspace=None, stream=None):
    """Attention of new tokens over the cache: q fp16 [T, heads, D] (rows any multiple of eight values apart), table
    [R, width], start [R + 1], kv_len [R] (new tokens included), tree [T, words] (None: a chain), scale (None:
    1 / sqrt(D)), workspace as qmv_tree_attn_workspace gives it (None: one is made for this call).
    Returns fp16 [T, heads, D]."""
    torch = _torch()
    fn = "qmv_tree_attn"
    at = q.get_device()
    if at != cache.index or at < 0:
        _on(fn, "cache", cache.k, at)
        raise TypeError(f"{fn}: q must be a CUDA tensor (no CPU path)")
    if q.dtype is not torch.float16:
        raise TypeError(f"{fn}: q must be float16")
    D = cache.head_dim
    shape, apart = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != D or ((apart[2] != 1 or (apart[1] != D and shape[1] > 1)) and q.numel()):
        raise ValueError(f"{fn}: q must be [T, heads, {D}] with dense rows")
    T, H, _ = shape
    table_ptr, start_ptr = _int32(fn, "table", table, 2, at), _int32(fn, "start", start, 1, at)
    R, width = table.shape
    len_ptr = _int32(fn, "kv_len", kv_len, 1, at)
    if start.shape[0] != R + 1 or kv_len.shape[0] != R:
        raise ValueError(f"{fn}: table [R, width], start [R + 1] and kv_len [R] must agree")
    tree_ptr, words = (0, 0) if tree is None else _tree_args(fn, tree, T, at)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None else \
            _output(shape, torch.float16, cache.device, at, stream)
    elif not (out.get_device() == at and out.dtype is torch.float16 and out.is_contiguous() and out.numel() == T * H * D):
        raise ValueError(f"{fn}: out must be a contiguous CUDA float16 tensor of {T}x{H}x{D}")
    if workspace is None:
        with torch.cuda.stream(_side_stream(at, stream)):     # (None: the current stream)
            workspace = qmv_tree_attn_workspace(cache.device)
    elif workspace.get_device() != at or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be a contiguous CUDA tensor")
    k, v, ks, vs = cache._ptrs()
    _call_on(fn, at, stream,
             (q.data_ptr(), apart[0] if T > 1 else H * D, k, v, ks, vs, cache.kind, cache.n_pages, cache.page,
              cache.page_stride, table_ptr, width, start_ptr, len_ptr, tree_ptr, words,
              None if scale is None else ctypes.byref(ctypes.c_float(scale)), out.data_ptr(), workspace.data_ptr(),
              workspace.nbytes, R, T, H, cache.kv_heads, D))
    return out
