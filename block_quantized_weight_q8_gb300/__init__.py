"""Python binding of libqmm (the C ABI declared in include/qmm.h).

Argument marshalling only: every function here has the name of the C entry
point it calls, converts tensors to device pointers and the current torch
stream to a cudaStream_t, and raises QmmError on a non-OK status.  All
arithmetic runs in the CUDA kernels of libqmm.so; there is no other path.
Tensors may be torch CUDA tensors or raw integer device addresses; the rotary,
paged-cache and mixture-of-experts calls take tensors only, read the sizes from them and raise
ValueError for one of another type, shape, layout or device.
"""
from __future__ import annotations

import ctypes
import os

from .buildlib import LIB, build  # noqa: F401

QMM_Q4_0, QMM_Q8_0, QMM_Q4_K, QMM_Q6_K, QMM_Q2_K, QMM_Q8_K, QMM_Q4_1, QMM_Q5_0, QMM_Q5_1, QMM_Q5_K = range(10)
TYPES = {"q4_0": QMM_Q4_0, "q8_0": QMM_Q8_0, "q4_K": QMM_Q4_K, "q6_K": QMM_Q6_K, "q2_K": QMM_Q2_K,
         "q8_K": QMM_Q8_K, "q4_1": QMM_Q4_1, "q5_0": QMM_Q5_0, "q5_1": QMM_Q5_1, "q5_K": QMM_Q5_K}
WEIGHT_TYPES = ("q4_0", "q8_0", "q4_K", "q6_K", "q2_K", "q4_1", "q5_0", "q5_1", "q5_K")

STATUS = {0: "QMM_OK", 1: "QMM_E_NULL", 2: "QMM_E_SHAPE", 3: "QMM_E_TYPE", 4: "QMM_E_ALIGN",
          5: "QMM_E_SCRATCH", 6: "QMM_E_CUDA", 7: "QMM_E_TIMEOUT", 8: "QMM_E_BOUNDS"}

# every entry point the header declares, with its argument kinds
# p: pointer, i: int64, s: size_t, t: int (type code), c: int, f: float, d: double, q: stream
SIGNATURES = {
    "qmm_block_bytes": ("t", ctypes.c_size_t),
    "qmm_block_values": ("t", ctypes.c_int),
    "qmm_row_bytes": ("ti", ctypes.c_size_t),
    "qmm_act_type": ("t", ctypes.c_int),
    "qmm_status_str": ("c", ctypes.c_char_p),
    "qmm_quantize_q8_0": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q8_K": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q4_0": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q4_K": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q6_K": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q2_K": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q4_1": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q5_0": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q5_1": ("ppiiq", ctypes.c_int),
    "qmm_quantize_q5_K": ("ppiiq", ctypes.c_int),
    "qmm_matvec_q4_0": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q8_0": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q4_K": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q6_K": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q2_K": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q4_1": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q5_0": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q5_1": ("pppiiq", ctypes.c_int),
    "qmm_matvec_q5_K": ("pppiiq", ctypes.c_int),
    "qmm_linear_q4_0": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q8_0": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q4_K": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q6_K": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q2_K": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q4_1": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q5_0": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q5_1": ("pppspiiiq", ctypes.c_int),
    "qmm_linear_q5_K": ("pppspiiiq", ctypes.c_int),
    "qmm_matmul_q4_0": ("pppiiiq", ctypes.c_int),
    "qmm_matmul_q8_0": ("pppiiiq", ctypes.c_int),
    "qmm_matmul_q4_1": ("pppiiiq", ctypes.c_int),
    "qmm_matmul_q5_0": ("pppiiiq", ctypes.c_int),
    "qmm_matmul_q5_1": ("pppiiiq", ctypes.c_int),
    "qmm_get_rows": ("tpppiiiq", ctypes.c_int),
    "qmm_linear_host": ("tppppsppiiiq", ctypes.c_int),
    "qmm_rmsnorm_quantize": ("tppfpiiq", ctypes.c_int),
    "qmm_linear_norm": ("ttppppfpspiiq", ctypes.c_int),
    "qmm_kv_row_bytes": ("i", ctypes.c_size_t),
    "qmm_kv_quantize": ("ppiiq", ctypes.c_int),
    "qmm_kv_scores": ("pppiiiifq", ctypes.c_int),
    "qmm_kv_wsum_scratch_bytes": ("iii", ctypes.c_size_t),
    "qmm_kv_wsum": ("pppps" + "iiiiq", ctypes.c_int),
    "qmm_rope_freqs": ("pidtddddq", ctypes.c_int),
    "qmm_rope": ("ppipipiiicq", ctypes.c_int),
    "qmm_kv_page_bytes": ("tiii", ctypes.c_size_t),
    "qmm_kv_store": ("ppipippippipiiq", ctypes.c_int),
    "qmm_kv_load": ("pppipipiq", ctypes.c_int),
    "qmm_kv_attend_scratch_bytes": ("iii", ctypes.c_size_t),
    "qmm_kv_attend": ("ppipppippsiifiq", ctypes.c_int),
    "qmm_add_rmsnorm_quantize": ("tppppfppiiq", ctypes.c_int),
    "qmm_route": ("ppipppiiq", ctypes.c_int),
    "qmm_experts_scratch_bytes": ("tiiiii", ctypes.c_size_t),
    "qmm_experts_glu": ("ttppppppsiiiiiq", ctypes.c_int),
    "qmm_experts_sum": ("tppppppps" + "iiiiiq", ctypes.c_int),
    "qmm_experts_path": ("ttiiiii", ctypes.c_int),
    "qmm_matmul_q4_K": ("pppiiiq", ctypes.c_int),
    "qmm_matmul_q6_K": ("pppiiiq", ctypes.c_int),
    "qmm_matmul_q5_K": ("pppiiiq", ctypes.c_int),
    "qmm_matmul_q2_K": ("pppiiiq", ctypes.c_int),
    "qmm_linear_noalloc": ("tpppiiiq", ctypes.c_int),
    "qmm_linear_group": ("ttppppspiiq", ctypes.c_int),
    "qmm_blocksums": ("tpppiiiq", ctypes.c_int),
    "qmm_test_wait_timeout": ("uq", ctypes.c_int),
    "qmm_device_status": ("c", ctypes.c_int),
}
_CT = {"p": ctypes.c_void_p, "i": ctypes.c_int64, "s": ctypes.c_size_t, "t": ctypes.c_int, "c": ctypes.c_int,
       "q": ctypes.c_void_p, "f": ctypes.c_float, "d": ctypes.c_double, "u": ctypes.c_uint64}

_lib = None


class QmmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (fn, STATUS.get(status, status), _status_str(status)))


def load(path: str = None):
    """Load libqmm.so (built in-tree by build()); raises if it is missing.  The environment
    variable QMM_LIBRARY names another build of the same library to load instead (the
    bounds-checked variant, block_quantized_weight_q8_gb300.buildlib.CHECKED_LIB)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("QMM_LIBRARY") or LIB
    if not os.path.exists(path):
        raise ImportError("libqmm.so is not built (%s): run block_quantized_weight_q8_gb300.build()" % path)
    L = ctypes.CDLL(path)
    for name, (kinds, res) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.argtypes = [_CT[k] for k in kinds]
        fn.restype = res
    _lib = L
    return L


def _status_str(status: int) -> str:
    try:
        return load().qmm_status_str(int(status)).decode()
    except Exception:
        return "?"


def ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


def stream_handle(stream=None) -> int:
    if stream is None:
        dev = _device()
        return _raw_stream(dev)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _call(name, *args):
    r = getattr(_lib or load(), name)(*args)
    if r != 0:
        raise QmmError(name, r)


def _type(t) -> int:
    return TYPES[t] if isinstance(t, str) else int(t)


# ---- formats
def qmm_block_bytes(t) -> int:
    return int(load().qmm_block_bytes(_type(t)))


def qmm_block_values(t) -> int:
    return int(load().qmm_block_values(_type(t)))


def qmm_row_bytes(t, K: int) -> int:
    return int(load().qmm_row_bytes(_type(t), int(K)))


def qmm_act_type(wtype) -> int:
    return int(load().qmm_act_type(_type(wtype)))


# ---- quantizers
def qmm_quantize_q8_0(x, xq, M, K, stream=None):
    _call("qmm_quantize_q8_0", ptr(x), ptr(xq), int(M), int(K), stream_handle(stream))


def qmm_quantize_q8_K(x, xq, M, K, stream=None):
    _call("qmm_quantize_q8_K", ptr(x), ptr(xq), int(M), int(K), stream_handle(stream))


def qmm_quantize_q4_0(w, wq, N, K, stream=None):
    _call("qmm_quantize_q4_0", ptr(w), ptr(wq), int(N), int(K), stream_handle(stream))


def qmm_quantize_q4_K(w, wq, N, K, stream=None):
    _call("qmm_quantize_q4_K", ptr(w), ptr(wq), int(N), int(K), stream_handle(stream))


def qmm_quantize_q6_K(w, wq, N, K, stream=None):
    _call("qmm_quantize_q6_K", ptr(w), ptr(wq), int(N), int(K), stream_handle(stream))


def qmm_quantize_q2_K(w, wq, N, K, stream=None):
    _call("qmm_quantize_q2_K", ptr(w), ptr(wq), int(N), int(K), stream_handle(stream))


def quantize(t, x, out, rows, K, stream=None):
    """qmm_quantize_<t> by type name (q8_0 also quantizes Q8_0 weights)."""
    _call("qmm_quantize_" + t, ptr(x), ptr(out), int(rows), int(K), stream_handle(stream))


# ---- matvec / linear / matmul
def _mv(name):
    def f(W, xq, y, N, K, stream=None):
        _call(name, ptr(W), ptr(xq), ptr(y), int(N), int(K), stream_handle(stream))
    f.__name__ = name
    return f


qmm_matvec_q4_0 = _mv("qmm_matvec_q4_0")
qmm_matvec_q8_0 = _mv("qmm_matvec_q8_0")
qmm_matvec_q4_K = _mv("qmm_matvec_q4_K")
qmm_matvec_q6_K = _mv("qmm_matvec_q6_K")
qmm_matvec_q2_K = _mv("qmm_matvec_q2_K")
qmm_matvec_q4_1 = _mv("qmm_matvec_q4_1")
qmm_matvec_q5_0 = _mv("qmm_matvec_q5_0")
qmm_matvec_q5_1 = _mv("qmm_matvec_q5_1")
qmm_matvec_q5_K = _mv("qmm_matvec_q5_K")


def matvec(wtype, W, xq, y, N, K, stream=None):
    _call("qmm_matvec_" + wtype, ptr(W), ptr(xq), ptr(y), int(N), int(K), stream_handle(stream))


def _lin(name):
    def f(W, x, scratch, scratch_bytes, y, M, N, K, stream=None):
        _call(name, ptr(W), ptr(x), ptr(scratch), int(scratch_bytes), ptr(y), int(M), int(N), int(K),
              stream_handle(stream))
    f.__name__ = name
    return f


qmm_linear_q4_0 = _lin("qmm_linear_q4_0")
qmm_linear_q8_0 = _lin("qmm_linear_q8_0")
qmm_linear_q4_K = _lin("qmm_linear_q4_K")
qmm_linear_q6_K = _lin("qmm_linear_q6_K")
qmm_linear_q2_K = _lin("qmm_linear_q2_K")
qmm_linear_q4_1 = _lin("qmm_linear_q4_1")
qmm_linear_q5_0 = _lin("qmm_linear_q5_0")
qmm_linear_q5_1 = _lin("qmm_linear_q5_1")
qmm_linear_q5_K = _lin("qmm_linear_q5_K")


def linear(wtype, W, x, scratch, scratch_bytes, y, M, N, K, stream=None):
    _call("qmm_linear_" + wtype, ptr(W), ptr(x), ptr(scratch), int(scratch_bytes), ptr(y), int(M), int(N), int(K),
          stream_handle(stream))


def qmm_linear_host(wtype, W, x_host, x_dev, scratch, scratch_bytes, y_dev, y_host, M, N, K, stream=None):
    """qmm_linear_<wtype> with host buffers: x_host (pinned) -> x_dev, the multiply, y_dev -> y_host, queued on
    the stream (synchronize it before reading y_host)."""
    _call("qmm_linear_host", _type(wtype), ptr(W), ptr(x_host), ptr(x_dev), ptr(scratch), int(scratch_bytes), ptr(y_dev),
          ptr(y_host), int(M), int(N), int(K), stream_handle(stream))


def qmm_linear_noalloc(wtype, W, x, y, M, N, K, stream=None):
    """qmm_linear_<wtype> without a workspace argument: the library's own 1 MiB device array holds the
    quantized rows (see include/qmm.h for the limit and the sharing rules)."""
    _call("qmm_linear_noalloc", _type(wtype), ptr(W), ptr(x), ptr(y), int(M), int(N), int(K), stream_handle(stream))


def qmm_linear_group(wtype, Ws, Ns, x, scratch, scratch_bytes, ys, M, K, stream=None):
    """qmm_linear_<wtype> for several matrices Ws (rows Ns) on the same rows x, outputs ys, one launch
    per token (see include/qmm.h)."""
    G = len(Ws)
    if not (len(Ns) == G and len(ys) == G):
        raise ValueError("Ws, Ns and ys must have the same length")
    w_arr = (ctypes.c_void_p * max(G, 1))(*[ptr(w) for w in Ws])
    n_arr = (ctypes.c_int64 * max(G, 1))(*[int(n) for n in Ns])
    y_arr = (ctypes.c_void_p * max(G, 1))(*[ptr(y) for y in ys])
    _call("qmm_linear_group", _type(wtype), G, ctypes.cast(w_arr, ctypes.c_void_p), ctypes.cast(n_arr, ctypes.c_void_p),
          ptr(x), ptr(scratch), int(scratch_bytes), ctypes.cast(y_arr, ctypes.c_void_p), int(M), int(K),
          stream_handle(stream))


def qmm_rmsnorm_quantize(act, x, w, eps, xq, M, K, stream=None):
    """Quantize the RMSNormed rows (x * s) * w to act ("q8_0" or "q8_K")."""
    _call("qmm_rmsnorm_quantize", _type(act), ptr(x), ptr(w), float(eps), ptr(xq), int(M), int(K), stream_handle(stream))


def qmm_linear_norm(wtype, Ws, Ns, x, w, eps, scratch, scratch_bytes, ys, M, K, stream=None):
    """qmm_linear_group on the RMSNormed rows of x (norm weight w, eps)."""
    G = len(Ws)
    if not (len(Ns) == G and len(ys) == G):
        raise ValueError("Ws, Ns and ys must have the same length")
    w_arr = (ctypes.c_void_p * max(G, 1))(*[ptr(m) for m in Ws])
    n_arr = (ctypes.c_int64 * max(G, 1))(*[int(n) for n in Ns])
    y_arr = (ctypes.c_void_p * max(G, 1))(*[ptr(y) for y in ys])
    _call("qmm_linear_norm", _type(wtype), G, ctypes.cast(w_arr, ctypes.c_void_p), ctypes.cast(n_arr, ctypes.c_void_p),
          ptr(x), ptr(w), float(eps), ptr(scratch), int(scratch_bytes), ctypes.cast(y_arr, ctypes.c_void_p), int(M),
          int(K), stream_handle(stream))


def qmm_matmul_q4_0(W, xq, Y, M, N, K, stream=None):
    _call("qmm_matmul_q4_0", ptr(W), ptr(xq), ptr(Y), int(M), int(N), int(K), stream_handle(stream))


def matmul(wtype, W, xq, Y, M, N, K, stream=None):
    """qmm_matmul_<wtype>: Y[M][N] for M quantized activation rows (Q8_0 for the 32-value formats, Q8_K for
    the K-quants)."""
    _call("qmm_matmul_" + wtype, ptr(W), ptr(xq), ptr(Y), int(M), int(N), int(K), stream_handle(stream))


def qmm_get_rows(wtype, W, ids, out, R, N, K, stream=None):
    """out[r] = dequantized row ids[r] of W (ids: int32 device tensor)."""
    _call("qmm_get_rows", _type(wtype), ptr(W), ptr(ids), ptr(out), int(R), int(N), int(K), stream_handle(stream))


# ---- the Q8 KV cache
def qmm_kv_row_bytes(hd):
    return int(load().qmm_kv_row_bytes(int(hd)))


def qmm_kv_quantize(x, out, rows, hd, stream=None):
    """rows head vectors (f32 [rows][hd]) into quantized rows (f32 d + int8 codes) at out."""
    _call("qmm_kv_quantize", ptr(x), ptr(out), int(rows), int(hd), stream_handle(stream))


def qmm_kv_scores(q, kc, scores, Hq, Hkv, P, hd, scale, stream=None):
    """scores[h][p] for the quantized query rows q against positions 0..P-1 of the K cache kc."""
    _call("qmm_kv_scores", ptr(q), ptr(kc), ptr(scores), int(Hq), int(Hkv), int(P), int(hd), float(scale),
          stream_handle(stream))


def qmm_kv_wsum_scratch_bytes(Hq, P, hd):
    return int(load().qmm_kv_wsum_scratch_bytes(int(Hq), int(P), int(hd)))


def qmm_kv_wsum(w, vc, out, scratch, scratch_bytes, Hq, Hkv, P, hd, stream=None):
    """out[h] = sum_p w[h][p] * (dequantized V row of position p, KV head h / (Hq/Hkv))."""
    _call("qmm_kv_wsum", ptr(w), ptr(vc), ptr(out), ptr(scratch), int(scratch_bytes), int(Hq), int(Hkv), int(P),
          int(hd), stream_handle(stream))


# ---- rotary positions and the paged KV cache
QMM_KV_Q8, QMM_KV_F16 = 0, 1
KV_TYPES = {"q8": QMM_KV_Q8, "f16": QMM_KV_F16}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "bands": 2, "yarn": 3}


_torch = _raw_stream = None


def _device() -> int:
    """The current device; imports torch on first use."""
    global _torch, _raw_stream
    if _torch is None:
        import torch
        torch.cuda.current_device()  # initializes CUDA
        # the stream's handle without a Stream object around it, where torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: int(torch.cuda.current_stream(dev).cuda_stream))
        _torch = torch
    return _torch.cuda.current_device()


def _refuse(name, t, dtype, shape, dev):
    raise ValueError("%s: %s of shape %s on the current device (cuda:%d), contiguous or with contiguous heads, is needed, "
                     "got %s of shape %s (strides %s) on %s" % (name, dtype, shape, dev, t.dtype, tuple(t.shape),
                                                                t.stride(), t.device))


def _heads(name, t, dev, T, H, hd):
    """(address, token stride) of f32 head rows [T][H][hd]: heads side by side, tokens any stride apart."""
    if t.dtype is not _torch.float32 or t.get_device() != dev or t.shape != (T, H, hd):
        _refuse(name, t, "float32", (T, H, hd), dev)
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != hd and H > 1):
        _refuse(name, t, "float32", (T, H, hd), dev)
    return t.data_ptr(), (s0 if T > 1 else H * hd)


def _plain(name, t, dev, dtype, dims):
    """The address of a contiguous tensor of this type and number of dimensions."""
    if t.dtype is not getattr(_torch, dtype) or t.get_device() != dev or not t.is_contiguous() or t.dim() != dims:
        _refuse(name, t, dtype, "of %d dimensions" % dims, dev)
    return t.data_ptr()


def _ints(name, t, dev, n):
    if t is None:
        return None
    if t.dtype is not _torch.int32 or t.get_device() != dev or t.shape != (n,) or not t.is_contiguous():
        _refuse(name, t, "int32", (n,), dev)
    return t.data_ptr()


def _ref(name, x, dev):
    if x.device != dev:
        raise ValueError("%s: on cuda:%d, the current device is cuda:%d" % (name, x.device, dev))
    return x.ref


class RopeSpec(ctypes.Structure):
    """qmm_rope_spec: a frequency table (int64 CUDA tensor [n_rot / 2], filled by qmm_rope_freqs), how values are
    paired ("half" or "interleaved") and the factor of the result.  Keeps the table alive."""
    _fields_ = [("freqs", ctypes.c_void_p), ("n_rot", ctypes.c_int64), ("layout", ctypes.c_int32),
                ("mscale", ctypes.c_float)]

    def __init__(self, freqs, layout="half", mscale=1.0):
        super().__init__(_plain("freqs", freqs, _device(), "int64", 1), 2 * freqs.shape[0], ROPE_LAYOUTS[layout], mscale)
        self.tensor, self.ref, self.device = freqs, ctypes.addressof(self), freqs.get_device()


class KvPages(ctypes.Structure):
    """qmm_kv_pages: pools k and v (uint8 CUDA tensors [num_pages][at least qmm_kv_page_bytes], pages a multiple of
    16 bytes apart), a page table (int32 CUDA tensor [num_seqs][max_pages]) and the shape.  Keeps the tensors alive."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("num_seqs", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("Hkv", ctypes.c_int64), ("hd", ctypes.c_int64),
                ("type", ctypes.c_int32), ("page_size", ctypes.c_int32)]

    def __init__(self, type, k, v, table, page_size, Hkv, hd):
        dev = _device()
        for name, t in (("k", k), ("v", v)):
            if t.dtype is not _torch.uint8 or t.get_device() != dev or t.dim() != 2:
                _refuse(name, t, "uint8", ("pages", "bytes"), dev)
        rows = _plain("table", table, dev, "int32", 2)
        need = qmm_kv_page_bytes(type, Hkv, page_size, hd)
        if need == 0:
            raise ValueError("no cache of type %r has %r heads of %r in pages of %r" % (type, Hkv, hd, page_size))
        if k.shape != v.shape or k.stride() != v.stride() or k.stride(1) != 1 or k.shape[1] < need:
            raise ValueError("k and v: pools of one shape and stride are needed, %d bytes a page at least" % need)
        stride = k.stride(0) if k.shape[0] > 1 else -(-k.shape[1] // 16) * 16
        super().__init__(k.data_ptr(), v.data_ptr(), rows, k.shape[0], stride, table.shape[0],
                         table.shape[1], Hkv, hd, KV_TYPES[type], page_size)
        self.tensors, self.ref, self.device = (k, v, table), ctypes.addressof(self), dev


def qmm_rope_freqs(freqs, base=10000.0, scaling="plain", factor=1.0, orig_len=0.0, lo=0.0, hi=0.0, stream=None):
    """Fills the frequency table freqs (int64 CUDA tensor [n_rot / 2])."""
    at = _plain("freqs", freqs, _device(), "int64", 1)
    _call("qmm_rope_freqs", at, 2 * freqs.shape[0], float(base), ROPE_SCALINGS[scaling], float(factor), float(orig_len),
          float(lo), float(hi), stream_handle(stream))


def qmm_rope(rope, x, y, pos, inverse=False, stream=None):
    """y = x ([T][H][hd] f32) rotated to the positions pos; y may be x."""
    dev = _device()
    if x.dim() != 3:
        _refuse("x", x, "float32", ("T", "H", "hd"), dev)
    T, H, hd = x.shape
    px, ldx = _heads("x", x, dev, T, H, hd)
    py, ldy = _heads("y", y, dev, T, H, hd)
    _call("qmm_rope", _ref("rope", rope, dev), px, ldx, py, ldy, _ints("pos", pos, dev, T), T, H, hd, 1 if inverse else 0,
          _raw_stream(dev) if stream is None else stream_handle(stream))


def qmm_kv_page_bytes(type, Hkv, page_size, hd):
    return int(load().qmm_kv_page_bytes(KV_TYPES[type], int(Hkv), int(page_size), int(hd)))


def qmm_kv_store(pages, k, v, pos, seq=None, rope=None, q=None, q_out=None, stream=None):
    """Stores keys k and values v ([T][Hkv][hd] f32) at positions pos of the sequences seq; with rope, keys are rotated
    first, and queries q ([T][Hq][hd]) into q_out."""
    dev, Hkv, hd = _device(), pages.Hkv, pages.hd
    if k.dim() != 3:
        _refuse("k", k, "float32", ("T", Hkv, hd), dev)
    T = k.shape[0]
    pk, ldk = _heads("k", k, dev, T, Hkv, hd)
    pv, ldv = _heads("v", v, dev, T, Hkv, hd)
    pq = ldq = po = ldo = Hq = 0
    if q is not None:
        if q_out is None or rope is None:
            raise ValueError("queries need q_out and rope")
        if q.dim() != 3:
            _refuse("q", q, "float32", (T, "Hq", hd), dev)
        Hq = q.shape[1]
        pq, ldq = _heads("q", q, dev, T, Hq, hd)
        po, ldo = _heads("q_out", q_out, dev, T, Hq, hd)
    _call("qmm_kv_store", _ref("pages", pages, dev), pk, ldk, pv, ldv, _ints("pos", pos, dev, T), _ints("seq", seq, dev, T), T,
          _ref("rope", rope, dev) if rope is not None else None, pq, ldq, po, ldo, Hq,
          _raw_stream(dev) if stream is None else stream_handle(stream))


def qmm_kv_load(pages, pos, k_out=None, v_out=None, seq=None, stream=None):
    """The rows at positions pos of the sequences seq as f32 ([T][Hkv][hd]); either output may be None."""
    dev, Hkv, hd = _device(), pages.Hkv, pages.hd
    if pos.dim() != 1:
        _refuse("pos", pos, "int32", ("T",), dev)
    T = pos.shape[0]
    pk, ldk = _heads("k_out", k_out, dev, T, Hkv, hd) if k_out is not None else (None, 0)
    pv, ldv = _heads("v_out", v_out, dev, T, Hkv, hd) if v_out is not None else (None, 0)
    _call("qmm_kv_load", _ref("pages", pages, dev), _ints("pos", pos, dev, T), _ints("seq", seq, dev, T), T, pk, ldk, pv, ldv,
          _raw_stream(dev) if stream is None else stream_handle(stream))


def qmm_kv_attend_scratch_bytes(Hq, Hkv, hd):
    return int(load().qmm_kv_attend_scratch_bytes(int(Hq), int(Hkv), int(hd)))


def qmm_kv_attend(pages, q, lens, out, scratch, scratch_bytes, scale, lse=None, seq=None, window=0, stream=None):
    """out[r] = the attention of query heads q[r] ([R][Hq][hd] f32) over the first lens[r] positions (the last window
    of them) of their sequences; lse ([R][Hq] f32) the log of the softmax's sum."""
    dev, hd = _device(), pages.hd
    if q.dim() != 3:
        _refuse("q", q, "float32", ("R", "Hq", hd), dev)
    R, Hq, _ = q.shape
    pq, ldq = _heads("q", q, dev, R, Hq, hd)
    po, ldo = _heads("out", out, dev, R, Hq, hd)
    pl = None
    if lse is not None:
        if (lse.dtype is not _torch.float32 or lse.get_device() != dev or lse.shape != (R, Hq)
                or not lse.is_contiguous()):
            _refuse("lse", lse, "float32", (R, Hq), dev)
        pl = lse.data_ptr()
    if scratch.get_device() != dev or scratch.nbytes < scratch_bytes or not scratch.is_contiguous():
        _refuse("scratch", scratch, "memory", "of %d bytes" % scratch_bytes, dev)
    _call("qmm_kv_attend", _ref("pages", pages, dev), pq, ldq, _ints("lens", lens, dev, R), _ints("seq", seq, dev, R), po, ldo,
          pl, scratch.data_ptr(), scratch_bytes, R, Hq, scale, window,
          _raw_stream(dev) if stream is None else stream_handle(stream))


# ---- mixture of experts
ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
GLU_KINDS = {"silu": 0, "gelu": 1}


def _unknown(what, names, name):
    raise ValueError("%s: one of %s is needed, got %r" % (what, ", ".join(sorted(names)), name))


class RouteSpec(ctypes.Structure):
    """qmm_route_spec: how tokens choose their experts."""
    _fields_ = [("score", ctypes.c_int32), ("k", ctypes.c_int32), ("groups", ctypes.c_int32), ("groups_kept", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


_formats = {}


def _format(t):
    """(code, bytes of a block, its values, activation type's code) of a type."""
    f = _formats.get(t)
    if f is None:
        if isinstance(t, str) and t not in TYPES:
            _unknown("type", TYPES, t)
        c = _type(t)
        f = _formats[t] = (c, qmm_block_bytes(c), qmm_block_values(c), qmm_act_type(c))
    return f


def _row(t, K):
    """qmm_row_bytes without the call; 0 where K is no whole number of blocks."""
    _, size, values, _ = _format(t)
    return K // values * size if values and K % values == 0 else 0


def _whole(name, t, dev, dtype, shape):
    """The address of a contiguous tensor of this type and shape (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, dtype, shape, dev)
    return t.data_ptr()


def _workspace(t, size, dev):
    if t.get_device() != dev or t.nbytes < size or not t.is_contiguous():
        _refuse("scratch", t, "memory", "of %d bytes" % size, dev)
    return t.data_ptr()


def qmm_add_rmsnorm_quantize(act, x, r, w, eps, xq=None, sum=None, h=None, stream=None):
    """sum = x + r, h = its RMSNorm with the weight w, xq = h quantized to act ("q8_0" or "q8_K"); x and r f32 [M][K], xq
    uint8 [M][qmm_row_bytes(act, K)]; sum (may be x or r) and one of h and xq may be None."""
    at = _format(act)[0]
    dev = _device()
    if x.dim() != 2:
        _refuse("x", x, "float32", ("M", "K"), dev)
    rows = M, K = x.shape
    _call("qmm_add_rmsnorm_quantize", at, _whole("x", x, dev, _torch.float32, rows), _whole("r", r, dev, _torch.float32, rows),
          _whole("sum", sum, dev, _torch.float32, rows), _whole("w", w, dev, _torch.float32, (K,)), eps,
          _whole("h", h, dev, _torch.float32, rows), _whole("xq", xq, dev, _torch.uint8, (M, _row(act, K))), M, K,
          _raw_stream(dev) if stream is None else stream_handle(stream))


def qmm_route(logits, ids, weights, score="softmax", bias=None, groups=1, groups_kept=1, group_top=1, renorm=True, scale=1.0,
              stream=None):
    """ids and weights ([T][k], int32 and f32): the experts that each token's logits ([T][E] f32, rows any stride apart)
    choose, and what they weigh (see include/qmm.h)."""
    if not isinstance(score, str) or score not in ROUTE_SCORES:
        _unknown("score", ROUTE_SCORES, score)
    if (groups | groups_kept | group_top) >> 31 > 0:  # the spec's fields have 32 bits (negative ones are the library's to refuse)
        raise ValueError("groups, groups_kept, group_top: got %r, %r, %r" % (groups, groups_kept, group_top))
    dev = _device()
    if logits.dtype is not _torch.float32 or logits.get_device() != dev or logits.dim() != 2 or (
            logits.stride(1) != 1 and logits.shape[1] > 1):
        _refuse("logits", logits, "float32", ("T", "E"), dev)
    T, E = logits.shape
    if ids.dim() != 2:
        _refuse("ids", ids, "int32", (T, "k"), dev)
    k = ids.shape[1]
    spec = RouteSpec(ROUTE_SCORES[score], k, groups, groups_kept, group_top, 1 if renorm else 0, scale)
    _call("qmm_route", ctypes.addressof(spec), logits.data_ptr(), logits.stride(0) if T > 1 else E,
          _whole("bias", bias, dev, _torch.float32, (E,)), _whole("ids", ids, dev, _torch.int32, (T, k)),
          _whole("weights", weights, dev, _torch.float32, (T, k)), T, E,
          _raw_stream(dev) if stream is None else stream_handle(stream))


def qmm_experts_scratch_bytes(wtype, T, k, E, N, K):
    return int(load().qmm_experts_scratch_bytes(_format(wtype)[0], int(T), int(k), int(E), int(N), int(K)))


def qmm_experts_path(wtype, gated, T, k, E, N, K):
    """0 where qmm_experts_glu (gated) or qmm_experts_sum streams each choice's weight rows at this shape, 1 where it goes by
    the tensor cores."""
    path = int(load().qmm_experts_path(_format(wtype)[0], 1 if gated else 0, int(T), int(k), int(E), int(N), int(K)))
    if path < 0:
        raise ValueError("no experts' products of type %r and shape %s" % (wtype, (T, k, E, N, K)))
    return path


def qmm_experts_glu(wtype, Wg, Wu, xq, ids, h, scratch, scratch_bytes, gate="silu", stream=None):
    """h[t][j] = gate(Wg[e] x_t) * (Wu[e] x_t), e = ids[t][j]: h f32 [T][k][N], Wg and Wu uint8 [E][N][row bytes], xq uint8
    [T][qmm_row_bytes(qmm_act_type(wtype), K)], ids int32 [T][k] (negative: no expert, zeros).  h overlaps no input."""
    if not isinstance(gate, str) or gate not in GLU_KINDS:
        _unknown("gate", GLU_KINDS, gate)
    wt, size, values, act = _format(wtype)
    dev = _device()
    if h.dim() != 3 or Wg.dim() != 3:
        _refuse("h, Wg", h if h.dim() != 3 else Wg, "float32, uint8", "of 3 dimensions", dev)
    T, k, N = h.shape
    matrix = E, _, row = Wg.shape
    if size == 0 or row == 0 or row % size:
        raise ValueError("Wg: rows of %d bytes are no whole blocks of type %r" % (row, wtype))
    K = row // size * values
    _call("qmm_experts_glu", wt, GLU_KINDS[gate], _whole("Wg", Wg, dev, _torch.uint8, (E, N, row)),
          _whole("Wu", Wu, dev, _torch.uint8, matrix), _whole("xq", xq, dev, _torch.uint8, (T, _row(act, K))),
          _whole("ids", ids, dev, _torch.int32, (T, k)), _whole("h", h, dev, _torch.float32, (T, k, N)),
          _workspace(scratch, scratch_bytes, dev), scratch_bytes, T, k, E, N, K,
          _raw_stream(dev) if stream is None else stream_handle(stream))


def qmm_experts_sum(wtype, W, h, ids, weights, y, scratch, scratch_bytes, residual=None, stream=None):
    """y[t] = residual[t] + sum_j weights[t][j] (W[ids[t][j]] q(h[t][j])): y f32 [T][N], W uint8 [E][N][row bytes], h f32
    [T][k][K] (quantized on the way), ids int32 and weights f32 (or None: 1) [T][k]; residual f32 [T][N], may be y, which
    overlaps no other input."""
    wt = _format(wtype)[0]
    dev = _device()
    if h.dim() != 3 or W.dim() != 3:
        _refuse("h, W", h if h.dim() != 3 else W, "float32, uint8", "of 3 dimensions", dev)
    T, k, K = h.shape
    E, N = W.shape[:2]
    _call("qmm_experts_sum", wt, _whole("W", W, dev, _torch.uint8, (E, N, _row(wt, K))),
          _whole("h", h, dev, _torch.float32, (T, k, K)), _whole("ids", ids, dev, _torch.int32, (T, k)),
          _whole("weights", weights, dev, _torch.float32, (T, k)), _whole("residual", residual, dev, _torch.float32, (T, N)),
          _whole("y", y, dev, _torch.float32, (T, N)), _workspace(scratch, scratch_bytes, dev), scratch_bytes, T, k, E, N, K,
          _raw_stream(dev) if stream is None else stream_handle(stream))


def qmm_blocksums(wtype, W, xq, s, M, N, K, stream=None):
    _call("qmm_blocksums", _type(wtype), ptr(W), ptr(xq), ptr(s), int(M), int(N), int(K), stream_handle(stream))


def qmm_test_wait_timeout(limit_ns: int, stream=None):
    _call("qmm_test_wait_timeout", int(limit_ns), stream_handle(stream))


def qmm_device_status(clear: bool = False) -> int:
    return int(load().qmm_device_status(1 if clear else 0))
