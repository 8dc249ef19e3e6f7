"""Python binding of libqx, the GB300 block-quantised GEMV library.

Argument marshalling only: every function here checks Python-side types,
allocates outputs with torch when the caller passes none, and calls the C ABI
of ``include/qx.h`` with raw device pointers and the current CUDA stream.  All
arithmetic runs in the CUDA kernels.  There is no fallback: if ``libqx.so`` is
missing or the device is not a GB300, calls raise ``QxError``.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

QX_Q8_0, QX_Q4_K, QX_Q6_K = 8, 12, 14
QX_Q6_K_SOA = 142  # Q6_K repacked at load time (qx_repack)
QX_MODE_F32, QX_MODE_W4A8, QX_MODE_W4A8_FUSED = 0, 1, 2
QX_FLAG_PDL = 0x100
QX_OK = 0
QX_ERR_ARG, QX_ERR_FMT, QX_ERR_SHAPE, QX_ERR_ALIGN = -1, -2, -3, -4
QX_ERR_MODE, QX_ERR_CUDA, QX_ERR_DEVICE_TIMEOUT, QX_ERR_UNSUPPORTED_DEVICE = -5, -6, -7, -8
QX_ERR_RANGE = -9
QX_MAX_MULTI = 8
QX_MAX_COLS = 32768
QX_CHAIN_MAX_JOBS = 128
QX_CHAIN_MAX_ENTRIES = 4
QX_F32, QX_F16, QX_BF16 = 0, 1, 30  # element types
QX_MAX_HEAD_DIM = 256
QX_MAX_GROUP = 128
QX_ATTN_COUNTER_BYTES = 2304

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqx.so")

EXPORTS = ["qx_quantize_act_q8", "qx_gemv", "qx_gemv_multi", "qx_gemm_prefill", "qx_gemm_prefill_ex",
           "qx_gemv_partials", "qx_gemv_chain", "qx_gemv_chain_noalloc", "qx_gemv_chain_scratch_bytes", "qx_row_bytes", "qx_repack",
           "qx_rope_append", "qx_attn_paged", "qx_attn_shared", "qx_attn_scratch_bytes", "qx_block_norm", "qx_stream_capture_id",
           "qx_device_check", "qx_debug_timeout_probe", "qx_debug_agree_probe", "qx_debug_mma_rate", "qx_debug_noalloc_fill",
           "qx_debug_trace_read", "qx_status_string", "qx_last_error", "qx_version"]


class QxError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = f" [{qx_last_error()}]" if status == QX_ERR_CUDA else ""
        super().__init__(f"{what}: {qx_status_string(status)} ({status}){detail}")


class _Act(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("d", ctypes.c_void_p), ("sum", ctypes.c_void_p),
                ("m", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _Job(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("n", ctypes.c_int), ("W", ctypes.c_void_p * 4),
                ("rows", ctypes.c_int64 * 4), ("y", ctypes.c_void_p * 4), ("cols", ctypes.c_int64),
                ("x", ctypes.c_void_p)]


class _Kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_size", ctypes.c_int), ("n_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("kv_len", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p), ("n_seqs", ctypes.c_int)]


class _Qkv(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("n_q_heads", ctypes.c_int), ("dtype", ctypes.c_int),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


class _Norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dtype", ctypes.c_int), ("res_dtype", ctypes.c_int),
                ("y", ctypes.c_void_p), ("r", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("w_post", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("alpha", ctypes.c_float), ("eps", ctypes.c_float),
                ("r_out", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y_stride", ctypes.c_int64),
                ("r_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("r_out_stride", ctypes.c_int64),
                ("x_stride", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libqx.so (built by ``build()``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libqx.so not found at {LIB_PATH}: build it with "
                               "`python -m block_quantized_gemv_q8_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.qx_quantize_act_q8.argtypes = [P, I64, I64, ctypes.POINTER(_Act), P]
        L.qx_gemv.argtypes = [I, P, I64, I64, P, P, I, P]
        L.qx_gemv_multi.argtypes = [I, P, P, P, I64, P, P, I, P]
        L.qx_gemm_prefill.argtypes = [I, P, I64, I64, ctypes.POINTER(_Act), P, P]
        L.qx_gemm_prefill_ex.argtypes = [I, P, I64, I64, ctypes.POINTER(_Act), P, I, P]
        L.qx_gemv_partials.argtypes = [I, P, I64, I64, ctypes.POINTER(_Act), P, P]
        L.qx_gemv_chain.argtypes = [I, ctypes.POINTER(_Job), P, P]
        L.qx_gemv_chain_noalloc.argtypes = [I, ctypes.POINTER(_Job), P]
        L.qx_gemv_chain_scratch_bytes.argtypes = [I]
        L.qx_gemv_chain_scratch_bytes.restype = ctypes.c_size_t
        L.qx_row_bytes.argtypes = [I, I64]
        L.qx_row_bytes.restype = ctypes.c_size_t
        L.qx_device_check.argtypes = [P]
        L.qx_repack.argtypes = [I, I, P, I64, I64, P, P]
        L.qx_rope_append.argtypes = [P, P, P, P, I64, I, I, P, P]
        L.qx_attn_paged.argtypes = [P, P, I64, I, I64, ctypes.c_float, I64, I64, P, I, P, P, P]
        L.qx_attn_shared.argtypes = [P, P, I64, I, I64, ctypes.c_float, I64, P, I, P, P, P]
        L.qx_attn_scratch_bytes.argtypes = [I64, I, I, I, I]
        L.qx_attn_scratch_bytes.restype = ctypes.c_size_t
        L.qx_block_norm.argtypes = [P, P]
        L.qx_stream_capture_id.argtypes = [P]
        L.qx_stream_capture_id.restype = ctypes.c_uint64
        L.qx_debug_mma_rate.argtypes = [I, ctypes.POINTER(ctypes.c_double), P]
        L.qx_debug_timeout_probe.argtypes = [ctypes.c_uint64, P]
        L.qx_debug_agree_probe.argtypes = [ctypes.c_uint64, P, P]
        L.qx_debug_noalloc_fill.argtypes = [ctypes.c_uint32, P]
        L.qx_debug_trace_read.argtypes = [P, ctypes.c_size_t]
        L.qx_status_string.argtypes = [I]
        L.qx_status_string.restype = ctypes.c_char_p
        L.qx_last_error.argtypes = []
        L.qx_last_error.restype = ctypes.c_char_p
        L.qx_version.argtypes = []
        L.qx_version.restype = ctypes.c_char_p
        for n in ("qx_quantize_act_q8", "qx_gemv", "qx_gemv_multi", "qx_gemm_prefill", "qx_gemm_prefill_ex",
                  "qx_gemv_partials", "qx_gemv_chain", "qx_gemv_chain_noalloc",
                  "qx_device_check", "qx_debug_timeout_probe", "qx_debug_agree_probe",
                  "qx_repack", "qx_rope_append", "qx_attn_paged", "qx_attn_shared", "qx_block_norm", "qx_debug_mma_rate", "qx_debug_noalloc_fill",
                  "qx_debug_trace_read"):
            getattr(L, n).restype = I
        _lib = L
    return _lib


def build_library(force: bool = False) -> str:
    """Compile libqx.so in-tree (nvcc, sm_103a)."""
    import importlib
    return importlib.import_module(__name__ + ".build").build(force=force)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    if not t.is_cuda:
        raise ValueError("qx operates on CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("qx needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _need(t: torch.Tensor, nbytes: int, what: str) -> torch.Tensor:
    """A CUDA, contiguous tensor holding at least nbytes: the library writes and
    reads through raw pointers, so a short buffer is refused here."""
    _ptr(t)
    if nbytes > 0 and _nbytes(t) < nbytes:
        raise ValueError(f"{what}: {_nbytes(t)} bytes, need {nbytes}")
    return t


def _need_weights(W: torch.Tensor, fmt: int, rows: int, cols: int, what: str = "W") -> torch.Tensor:
    rb = qx_row_bytes(fmt, cols)
    return _need(W, rows * rb, what) if rb > 0 and rows > 0 else W  # invalid shapes: the library names them


def _served_cols(fmt: int, cols: int) -> int:
    """cols when the format serves that width, else 0: an invalid shape is left
    to the library, which names it (QX_ERR_SHAPE / QX_ERR_FMT)."""
    return cols if qx_row_bytes(fmt, cols) > 0 else 0


def _need_act(a: "ActQ8", m: int, cols: int, what: str):
    _need(a.q, m * cols, what + ".q")
    _need(a.d, m * (cols // 32) * 4, what + ".d")
    _need(a.sum, m * (cols // 32) * 4, what + ".sum")


def _check(st: int, what: str):
    if st != QX_OK:
        raise QxError(st, what)


@dataclass
class ActQ8:
    """An int8-quantised activation: q [m, cols] int8, d and sum [m, cols/32]."""
    q: torch.Tensor
    d: torch.Tensor
    sum: torch.Tensor

    @property
    def m(self) -> int:
        return self.q.shape[0]

    @property
    def cols(self) -> int:
        return self.q.shape[1]

    @staticmethod
    def empty(m: int, cols: int, device=None) -> "ActQ8":
        device = device or torch.device("cuda")
        return ActQ8(torch.empty((m, cols), dtype=torch.int8, device=device),
                     torch.empty((m, cols // 32), dtype=torch.float32, device=device),
                     torch.empty((m, cols // 32), dtype=torch.int32, device=device))

    def c_struct(self) -> _Act:
        return _Act(_ptr(self.q).value, _ptr(self.d).value, _ptr(self.sum).value, self.m, self.cols)

    def row(self, i: int) -> "ActQ8":
        return ActQ8(self.q[i:i + 1], self.d[i:i + 1], self.sum[i:i + 1])


def qx_row_bytes(fmt: int, cols: int) -> int:
    return int(lib().qx_row_bytes(fmt, cols))


def qx_repack(from_fmt: int, to_fmt: int, W: torch.Tensor, rows: int, cols: int, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Repack rows x cols weights between QX_Q6_K and QX_Q6_K_SOA (device to device)."""
    nbytes = rows * qx_row_bytes(to_fmt, cols)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    _need_weights(W, from_fmt, rows, cols)
    _need(out, nbytes, "out")
    _check(lib().qx_repack(from_fmt, to_fmt, _ptr(W), rows, cols, _ptr(out), _stream(stream)), "qx_repack")
    return out


def qx_status_string(st: int) -> str:
    return lib().qx_status_string(st).decode()


def qx_last_error() -> str:
    return lib().qx_last_error().decode()


def qx_version() -> str:
    return lib().qx_version().decode()


def qx_quantize_act_q8(x: torch.Tensor, out: ActQ8 | None = None, stream=None) -> ActQ8:
    """x f32 [m, cols] (or [cols]) -> ActQ8 (int8 per block of 32 with an f32 absmax scale)."""
    if x.dtype != torch.float32:
        raise TypeError("qx_quantize_act_q8 takes float32 activations")
    x2 = x.reshape(1, -1) if x.dim() == 1 else x
    m, cols = x2.shape
    out = out or ActQ8.empty(m, cols, x.device)
    _need_act(out, m, cols, "out")
    a = out.c_struct()
    _check(lib().qx_quantize_act_q8(_ptr(x2), m, cols, ctypes.byref(a), _stream(stream)), "qx_quantize_act_q8")
    return out


def _x_arg(x, mode, cols: int = 0):
    if (mode & 0xFF) in (QX_MODE_F32, QX_MODE_W4A8_FUSED):
        if not isinstance(x, torch.Tensor) or x.dtype != torch.float32:
            raise TypeError("f32 and fused-W4A8 modes take a float32 activation tensor")
        return _ptr(_need(x, cols * 4, "x")), None
    if not isinstance(x, ActQ8):
        raise TypeError("W4A8 mode takes an ActQ8 (from qx_quantize_act_q8)")
    _need_act(x, 1, cols, "x")
    a = x.c_struct()
    return ctypes.cast(ctypes.pointer(a), ctypes.c_void_p), a


def qx_gemv(fmt: int, W: torch.Tensor, rows: int, cols: int, x, y: torch.Tensor | None = None,
            mode: int = QX_MODE_W4A8, stream=None) -> torch.Tensor:
    """y[rows] = W . x for block-quantised W (uint8 bytes).

    mode: QX_MODE_F32 (x f32), QX_MODE_W4A8 (x an ActQ8) or QX_MODE_W4A8_FUSED
    (x f32, quantised inside the launch), optionally | QX_FLAG_PDL."""
    y = y if y is not None else torch.empty(rows, dtype=torch.float32, device=W.device)
    _need_weights(W, fmt, rows, cols)
    _need(y, rows * 4, "y")
    xp, keep = _x_arg(x, mode, _served_cols(fmt, cols))
    _check(lib().qx_gemv(fmt, _ptr(W), rows, cols, xp, _ptr(y), mode, _stream(stream)), "qx_gemv")
    return y


def qx_gemv_multi(fmts, Ws, rows, cols: int, x, ys=None, mode: int = QX_MODE_W4A8, stream=None):
    """Several GEMVs over one activation in one launch per format."""
    n = len(Ws)
    ys = ys if ys is not None else [torch.empty(r, dtype=torch.float32, device=Ws[0].device) for r in rows]
    if not (len(fmts) == len(rows) == len(ys) == n):
        raise ValueError("qx_gemv_multi: fmts, Ws, rows and ys differ in length")
    for f, w, r, y in zip(fmts, Ws, rows, ys):
        _need_weights(w, f, r, cols)
        _need(y, r * 4, "y")
    F = (ctypes.c_int * n)(*fmts)
    Wp = (ctypes.c_void_p * n)(*[_ptr(w).value for w in Ws])
    R = (ctypes.c_int64 * n)(*rows)
    Yp = (ctypes.c_void_p * n)(*[_ptr(t).value for t in ys])
    xp, keep = _x_arg(x, mode, min(_served_cols(f, cols) for f in fmts) if n else 0)
    _check(lib().qx_gemv_multi(n, F, Wp, R, cols, xp, Yp, mode, _stream(stream)), "qx_gemv_multi")
    return ys


def qx_gemv_partials(fmt: int, W: torch.Tensor, rows: int, cols: int, x: ActQ8, P: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Exact int32 partial sums [rows, cols/32] (Q4_K, Q8_0) or [rows, cols/16] (Q6_K, QX_Q6_K_SOA)."""
    g = 16 if fmt in (QX_Q6_K, QX_Q6_K_SOA) else 32
    P = P if P is not None else torch.empty((rows, cols // g), dtype=torch.int32, device=W.device)
    _need_weights(W, fmt, rows, cols)
    _need(P, rows * (cols // g) * 4, "P")
    _need_act(x, 1, _served_cols(fmt, cols), "x")
    a = x.c_struct()
    _check(lib().qx_gemv_partials(fmt, _ptr(W), rows, cols, ctypes.byref(a), _ptr(P), _stream(stream)),
           "qx_gemv_partials")
    return P


def qx_gemm_prefill(fmt: int, W: torch.Tensor, rows: int, cols: int, X: ActQ8, Y: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Y [X.m, rows] = X' . W^T for a quantised activation batch X."""
    return qx_gemm_prefill_ex(fmt, W, rows, cols, X, Y, 0, stream)


def qx_gemm_prefill_ex(fmt: int, W: torch.Tensor, rows: int, cols: int, X: ActQ8, Y: torch.Tensor | None = None,
                       path: int = 0, stream=None) -> torch.Tensor:
    Y = Y if Y is not None else torch.empty((X.m, rows), dtype=torch.float32, device=W.device)
    _need_weights(W, fmt, rows, cols)
    _need(Y, X.m * rows * 4, "Y")
    _need_act(X, X.m, _served_cols(fmt, cols), "X")
    a = X.c_struct()
    _check(lib().qx_gemm_prefill_ex(fmt, _ptr(W), rows, cols, ctypes.byref(a), _ptr(Y), path, _stream(stream)),
           "qx_gemm_prefill_ex")
    return Y


@dataclass
class GemvJob:
    """One job of a chain: y[k] = W[k] . x for its entries (W4A8, in-kernel quantisation)."""
    fmt: int
    W: list
    rows: list
    cols: int
    x: torch.Tensor
    y: list | None = None


def qx_gemv_chain_scratch_bytes(n_jobs: int) -> int:
    return int(lib().qx_gemv_chain_scratch_bytes(n_jobs))


def chain_scratch(n_jobs: int, device=None) -> torch.Tensor:
    """Zero-filled scratch for a chain of n_jobs (reusable across calls)."""
    return torch.zeros(qx_gemv_chain_scratch_bytes(n_jobs), dtype=torch.uint8, device=device or "cuda")


def make_chain(jobs) -> ctypes.Array:
    """Marshal a list of GemvJob into the C array (outputs allocated if missing)."""
    arr = (_Job * len(jobs))()
    for j, job in enumerate(jobs):
        if job.y is None:
            job.y = [torch.empty(r, dtype=torch.float32, device=job.W[0].device) for r in job.rows]
        c = arr[j]
        c.fmt, c.n, c.cols = job.fmt, len(job.W), job.cols
        for k, (W, r, y) in enumerate(zip(job.W, job.rows, job.y)):
            _need_weights(W, job.fmt, r, job.cols)
            _need(y, r * 4, "y")
            c.W[k] = _ptr(W).value
            c.rows[k] = r
            c.y[k] = _ptr(y).value
        c.x = _ptr(_need(job.x, _served_cols(job.fmt, job.cols) * 4, "x")).value
    return arr


def qx_gemv_chain(jobs, scratch: torch.Tensor, stream=None, marshalled=None):
    """Run a chain of dependent GEMVs in one launch; returns the jobs (with y)."""
    arr = marshalled if marshalled is not None else make_chain(jobs)
    _check(lib().qx_gemv_chain(len(arr), arr, _ptr(scratch), _stream(stream)), "qx_gemv_chain")
    return jobs


def qx_gemv_chain_noalloc(jobs, stream=None, marshalled=None):
    """qx_gemv_chain with the library's own arrival counters (no scratch; at
    most QX_CHAIN_MAX_JOBS jobs; calls on one device must not overlap)."""
    arr = marshalled if marshalled is not None else make_chain(jobs)
    _check(lib().qx_gemv_chain_noalloc(len(arr), arr, _stream(stream)), "qx_gemv_chain_noalloc")
    return jobs


_F32 = torch.float32
_DTYPE = {torch.float32: QX_F32, torch.float16: QX_F16, torch.bfloat16: QX_BF16}


# These calls are short, so their marshalling is kept short too: the C structs
# are packed as bytes in one step, and the current stream is asked for by its
# number (torch.cuda.current_stream builds an object, 2 us).
_PACK_QKV = struct.Struct("qiiPPPqqq")
_PACK_NORM = struct.Struct("qqiiPPPPPffPPqqqqq")
assert _PACK_QKV.size == ctypes.sizeof(_Qkv) and _PACK_NORM.size == ctypes.sizeof(_Norm)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _raw_stream(stream, index: int) -> int:
    if stream is None:
        return _current_raw_stream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output for a call on `stream` (None: the current one).

    It is the call's stream's memory: another stream's could still be in use
    there, or be given to others there while the call writes it.  The current
    stream, whose program holds it, is noted as a user."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _heads(t: torch.Tensor, shape: tuple, dtype, index: int, what: str) -> int:
    """Token stride of a [tokens, heads, dim] tensor on GPU `index` whose heads of a token lie one after another."""
    if t.get_device() != index:
        raise ValueError(f"{what} is not on the cache's GPU" if t.is_cuda else "qx operates on CUDA tensors only")
    if t.dtype != dtype:
        raise TypeError(f"{what}: {t.dtype}, need {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, need {shape}")
    a, b, c = t.stride()
    if (c != 1 and shape[2] > 1) or (b != shape[2] and shape[1] > 1):
        raise ValueError(f"{what}: a token's heads must lie one after another (strides {(a, b, c)})")
    return a if shape[0] > 1 else shape[1] * shape[2]


def _cleared(index: int, stream: int, nbytes: int):
    """`nbytes` of GPU memory for attention calls on `stream`, their counters zeroed in the stream's order."""
    device = torch.device("cuda", index)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device)):
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        buf[:QX_ATTN_COUNTER_BYTES].zero_()
    return buf.data_ptr(), buf


class _Scratch:
    """The attention calls' scratch: a buffer for each stream, and buffers for captures.

    A stream's buffer grows when a call needs more; the old one goes back to
    the allocator, which reuses it in the stream's order.  A call under capture
    never gets it: the graph would keep an address that is given back one day,
    and its replays may run beside the stream's own calls.  Its buffer is part
    of the graph's memory, like any tensor made under capture, and is cleared by
    a node of the graph, so that each replay starts from zeroed counters; the
    calls of one capture on one stream share it."""

    def __init__(self, allocate=_cleared):
        self._allocate = allocate  # (index, stream, bytes) -> address, owner
        self._streams: dict = {}   # (index, stream) -> bytes, address, owner
        self._captures: dict = {}  # capture -> the same for its streams

    def get(self, index: int, stream: int, capture: int, need: int) -> int:
        """Address of at least `need` bytes for a call on a stream, in capture `capture` (0: none)."""
        if capture:
            held = self._captures.get(capture)
            if held is None:
                held = {}
                # Captures that are over need nothing of ours, and one that is
                # not gets another cleared buffer.
                self._captures = {capture: held}
        else:
            held = self._streams
        have = held.get((index, stream))
        if have is None or have[0] < need:
            address, owner = self._allocate(index, stream, need)
            have = held[index, stream] = (need, address, owner)
        return have[1]

    def drop(self):
        """Let all buffers go: calls that did not complete may have left their counters anywhere."""
        self._streams, self._captures = {}, {}


class PagedKV:
    """A paged key/value cache and the batch that calls run on (``qx_kv``).

    k, v: float16 or bfloat16 [n_pages, heads, page_size, head_dim], the last
    dimension contiguous (other orders as permuted views: a [page, slot, head,
    dim] cache is ``cache.transpose(1, 2)``); table: int32 [n_seqs, pages];
    kv_len: int32 [n_seqs]; q_start: int32 [n_seqs + 1].  The tensors are the
    caller's: the program updates the contents of table, kv_len and q_start in
    place from step to step (also between replays of a captured graph) and the
    calls read them on the GPU.  The object keeps them alive.  The attention
    calls' scratch is shared by all caches, one for each stream; calls under
    capture take theirs from the graph's own memory."""

    # Calls on one stream run one after another, so the caches of a stack's
    # layers share its buffer (32 query heads of 128, 265 tokens or more: 144 MB).
    _scratch = _Scratch()

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, kv_len: torch.Tensor,
                 q_start: torch.Tensor):
        for t, what in ((k, "k"), (v, "v"), (table, "table"), (kv_len, "kv_len"), (q_start, "q_start")):
            if not t.is_cuda:
                raise ValueError("qx operates on CUDA tensors only")
            if t.device != k.device:
                raise ValueError(f"{what} is on {t.device}, k on {k.device}")
        if k.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("a cache holds float16 or bfloat16")
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v need one shape [n_pages, heads, page_size, head_dim], one type and one layout")
        if k.stride(3) != 1:
            raise ValueError("the elements of a head must be contiguous")
        for t, what in ((table, "table"), (kv_len, "kv_len"), (q_start, "q_start")):
            if t.dtype != torch.int32:
                raise TypeError(f"{what}: {t.dtype}, need int32")
            if not t.is_contiguous():
                raise ValueError("qx needs contiguous tensors")
        n = kv_len.numel()
        if table.dim() != 2 or table.shape[0] != n or q_start.numel() != n + 1:
            raise ValueError("table [n_seqs, pages], kv_len [n_seqs] and q_start [n_seqs + 1] differ in n_seqs")
        self.k, self.v, self.table, self.kv_len, self.q_start = k, v, table, kv_len, q_start
        self.dtype, self.device, self.n_seqs, self._index = k.dtype, k.device, n, k.get_device()
        pages, self.heads, self.page_size, self.head_dim = k.shape
        self._c = _Kv(k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], self.heads, self.head_dim, self.page_size, pages,
                      k.stride(0), k.stride(1), k.stride(2), table.data_ptr(), table.shape[1], kv_len.data_ptr(),
                      q_start.data_ptr(), n)
        self._ref = ctypes.byref(self._c)
        self._needs: dict = {}

    def scratch(self, tokens: int, q_heads: int, stream: int, capture: int = 0) -> int:
        """Address of the scratch of a call of these sizes on `stream`, in capture `capture` (0: none)."""
        need = self._needs.get((tokens, q_heads))
        if need is not None and not capture:  # (the common case in line)
            have = self._scratch._streams.get((self._index, stream))
            if have is not None and have[0] >= need:
                return have[1]
        if need is None:
            if len(self._needs) >= 256:
                self._needs.clear()
            need = max(256, int(lib().qx_attn_scratch_bytes(tokens, q_heads, self.heads, self.head_dim, self.n_seqs)))
            self._needs[tokens, q_heads] = need
        return self._scratch.get(self._index, stream, capture, need)


def qx_rope_append(kv: PagedKV, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                   cos: torch.Tensor | None = None, sin: torch.Tensor | None = None, interleaved: bool = False,
                   q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Rotate q [tokens, q_heads, dim] and k [tokens, heads, dim] by position, append k and v to the cache.

    cos, sin: float32 [positions, rot / 2] (None: no rotation); interleaved:
    pairs (2i, 2i + 1) instead of (i, i + rot / 2).  Returns the rotated
    queries in the cache's type."""
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k and v: need [tokens, heads, dim]")
    index, dim, dt = kv._index, kv.head_dim, k.dtype
    code = _DTYPE.get(dt)
    if code is None:
        raise TypeError(f"k: {dt} is not float32, float16 or bfloat16")
    shape = k.shape
    n = shape[0]
    (k_stride, kb, kc), (v_stride, vb, vc) = k.stride(), v.stride()
    # (the common case in line: a call of a helper costs as much as its checks)
    if not (shape == (n, kv.heads, dim) and v.shape == shape and v.dtype is dt and kb == vb == dim and kc == vc == 1
            and k.get_device() == index and v.get_device() == index):
        own = (n, kv.heads, dim)
        k_stride, v_stride = _heads(k, own, dt, index, "k"), _heads(v, own, dt, index, "v")
    hq = q_ptr = q_stride = n_pos = half = 0
    out = cp = sp = None
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q: need [tokens, heads, dim]")
        hq = q.shape[1]
        (q_stride, qb, qc), q_ptr = q.stride(), q.data_ptr()
        if not (q.shape == (n, hq, dim) and q.dtype is dt and qb == dim and qc == 1 and q.get_device() == index):
            q_stride = _heads(q, (n, hq, dim), dt, index, "q")
        if q_out is None:
            q_out = _empty((n, hq, dim), kv.dtype, kv.device, stream)
        elif q_out.dtype != kv.dtype or q_out.shape != q.shape or not q_out.is_contiguous() or q_out.get_device() != index:
            raise ValueError("q_out: need a contiguous tensor on the cache's GPU, of q's shape and the cache's type")
        out = q_out.data_ptr()
    if cos is not None:
        if sin is None or cos.shape != sin.shape or cos.dim() != 2:
            raise ValueError("cos and sin need one shape [positions, rot / 2]")
        if cos.dtype != torch.float32 or sin.dtype != torch.float32:
            raise TypeError("cos and sin are float32")
        if cos.get_device() != index or sin.get_device() != index or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin: need contiguous tensors on the cache's GPU")
        n_pos, half = cos.shape
        cp, sp = cos.data_ptr(), sin.data_ptr()
    if n == 1:  # a single token's stride means nothing, and may be anything
        k_stride = v_stride = q_stride = dim
    a = _PACK_QKV.pack(n, hq, code, q_ptr, k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride)
    st = lib().qx_rope_append(kv._ref, a, cp, sp, n_pos, 2 * half, 1 if interleaved else 0, out, _raw_stream(stream, index))
    if st:
        _check(st, "qx_rope_append")
    return q_out


def _attn(kv: PagedKV, q: torch.Tensor, scale, out, lse, stream):
    """The arguments before and after the mask's in the C calls."""
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q: need [tokens, heads, dim]")
    n, hq, dim = shape
    index = kv._index
    q_stride = _heads(q, (n, hq, kv.head_dim), kv.dtype, index, "q")
    if out is None:
        out = _empty(shape, kv.dtype, kv.device, stream)
    elif out.shape != shape or not out.is_contiguous() or out.get_device() != index:
        raise ValueError("out: need a contiguous tensor on the cache's GPU, of q's shape")
    code = _DTYPE.get(out.dtype)
    if code is None:
        raise TypeError(f"out: {out.dtype} is not float32, float16 or bfloat16")
    lp = None
    if lse is not None:
        if lse.dtype != torch.float32:
            raise TypeError("lse is float32")
        lp = _ptr(_need(lse, n * hq * 4, "lse"))
    s = _raw_stream(stream, index)
    # (the question about the current stream takes 0.1 us, the other one 0.5)
    capture = 0 if stream is None and not _capturing() else lib().qx_stream_capture_id(s)
    return (kv._ref, q.data_ptr(), n, hq, q_stride, dim ** -0.5 if scale is None else scale), out, \
        (out.data_ptr(), code, lp, kv.scratch(n, hq, s, capture), s)


def qx_attn_paged(kv: PagedKV, q: torch.Tensor, scale: float | None = None, window: int = 0, sinks: int = 0,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of q [tokens, q_heads, dim] over the cache; scale None: dim ** -0.5.

    window > 0: a token sees the last `window` keys up to its own and the first
    `sinks`.  out: the cache's type or float32; lse: float32 [tokens, q_heads],
    filled with the rows' log-sum-exp."""
    head, out, tail = _attn(kv, q, scale, out, lse, stream)
    st = lib().qx_attn_paged(*head, window, sinks, *tail)
    if st:
        _check(st, "qx_attn_paged")
    return out


def qx_attn_shared(kv: PagedKV, q: torch.Tensor, shared_len: int, scale: float | None = None,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qx_attn_paged for sequences that all begin with the same `shared_len` keys and values, read once for all."""
    head, out, tail = _attn(kv, q, scale, out, lse, stream)
    st = lib().qx_attn_shared(*head, shared_len, *tail)
    if st:
        _check(st, "qx_attn_shared")
    return out


def _rows(t: torch.Tensor, shape, dtype, index: int, what: str) -> int:
    """Row stride of a [rows, cols] tensor on GPU `index` with contiguous rows."""
    if t.get_device() != index:
        raise ValueError(f"{what} is not on r's GPU" if t.is_cuda else "qx operates on CUDA tensors only")
    if t.dtype != dtype:
        raise TypeError(f"{what}: {t.dtype}, need {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, need {tuple(shape)}")
    a, b = t.stride()
    if b != 1 and shape[1] > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return a if shape[0] > 1 else shape[1]


def _vector(t: torch.Tensor, cols: int, dtype, index: int, what: str) -> int:
    """Address of a contiguous vector of `cols` elements on GPU `index`."""
    if t.get_device() != index:
        raise ValueError(f"{what} is not on r's GPU" if t.is_cuda else "qx operates on CUDA tensors only")
    if t.dtype != dtype:
        raise TypeError(f"{what}: {t.dtype}, need {dtype}")
    if t.numel() != cols or not t.is_contiguous():
        raise ValueError(f"{what}: need {cols} contiguous elements")
    return t.data_ptr()


def qx_block_norm(y: torch.Tensor | None, r: torch.Tensor, w_post: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, alpha: float = 1.0, w_pre: torch.Tensor | None = None,
                  eps: float = 1e-5, r_out: torch.Tensor | None = None, x_out: torch.Tensor | None = None, stream=None):
    """r' = r + alpha * gate * norm(y) and x = norm(r'), a row at a time; returns (r', x).

    y (a block's output; None: x is the norm of r), gate ([rows, cols], or
    [cols] for all rows) and x share a type, r and r' another; w_post (None:
    y as it is) and w_pre (None: no x) are float32 [cols].  r_out may be r, and
    x_out may be y."""
    shape = r.shape
    if len(shape) != 2:
        raise ValueError("r: need [rows, cols]")
    index, res, cols = r.get_device(), r.dtype, shape[1]
    if index < 0:
        raise ValueError("qx operates on CUDA tensors only")
    act = y.dtype if y is not None else x_out.dtype if x_out is not None else res
    code, res_code = _DTYPE.get(act), _DTYPE.get(res)
    if code is None or res_code is None:
        raise TypeError("qx_block_norm takes float32, float16 and bfloat16")
    # (the common case of each tensor in line: a call of a helper costs as much as its checks)
    strides = r.stride()
    r_stride = strides[0] if strides[1] == 1 else _rows(r, shape, res, index, "r")
    y_ptr = gate_ptr = post = pre = ro_ptr = x_ptr = y_stride = gate_stride = ro_stride = x_stride = 0
    if y is not None:
        strides, y_ptr = y.stride(), y.data_ptr()
        y_stride = strides[0] if y.dtype is act and y.shape == shape and strides[1] == 1 and y.get_device() == index else \
            _rows(y, shape, act, index, "y")
    if gate is not None:
        if gate.dim() == 1:
            gate_ptr = _vector(gate, cols, act, index, "gate")
        else:
            gate_ptr, gate_stride = gate.data_ptr(), _rows(gate, shape, act, index, "gate")
    if w_post is not None:
        post = w_post.data_ptr()
        if not (w_post.dtype is _F32 and w_post.get_device() == index and w_post.shape == (cols,) and w_post.is_contiguous()):
            _vector(w_post, cols, _F32, index, "w_post")
    if y is None and r_out is None:
        r_out = r  # unchanged
    else:
        if r_out is None:
            r_out = _empty(shape, res, r.device, stream)
        strides, ro_ptr = r_out.stride(), r_out.data_ptr()
        ro_stride = strides[0] if r_out.dtype is res and r_out.shape == shape and strides[1] == 1 and r_out.get_device() == index else \
            _rows(r_out, shape, res, index, "r_out")
    if w_pre is not None:
        pre = w_pre.data_ptr()
        if not (w_pre.dtype is _F32 and w_pre.get_device() == index and w_pre.shape == (cols,) and w_pre.is_contiguous()):
            _vector(w_pre, cols, _F32, index, "w_pre")
        if x_out is None:
            x_out = _empty(shape, act, r.device, stream)
        strides, x_ptr = x_out.stride(), x_out.data_ptr()
        x_stride = strides[0] if x_out.dtype is act and x_out.shape == shape and strides[1] == 1 and x_out.get_device() == index else \
            _rows(x_out, shape, act, index, "x_out")
    else:
        x_out = None
    a = _PACK_NORM.pack(shape[0], cols, code, res_code, y_ptr, r.data_ptr(), gate_ptr, post, pre, alpha, eps, ro_ptr, x_ptr, y_stride,
                        r_stride, gate_stride, ro_stride, x_stride)
    st = lib().qx_block_norm(a, _raw_stream(stream, index))
    if st:
        _check(st, "qx_block_norm")
    return r_out, x_out


def qx_debug_mma_rate(kind: int, stream=None) -> float:
    """Measured mma.sync rate (multiply-adds x 2 per second): kind 0 int8 m16n8k32, 1 f16 m16n8k16."""
    v = ctypes.c_double(0.0)
    _check(lib().qx_debug_mma_rate(kind, ctypes.byref(v), _stream(stream)), "qx_debug_mma_rate")
    return v.value


def qx_device_check(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status.

    After a wait that ran out the attention calls start from new scratch."""
    st = int(lib().qx_device_check(_stream(stream)))
    if st == QX_ERR_DEVICE_TIMEOUT:
        PagedKV._scratch.drop()
    return st


def qx_debug_timeout_probe(limit_ns: int, stream=None):
    _check(lib().qx_debug_timeout_probe(limit_ns, _stream(stream)), "qx_debug_timeout_probe")


def qx_debug_agree_probe(limit_ns: int, got: torch.Tensor, stream=None):
    """Four waiting warps of which one gives up; got (int32 [4]): see qx_debug.h."""
    _check(lib().qx_debug_agree_probe(limit_ns, _ptr(_need(got, 16, "got")), _stream(stream)), "qx_debug_agree_probe")


def qx_debug_noalloc_fill(value: int, stream=None):
    """Fill the library's no-alloc chain counter array with `value` (test hook)."""
    _check(lib().qx_debug_noalloc_fill(value, _stream(stream)), "qx_debug_noalloc_fill")
