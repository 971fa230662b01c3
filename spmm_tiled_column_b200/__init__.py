"""spmm_tiled_column_b200 -- Python binding of libspw.so, the sparse-weight SpMV/SpMM library.

Argument marshalling only: every function below checks tensor dtypes/devices, allocates
outputs with torch when the caller did not pass them, and calls the C function of the
same name in libspw.so (see include/spw.h) on torch's current CUDA stream.  All compute
runs in the library's CUDA kernels; there is no CPU path.  If libspw.so is missing or
cannot be loaded, the first call raises.

Tensors: fp16 weights / activations as torch.float16 (or int16/uint16 bit views), the
mask as torch.uint8 (nonzero = kept), TCB buffers as torch.uint8, bitmaps as torch.int32.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspw.so")

SPW_OK = 0
SPW_ERR_INVALID_ARG = 1
SPW_ERR_ALIGNMENT = 2
SPW_ERR_BUFFER_TOO_SMALL = 3
SPW_ERR_FORMAT = 4
SPW_ERR_UNSUPPORTED = 5
SPW_ERR_CUDA = 6
SPW_ERR_TIMEOUT = 7

# Activations of the epilogues and of the gated block, by number or by name
SPW_ACT_NONE = 0
SPW_ACT_RELU = 1
SPW_ACT_SILU = 2
SPW_ACT_GELU = 3
SPW_ACT_GELU_TANH = 4
ACTIVATIONS = {"none": SPW_ACT_NONE, "relu": SPW_ACT_RELU, "silu": SPW_ACT_SILU,
               "gelu": SPW_ACT_GELU, "gelu_tanh": SPW_ACT_GELU_TANH}

# C function name -> (argtypes, restype)
_P = ctypes.c_void_p
_I = ctypes.c_int
_U64 = ctypes.c_uint64
_F = ctypes.c_float


class spw_format(ctypes.Structure):
    """Host copy of the TCB v1 header (same layout as the C struct)."""
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("N", ctypes.c_uint32), ("K", ctypes.c_uint32),
                ("TN", ctypes.c_uint32), ("TK", ctypes.c_uint32),
                ("n_strips", ctypes.c_uint32), ("n_ktiles", ctypes.c_uint32),
                ("nnz", ctypes.c_uint64), ("bytes_total", ctypes.c_uint64),
                ("off_bitmaps", ctypes.c_uint64), ("off_tileptr", ctypes.c_uint64),
                ("off_values", ctypes.c_uint64), ("max_tile_units", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


_FP = ctypes.POINTER(spw_format)


class spw_spmm_plan_info(ctypes.Structure):
    _fields_ = [("token_tile", ctypes.c_int32), ("token_tiles", ctypes.c_int32),
                ("weight_tiles", ctypes.c_int32), ("k_parts", ctypes.c_int32),
                ("whole_tiles", ctypes.c_int32), ("ctas", ctypes.c_int32),
                ("cta_pair", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_uint64)]


class spw_epilogue(ctypes.Structure):
    """bias, residual (with its leading dimension) and activation of a product's epilogue."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ldr", ctypes.c_int32), ("act", ctypes.c_int32)]


_EP = ctypes.POINTER(spw_epilogue)
SIGNATURES = {
    "spw_status_string": ([_I], ctypes.c_char_p),
    "spw_version": ([], _I),
    "spw_set_launch_overlap": ([_I], _I),
    "spw_set_wait_limit_cycles": ([_U64], _U64),
    "spw_set_column_fetch": ([_I], _I),
    "spw_format_query": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "spw_compress": ([_P, _I, _P, _I, _I, _I, _P, _U64, _FP, _P], _I),
    "spw_format_read": ([_P, _U64, _FP, _P], _I),
    "spw_decompress": ([_FP, _P, _P, _I, _P], _I),
    "spw_select_threshold": ([_P, _I, _I, _I, _F, _P, _P, _P], _I),
    "spw_select_topk": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "spw_spmv_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmv": ([_FP, _P, _P, _I, _I, _F, _P, _P, _I, _P, _U64, _P], _I),
    "spw_spmm_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmm": ([_FP, _P, _P, _I, _I, _P, _I, _P, _U64, _P], _I),
    "spw_spmv_tc_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmv_tc": ([_FP, _P, _P, _I, _I, _F, _P, _P, _I, _P, _U64, _P], _I),
    "spw_spmv_auto_path": ([_I], _I),
    "spw_spmv_auto_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmv_auto": ([_FP, _P, _P, _I, _I, _F, _P, _P, _I, _P, _U64, _P], _I),
    "spw_last_device_status": ([_P, _P], _I),
    "spw_spmv_group_workspace_bytes": ([_I, _FP, _I], _U64),
    "spw_spmv_group": ([_I, _FP, _P, _P, _P, _P, _P, _P, _I, _F, _P, _U64, _P], _I),
    "spw_spmv_noalloc_max_scratch_bytes": ([], _U64),
    "spw_spmv_noalloc": ([_FP, _P, _P, _I, _I, _F, _P, _P, _I, _P], _I),
    "spw_spmv_ffn_workspace_bytes": ([_FP, _FP, _I], _U64),
    "spw_spmm_plan": ([_FP, _I, _I, ctypes.POINTER(spw_spmm_plan_info)], _I),
    "spw_spmv_ffn": ([_FP, _P, _FP, _P, _P, _I, _I, _F, _P, _I, _P, _P, _U64, _P], _I),
    "spw_group_tokens_workspace_bytes": ([_I, _I], _U64),
    "spw_group_tokens": ([_P, _I, _I, _I, _F, _I, _P, _I, _P, _P, _P, _U64, _P], _I),
    "spw_spmm_tokens_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmm_tokens_plan": ([_FP, _I, _I, ctypes.POINTER(spw_spmm_plan_info)], _I),
    "spw_spmm_tokens": ([_FP, _P, _P, _I, _I, _F, _P, _I, _P, _U64, _P], _I),
    "spw_s24_bytes": ([_I, _I], _U64),
    "spw_split24": ([_P, _I, _P, _I, _I, _I, _P, _U64, _P, _I, _P], _I),
    "spw_spmm24_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmm24_plan": ([_FP, _I, _I, ctypes.POINTER(spw_spmm_plan_info)], _I),
    "spw_spmm24": ([_FP, _P, _P, _U64, _P, _I, _I, _P, _I, _P, _U64, _P], _I),
    "spw_spmv_ep_path": ([_FP, _I], _I),
    "spw_spmv_ep_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmv_ep": ([_FP, _P, _P, _I, _I, _F, _P, _EP, _P, _I, _P, _U64, _P], _I),
    "spw_spmm_ep_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmm_ep": ([_FP, _P, _P, _I, _I, _EP, _P, _I, _P, _U64, _P], _I),
    "spw_spmm_ffn_workspace_bytes": ([_FP, _FP, _I], _U64),
    "spw_spmm_ffn": ([_FP, _P, _FP, _P, _P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _U64, _P], _I),
    "spw_spmm_ffn_backward_workspace_bytes": ([_FP, _FP, _I], _U64),
    "spw_spmm_ffn_backward": ([_FP, _P, _FP, _P, _P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _P,
                               _P, _U64, _P], _I),
    "spw_spmm_backward_workspace_bytes": ([_FP, _I], _U64),
    "spw_spmm_backward": ([_FP, _P, _P, _I, _I, _P, _I, _P, _I, _P, _P, _U64, _P], _I),
}


class SpwError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libspw.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing; build it with "
                               "`python -m spmm_tiled_column_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().spw_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != SPW_OK:
        raise SpwError(fn, status)


def _stream(stream=None):
    if stream is None:  # the handle alone: building a Stream object costs 3 us a call
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def _on_stream(fn):
    """Gives a call its `stream` argument (by keyword, or after all others).  The call runs with
    that stream current, so that what it allocates belongs to the stream that uses it, and what it
    clears is cleared there."""
    n = fn.__code__.co_argcount

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if len(args) == n + 1:
            args, stream = args[:n], args[n]
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _half(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype in (torch.int16, torch.uint16):
        t = t.view(torch.float16)
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be float16 (or a 16-bit bit view), got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t


def _rows(t: torch.Tensor, name: str) -> tuple[torch.Tensor, int]:
    """2-D row-major view and its leading dimension (elements)."""
    if t.dim() == 1:
        t = t.unsqueeze(0)
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return t, _ld(t.stride(0), t.shape[0], t.shape[1], name)


_INT_MAX = 2 ** 31 - 1


def _ld(ld: int, m: int, n: int, name: str) -> int:
    """Leading dimension of an m x n view with rows ld elements apart and unit column stride.  The
    library steps from row to row by it, so rows that overlap (a broadcast, a sliding window)
    cannot be handed over; M and ld are C ints, and ctypes would cut longer numbers to 32 bits."""
    if m <= 1:  # any stride
        return n if ld > _INT_MAX else max(ld, n)
    if n <= ld <= _INT_MAX and m <= _INT_MAX:
        return ld
    if ld < n:
        raise ValueError(f"{name} is {m} x {n} with rows {ld} elements apart: they overlap "
                         "(make it contiguous)")
    raise ValueError(f"{name} is {m} x {n} with rows {ld} elements apart: the library counts both "
                     f"up to {_INT_MAX}")


def _need(t: torch.Tensor, rows: int, cols: int, name: str):
    """A 2-D view must hold at least rows x cols elements: the library reads or writes
    that much through its pointer and cannot see the tensor's size."""
    if t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError(f"{name} is {tuple(t.shape)}; the call needs at least {rows} x {cols}")


def _need_buf(buf: torch.Tensor, h, name: str = "buf"):
    if not buf.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if buf.numel() * buf.element_size() < h.bytes_total:
        raise ValueError(f"{name} holds {buf.numel() * buf.element_size()} bytes; the format "
                         f"header says {h.bytes_total}")


def _nbytes(t: torch.Tensor | None, name: str = "ws") -> int:
    """Bytes of a raw buffer handed to the library with its size (0 for None); the
    library writes through its pointer on the device, so it must be a CUDA tensor."""
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.numel() * t.element_size()


def _need_words(a: torch.Tensor | None, n: int, name: str = "act_bits"):
    """A column-set or output bit array of ceil(n / 32) 32-bit words, on the GPU."""
    if a is not None and _nbytes(a, name) < 4 * ((n + 31) // 32):
        raise ValueError(f"{name} needs at least {(n + 31) // 32} 32-bit words")


def _need_u32(a: torch.Tensor, n: int, name: str):
    """An output array of n 32-bit entries, on the GPU."""
    if _nbytes(a, name) < 4 * n:
        raise ValueError(f"{name} needs at least {n} 32-bit entries")


def _mask_like(mask: torch.Tensor, N: int, K: int) -> tuple[torch.Tensor, int]:
    """An N x K uint8 CUDA mask with unit column stride, and its leading dimension."""
    m, ld = _rows(mask, "mask")
    if m.dtype != torch.uint8 or not m.is_cuda:
        raise TypeError("mask must be a CUDA uint8 tensor")
    if tuple(m.shape) != (N, K):
        raise ValueError(f"mask is {tuple(m.shape)}; the weight is {N} x {K}")
    return m, ld


def _hdr(h) -> spw_format:
    if isinstance(h, spw_format):
        return h
    f = spw_format()
    for k, v in dict(h).items():
        setattr(f, k, int(v))
    return f


def spw_set_launch_overlap(enable: bool) -> bool:
    """Enable/disable programmatic launch overlap of consecutive spw_spmv calls (see
    include/spw.h for the one condition it needs); returns the previous setting."""
    return bool(lib().spw_set_launch_overlap(1 if enable else 0))


def spw_set_column_fetch(mode: int) -> int:
    """Decode column fetch: 0 whole tiles (default), 1 when a call carries a column set or a
    threshold above zero, 2 always; returns the previous mode (see include/spw.h)."""
    prev = int(lib().spw_set_column_fetch(int(mode)))
    if prev < 0:
        raise ValueError("column fetch mode must be 0, 1 or 2")
    return prev


def spw_set_wait_limit_cycles(cycles: int) -> int:
    """Set the limit of the kernels' bounded pipeline waits in SM cycles (0: the default,
    about one second); returns the previous limit.  A test hook for the timeout path (see
    include/spw.h)."""
    return int(lib().spw_set_wait_limit_cycles(int(cycles)))


# ------------------------------------------------------------------ format

def spw_format_query(mask: torch.Tensor, stream=None) -> tuple[int, int]:
    """(bytes_total, nnz) of the TCB v1 buffer for an N x K uint8 mask."""
    mask, ld = _rows(mask, "mask")
    if mask.dtype != torch.uint8 or not mask.is_cuda:
        raise TypeError("mask must be a CUDA uint8 tensor")
    nbytes, nnz = ctypes.c_uint64(), ctypes.c_uint64()
    _check("spw_format_query", lib().spw_format_query(
        _ptr(mask), mask.shape[0], mask.shape[1], ld, ctypes.byref(nbytes), ctypes.byref(nnz),
        _stream(stream)))
    return nbytes.value, nnz.value


@_on_stream
def spw_compress(W: torch.Tensor, mask: torch.Tensor, buf: torch.Tensor | None = None) -> tuple[torch.Tensor, spw_format]:
    """Compress W * mask into a TCB v1 buffer; returns (uint8 device buffer, header)."""
    W, ldw = _rows(_half(W, "W"), "W")
    N, K = W.shape
    mask, ldm = _mask_like(mask, N, K)
    if buf is None:
        nbytes, _ = spw_format_query(mask)
        buf = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    hdr = spw_format()
    _check("spw_compress", lib().spw_compress(
        _ptr(W), ldw, _ptr(mask), ldm, N, K, _ptr(buf), _nbytes(buf, "buf"), ctypes.byref(hdr),
        _stream()))
    return buf, hdr


def spw_format_read(buf: torch.Tensor, stream=None) -> spw_format:
    hdr = spw_format()
    _check("spw_format_read", lib().spw_format_read(_ptr(buf), _nbytes(buf, "buf"), ctypes.byref(hdr),
                                                    _stream(stream)))
    return hdr


@_on_stream
def spw_decompress(hdr, buf: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Dense masked weight (fp16, N x K) from a TCB v1 buffer."""
    h = _hdr(hdr)
    if out is None:
        out = torch.empty((h.N, h.K), dtype=torch.float16, device=buf.device)
    out2, ld = _rows(_half(out, "out"), "out")
    _need_buf(buf, h)
    _need(out2, h.N, h.K, "out")
    _check("spw_decompress", lib().spw_decompress(ctypes.byref(h), _ptr(buf), _ptr(out2), ld,
                                                  _stream()))
    return out


# ------------------------------------------------------------------ selection

def _act_words(K: int) -> int:
    return (K + 31) // 32


@_on_stream
def spw_select_threshold(x: torch.Tensor, t: float, act_bits: torch.Tensor | None = None,
                         count: torch.Tensor | None = None):
    """(act_bits int32[ceil(K/32)], count int32[1]) for the threshold rule."""
    x, ldx = _rows(_half(x, "x"), "x")
    B, K = x.shape
    if act_bits is None:
        act_bits = torch.empty(_act_words(K) + 3, dtype=torch.int32, device=x.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=x.device)
    _need_words(act_bits, K)
    _need_u32(count, 1, "count")
    _check("spw_select_threshold", lib().spw_select_threshold(
        _ptr(x), B, K, ldx, float(t), _ptr(act_bits), _ptr(count), _stream()))
    return act_bits, count


@_on_stream
def spw_select_topk(x: torch.Tensor, k: int, act_bits: torch.Tensor | None = None,
                    idx: torch.Tensor | None = None):
    """(act_bits int32[ceil(K/32)], ascending idx int32[k]) of the top-k columns."""
    x, ldx = _rows(_half(x, "x"), "x")
    B, K = x.shape
    if act_bits is None:
        act_bits = torch.empty(_act_words(K) + 3, dtype=torch.int32, device=x.device)
    if idx is None:
        idx = torch.empty(max(int(k), 1), dtype=torch.int32, device=x.device)
    _need_words(act_bits, K)
    _need_u32(idx, int(k), "idx")
    _check("spw_select_topk", lib().spw_select_topk(
        _ptr(x), B, K, ldx, int(k), _ptr(act_bits), _ptr(idx), _stream()))
    return act_bits, idx[:k]


# ------------------------------------------------------------------ products

def spw_spmv_workspace_bytes(hdr, B: int) -> int:
    h = _hdr(hdr)
    return int(lib().spw_spmv_workspace_bytes(ctypes.byref(h), int(B)))


@_on_stream
def spw_spmv(hdr, buf: torch.Tensor, x: torch.Tensor, threshold: float = 0.0,
             act_bits: torch.Tensor | None = None, y: torch.Tensor | None = None,
             ws: torch.Tensor | None = None) -> torch.Tensor:
    """Decode y (B x N fp16) = W_masked . x~ with column skipping.

    ws: a zero-initialised uint8 workspace of spw_spmv_workspace_bytes(hdr, B) bytes
    (allocated here with torch.zeros when not given)."""
    h = _hdr(hdr)
    x2, ldx = _rows(_half(x, "x"), "x")
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, h.N), dtype=torch.float16, device=x.device)
    y2, ldy = _rows(_half(y, "y"), "y")
    _need_buf(buf, h)
    _need(x2, B, h.K, "x")
    _need(y2, B, h.N, "y")
    _need_words(act_bits, h.K)
    if ws is None:
        ws = torch.zeros(max(spw_spmv_workspace_bytes(h, B), 16), dtype=torch.uint8,
                         device=x.device)
    _check("spw_spmv", lib().spw_spmv(
        ctypes.byref(h), _ptr(buf), _ptr(x2), B, ldx, float(threshold), _ptr(act_bits),
        _ptr(y2), ldy, _ptr(ws), _nbytes(ws), _stream()))
    return y


def _hdr_array(hdrs) -> ctypes.Array:
    arr = (spw_format * len(hdrs))()
    for i, h in enumerate(hdrs):
        arr[i] = _hdr(h)
    return arr


def spw_spmv_group_workspace_bytes(hdrs, B: int) -> int:
    return int(lib().spw_spmv_group_workspace_bytes(len(hdrs), _hdr_array(hdrs), int(B)))


@_on_stream
def spw_spmv_group(hdrs, bufs, xs, threshold: float = 0.0, act_bits=None, ys=None, ws=None):
    """Decode several layers in one launch; returns the list of outputs (B x N_l each)."""
    n = len(hdrs)
    harr = _hdr_array(hdrs)
    x2 = [_rows(_half(x, "x"), "x") for x in xs]
    B = x2[0][0].shape[0]
    if ys is None:
        ys = [torch.empty((B, int(h.N)), dtype=torch.float16, device=xs[0].device) for h in harr]
    y2 = [_rows(_half(y, "y"), "y") for y in ys]
    if len(bufs) != n or len(x2) != n or len(y2) != n or (act_bits is not None and len(act_bits) != n):
        raise ValueError(f"expected {n} buffers, inputs and outputs (and column sets)")
    for i, h in enumerate(harr):
        _need_buf(bufs[i], h, f"bufs[{i}]")
        _need(x2[i][0], B, h.K, f"xs[{i}]")
        _need(y2[i][0], B, h.N, f"ys[{i}]")
        _need_words(None if act_bits is None else act_bits[i], h.K, f"act_bits[{i}]")
    if ws is None:
        ws = torch.zeros(max(spw_spmv_group_workspace_bytes(hdrs, B), 16), dtype=torch.uint8,
                         device=xs[0].device)
    P = ctypes.c_void_p * n
    I = ctypes.c_int * n
    ab = None if act_bits is None else P(*[None if a is None else a.data_ptr() for a in act_bits])
    _check("spw_spmv_group", lib().spw_spmv_group(
        n, harr, P(*[b.data_ptr() for b in bufs]), P(*[t.data_ptr() for t, _ in x2]),
        I(*[ld for _, ld in x2]), ab, P(*[t.data_ptr() for t, _ in y2]), I(*[ld for _, ld in y2]),
        B, float(threshold), _ptr(ws), _nbytes(ws), _stream()))
    return ys


@_on_stream
def spw_spmv_noalloc(hdr, buf: torch.Tensor, x: torch.Tensor, threshold: float = 0.0,
                     act_bits: torch.Tensor | None = None, y: torch.Tensor | None = None) -> torch.Tensor:
    """Decode like spw_spmv, with the library's own fixed scratch instead of a workspace.

    For callers that cannot allocate device memory; see include/spw.h for the size
    limit and for why overlapping calls race."""
    h = _hdr(hdr)
    x2, ldx = _rows(_half(x, "x"), "x")
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, h.N), dtype=torch.float16, device=x.device)
    y2, ldy = _rows(_half(y, "y"), "y")
    _need_buf(buf, h)
    _need(x2, x2.shape[0], h.K, "x")
    _need(y2, x2.shape[0], h.N, "y")
    _need_words(act_bits, h.K)
    _check("spw_spmv_noalloc", lib().spw_spmv_noalloc(
        ctypes.byref(h), _ptr(buf), _ptr(x2), B, ldx, float(threshold), _ptr(act_bits),
        _ptr(y2), ldy, _stream()))
    return y


def spw_spmm_workspace_bytes(hdr, M: int) -> int:
    h = _hdr(hdr)
    return int(lib().spw_spmm_workspace_bytes(ctypes.byref(h), int(M)))


@_on_stream
def spw_spmm(hdr, buf: torch.Tensor, X: torch.Tensor, Y: torch.Tensor | None = None,
             ws: torch.Tensor | None = None) -> torch.Tensor:
    """Prefill Y (M x N fp16) = X . W_masked^T on tcgen05 tensor cores."""
    h = _hdr(hdr)
    X2, ldx = _rows(_half(X, "X"), "X")
    M = X2.shape[0]
    if Y is None:
        Y = torch.empty((M, h.N), dtype=torch.float16, device=X.device)
    Y2, ldy = _rows(_half(Y, "Y"), "Y")
    _need_buf(buf, h)
    _need(X2, M, h.K, "X")
    _need(Y2, M, h.N, "Y")
    need = spw_spmm_workspace_bytes(h, M)
    if ws is None and need:
        ws = torch.zeros(need, dtype=torch.uint8, device=X.device)
    _check("spw_spmm", lib().spw_spmm(
        ctypes.byref(h), _ptr(buf), _ptr(X2), M, ldx, _ptr(Y2), ldy, _ptr(ws),
        _nbytes(ws), _stream()))
    return Y


def spw_spmm_plan(hdr, M: int, sm_count: int = 0) -> dict:
    """The launch plan of spw_spmm for M tokens on sm_count SMs (0: the current device)."""
    info = spw_spmm_plan_info()
    _check("spw_spmm_plan", lib().spw_spmm_plan(ctypes.byref(_hdr(hdr)), int(M), int(sm_count),
                                                ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in info._fields_}


def spw_group_tokens_workspace_bytes(M: int, K: int) -> int:
    return int(lib().spw_group_tokens_workspace_bytes(int(M), int(K)))


@_on_stream
def spw_group_tokens(X: torch.Tensor, t: float, token_tile: int, ws: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Token grouping of X (M x K fp16): (Xg M x ceil8(K) fp16, perm int32[M], tile_sig
    int64[ceil(M / token_tile), words]); see spw_group_tokens in include/spw.h."""
    X2, ldx = _rows(_half(X, "X"), "X")
    M, K = X2.shape[0], X2.shape[1]
    words = ((K + 63) // 64 + 63) // 64
    ldg = (K + 7) // 8 * 8
    Xg = torch.empty((M, ldg), dtype=torch.float16, device=X.device)
    perm = torch.empty(M, dtype=torch.int32, device=X.device)
    tsig = torch.empty((-(-M // int(token_tile)), words), dtype=torch.int64, device=X.device)
    need = spw_group_tokens_workspace_bytes(M, K)
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=X.device)
    _check("spw_group_tokens", lib().spw_group_tokens(
        _ptr(X2), M, K, ldx, ctypes.c_float(t), int(token_tile), _ptr(Xg), ldg, _ptr(perm),
        _ptr(tsig), _ptr(ws), _nbytes(ws), _stream()))
    return Xg, perm, tsig


def spw_spmm_tokens_workspace_bytes(hdr, M: int) -> int:
    return int(lib().spw_spmm_tokens_workspace_bytes(ctypes.byref(_hdr(hdr)), int(M)))


def spw_spmm_tokens_plan(hdr, M: int, sm_count: int = 0) -> dict:
    """The launch plan of spw_spmm_tokens (its token tile is the grouping's T)."""
    info = spw_spmm_plan_info()
    _check("spw_spmm_tokens_plan", lib().spw_spmm_tokens_plan(
        ctypes.byref(_hdr(hdr)), int(M), int(sm_count), ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in info._fields_}


@_on_stream
def spw_spmm_tokens(hdr, buf: torch.Tensor, X: torch.Tensor, threshold: float,
                    Y: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Prefill with per-token index sets: Y = X~ . W_masked^T, tokens grouped by the
    k-tiles they use (see spw_spmm_tokens in include/spw.h).  ws: a uint8 workspace of
    spw_spmm_tokens_workspace_bytes(hdr, M) bytes whose first (split-K counter) bytes are
    zero; allocated zeroed here when omitted."""
    h = _hdr(hdr)
    X2, ldx = _rows(_half(X, "X"), "X")
    M = X2.shape[0]
    if Y is None:
        Y = torch.empty((M, h.N), dtype=torch.float16, device=X.device)
    Y2, ldy = _rows(_half(Y, "Y"), "Y")
    _need_buf(buf, h)
    _need(X2, M, h.K, "X")
    _need(Y2, M, h.N, "Y")
    if ws is None:
        ws = torch.zeros(max(spw_spmm_tokens_workspace_bytes(h, M), 16), dtype=torch.uint8,
                         device=X.device)
    _check("spw_spmm_tokens", lib().spw_spmm_tokens(
        ctypes.byref(h), _ptr(buf), _ptr(X2), M, ldx, ctypes.c_float(threshold), _ptr(Y2), ldy,
        _ptr(ws), _nbytes(ws), _stream()))
    return Y


def spw_spmv_tc_workspace_bytes(hdr, B: int) -> int:
    h = _hdr(hdr)
    return int(lib().spw_spmv_tc_workspace_bytes(ctypes.byref(h), int(B)))


@_on_stream
def spw_spmv_tc(hdr, buf: torch.Tensor, x: torch.Tensor, threshold: float = 0.0,
                act_bits: torch.Tensor | None = None, y: torch.Tensor | None = None,
                ws: torch.Tensor | None = None) -> torch.Tensor:
    """Decode y (B x N fp16) on tensor cores; arguments as spw_spmv.  ws: a zero-initialised
    uint8 workspace of spw_spmv_tc_workspace_bytes(hdr, B) bytes (allocated here when
    needed and not given)."""
    h = _hdr(hdr)
    x2, ldx = _rows(_half(x, "x"), "x")
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, h.N), dtype=torch.float16, device=x.device)
    y2, ldy = _rows(_half(y, "y"), "y")
    _need_buf(buf, h)
    _need(x2, B, h.K, "x")
    _need(y2, B, h.N, "y")
    _need_words(act_bits, h.K)
    need = spw_spmv_tc_workspace_bytes(h, B)
    if ws is None and need:
        ws = torch.zeros(need, dtype=torch.uint8, device=x.device)
    _check("spw_spmv_tc", lib().spw_spmv_tc(
        ctypes.byref(h), _ptr(buf), _ptr(x2), B, ldx, float(threshold), _ptr(act_bits),
        _ptr(y2), ldy, _ptr(ws), _nbytes(ws), _stream()))
    return y


def spw_spmv_auto_path(B: int) -> int:
    """0 when spw_spmv_auto takes the CUDA-core decode for batch B, 1 for the tensor-core
    decode, -1 for B outside 1..16."""
    return int(lib().spw_spmv_auto_path(int(B)))


def spw_spmv_auto_workspace_bytes(hdr, B: int) -> int:
    h = _hdr(hdr)
    return int(lib().spw_spmv_auto_workspace_bytes(ctypes.byref(h), int(B)))


@_on_stream
def spw_spmv_auto(hdr, buf: torch.Tensor, x: torch.Tensor, threshold: float = 0.0,
                  act_bits: torch.Tensor | None = None, y: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None) -> torch.Tensor:
    """Decode y (B x N fp16) on the path chosen by batch size; arguments as spw_spmv.  ws:
    a zero-initialised uint8 workspace of spw_spmv_auto_workspace_bytes(hdr, B) bytes
    (allocated here when needed and not given)."""
    h = _hdr(hdr)
    x2, ldx = _rows(_half(x, "x"), "x")
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, h.N), dtype=torch.float16, device=x.device)
    y2, ldy = _rows(_half(y, "y"), "y")
    _need_buf(buf, h)
    _need(x2, B, h.K, "x")
    _need(y2, B, h.N, "y")
    _need_words(act_bits, h.K)
    need = spw_spmv_auto_workspace_bytes(h, B)
    if ws is None and need:
        ws = torch.zeros(need, dtype=torch.uint8, device=x.device)
    _check("spw_spmv_auto", lib().spw_spmv_auto(
        ctypes.byref(h), _ptr(buf), _ptr(x2), B, ldx, float(threshold), _ptr(act_bits),
        _ptr(y2), ldy, _ptr(ws), _nbytes(ws), _stream()))
    return y


def spw_spmv_ffn_workspace_bytes(hdr_gate, hdr_up, B: int) -> int:
    return int(lib().spw_spmv_ffn_workspace_bytes(ctypes.byref(_hdr(hdr_gate)),
                                                  ctypes.byref(_hdr(hdr_up)), B))


@_on_stream
def spw_spmv_ffn(hdr_gate, buf_gate: torch.Tensor, hdr_up, buf_up: torch.Tensor, x: torch.Tensor,
                 threshold: float = 0.0, h: torch.Tensor | None = None,
                 act_bits: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Fused FFN activation: h (B x N fp16) = SiLU(W_gate x) * (W_up x) and the column-set
    words of h under the threshold rule, in one launch.  ws: a zero-initialised uint8
    workspace of spw_spmv_ffn_workspace_bytes(hdr_gate, hdr_up, B) bytes (allocated here
    when not given).  Returns (h, act_bits)."""
    hg, hu = _hdr(hdr_gate), _hdr(hdr_up)
    x2, ldx = _rows(_half(x, "x"), "x")
    B = x2.shape[0]
    if h is None:
        h = torch.empty((B, hg.N), dtype=torch.float16, device=x.device)
    h2, ldh = _rows(_half(h, "h"), "h")
    _need_buf(buf_gate, hg, "buf_gate")
    _need_buf(buf_up, hu, "buf_up")
    _need(x2, B, hg.K, "x")
    _need(h2, B, hg.N, "h")
    if act_bits is None:
        act_bits = torch.empty(((hg.N + 31) // 32,), dtype=torch.int32, device=x.device)
    _need_words(act_bits, hg.N)
    if ws is None:
        need = spw_spmv_ffn_workspace_bytes(hg, hu, B)
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=x.device)
    _check("spw_spmv_ffn", lib().spw_spmv_ffn(
        ctypes.byref(hg), _ptr(buf_gate), ctypes.byref(hu), _ptr(buf_up), _ptr(x2), B, ldx,
        float(threshold), _ptr(h2), ldh, _ptr(act_bits), _ptr(ws), _nbytes(ws), _stream()))
    return h, act_bits


_timeouts = 0  # timeouts reported so far: the holders' workspaces from before the last are void


def spw_last_device_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the device status word (see include/spw.h).
    After SPW_ERR_TIMEOUT the split counters of a decode workspace are undefined: the holders below
    replace theirs at their next call; a caller's own has to be zeroed."""
    global _timeouts
    code = ctypes.c_int()
    _check("spw_last_device_status", lib().spw_last_device_status(_stream(stream),
                                                                  ctypes.byref(code)))
    if code.value == SPW_ERR_TIMEOUT:
        _timeouts += 1
    return code.value


class DecodeGroup:
    """A prepared spw_spmv_group call for a fixed set of layers and batch size.

    The header array, weight pointers and workspace are built once; each call only
    refreshes the input and output pointers and leading dimensions, so the per-call host
    cost is one library call (serving loops that decode the same layers every step).  Its
    workspace `ws` is one for all calls: they must not overlap, and after a reported timeout
    it has to be zeroed."""

    def __init__(self, hdrs, bufs, B: int, ws: torch.Tensor | None = None):
        self.n = len(hdrs)
        if self.n != len(bufs):
            raise ValueError("one weight buffer per header")
        self.B = int(B)
        self._harr = _hdr_array(hdrs)
        for i, h in enumerate(self._harr):
            _need_buf(bufs[i], h, f"bufs[{i}]")
        self._K = [int(h.K) for h in self._harr]
        self._N = [int(h.N) for h in self._harr]
        self._bufs = list(bufs)  # keeps the weights alive
        P = ctypes.c_void_p * self.n
        I = ctypes.c_int * self.n
        self._pbufs = P(*[b.data_ptr() for b in bufs])
        self._px, self._py, self._pab = P(), P(), P()
        self._ldx, self._ldy = I(), I()
        if ws is None:
            need = spw_spmv_group_workspace_bytes(self._harr, self.B)
            ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=bufs[0].device)
        self.ws = ws

    def __call__(self, xs, ys, threshold: float = 0.0, act_bits=None, stream=None):
        """Decode into ys (one B x N_l fp16 tensor per layer) from xs (B x K_l each)."""
        if len(xs) != self.n or len(ys) != self.n:
            raise ValueError(f"expected {self.n} inputs and outputs")
        for i in range(self.n):
            x, y = xs[i], ys[i]
            if x.dtype != torch.float16 or y.dtype != torch.float16:
                raise TypeError("inputs and outputs must be float16")
            if not (x.is_cuda and y.is_cuda):
                raise ValueError("inputs and outputs must be CUDA tensors")
            xr = x.shape[0] if x.dim() == 2 else 1
            yr = y.shape[0] if y.dim() == 2 else 1
            if xr < self.B or x.shape[-1] < self._K[i] or yr < self.B or y.shape[-1] < self._N[i]:
                raise ValueError(f"layer {i}: x needs {self.B} x {self._K[i]}, y {self.B} x {self._N[i]}")
            self._px[i] = x.data_ptr()
            self._ldx[i] = x.stride(0) if x.dim() == 2 and x.shape[0] > 1 else x.shape[-1]
            self._py[i] = y.data_ptr()
            self._ldy[i] = y.stride(0) if y.dim() == 2 and y.shape[0] > 1 else y.shape[-1]
        ab = None
        if act_bits is not None:
            for i in range(self.n):
                _need_words(act_bits[i], self._K[i], f"act_bits[{i}]")
                self._pab[i] = None if act_bits[i] is None else act_bits[i].data_ptr()
            ab = self._pab
        _check("spw_spmv_group", lib().spw_spmv_group(
            self.n, self._harr, self._pbufs, self._px, self._ldx, ab, self._py, self._ldy,
            self.B, float(threshold), _ptr(self.ws), _nbytes(self.ws), _stream(stream)))
        return ys


def spw_s24_bytes(N: int, K: int) -> int:
    return int(lib().spw_s24_bytes(int(N), int(K)))


@_on_stream
def spw_split24(W: torch.Tensor, mask: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """2:4 + residual split: (s24 uint8 buffer of the 2:4 part, residual mask uint8 N x K);
    see spw_split24 in include/spw.h."""
    W2, ldw = _rows(_half(W, "W"), "W")
    N, K = W2.shape
    m2, ldm = _mask_like(mask, N, K)
    s24 = torch.empty(spw_s24_bytes(N, K), dtype=torch.uint8, device=W.device)
    mask_r = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    _check("spw_split24", lib().spw_split24(_ptr(W2), ldw, _ptr(m2), ldm, N, K, _ptr(s24), _nbytes(s24, "s24"),
                                            _ptr(mask_r), K, _stream()))
    return s24, mask_r


def spw_spmm24_workspace_bytes(hdr_r, M: int) -> int:
    return int(lib().spw_spmm24_workspace_bytes(ctypes.byref(_hdr(hdr_r)), int(M)))


def spw_spmm24_plan(hdr_r, M: int, sm_count: int = 0) -> dict:
    info = spw_spmm_plan_info()
    _check("spw_spmm24_plan", lib().spw_spmm24_plan(ctypes.byref(_hdr(hdr_r)), int(M), int(sm_count),
                                                    ctypes.byref(info)))
    return {name: getattr(info, name) for name, _ in info._fields_}


@_on_stream
def spw_spmm24(hdr_r, buf_r: torch.Tensor, s24: torch.Tensor, X: torch.Tensor,
               Y: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Prefill on the 2:4 + residual split: Y = X . (S + R)^T, S on sparse tensor cores."""
    h = _hdr(hdr_r)
    X2, ldx = _rows(_half(X, "X"), "X")
    M = X2.shape[0]
    if Y is None:
        Y = torch.empty((M, h.N), dtype=torch.float16, device=X.device)
    Y2, ldy = _rows(_half(Y, "Y"), "Y")
    _need_buf(buf_r, h, "buf_r")
    _need(X2, M, h.K, "X")
    _need(Y2, M, h.N, "Y")
    need = spw_spmm24_workspace_bytes(h, M)
    if ws is None and need:
        ws = torch.zeros(need, dtype=torch.uint8, device=X.device)
    _check("spw_spmm24", lib().spw_spmm24(
        ctypes.byref(h), _ptr(buf_r), _ptr(s24), _nbytes(s24, "s24"), _ptr(X2), M, ldx, _ptr(Y2), ldy,
        _ptr(ws), _nbytes(ws), _stream()))
    return Y


# ------------------------------------------------------------------ epilogues, gated block, gradients

def _act(act) -> int:
    """An activation's number from its number or name."""
    if isinstance(act, str):
        if act not in ACTIVATIONS:
            raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}")
        return ACTIVATIONS[act]
    return int(act)


def _same_device(*tensors):
    """The library works on the current device: every tensor has to live there."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}; the current CUDA "
                             f"device is cuda:{dev}")


def _whole(names: str, *tensors):
    """Raw buffers go over as a pointer and a number of bytes, so a tensor with gaps or repeats
    (whose storage holds other or fewer bytes than its size says) cannot."""
    for t in tensors:
        if t is not None and not t.is_contiguous():
            name = names.split()[[u is t for u in tensors].index(True)]
            raise ValueError(f"{name} must be contiguous")


def _mat(t: torch.Tensor, rows: int | None, cols: int, name: str) -> tuple[torch.Tensor, int, int]:
    """An fp16 operand of exactly rows x cols (any number of rows for None), unit column
    stride: (2-D view, rows, leading dimension)."""
    if t.dtype is not torch.float16:
        t = _half(t, name)
    if t.dim() == 1:
        t = t.unsqueeze(0)
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    m, n = t.shape
    if n != cols or (rows is not None and m != rows):
        raise ValueError(f"{name} is {m} x {n}; the call takes {'any' if rows is None else rows} rows of "
                         f"{cols} columns")
    return t, m, _ld(t.stride(0), m, n, name)


def _out(t: torch.Tensor | None, rows: int, cols: int, like: torch.Tensor, name: str):
    """An fp16 output of at least rows x cols (allocated when not given): (tensor, address, ld)."""
    if t is None:
        t = torch.empty_strided((rows, cols), (cols, 1), dtype=torch.float16, device=like.device)
        return t, t.data_ptr(), cols
    v, ld = _rows(_half(t, name), name)
    _need(v, rows, cols, name)
    return t, v.data_ptr(), ld


def _values_len(h) -> int:
    return (h.bytes_total - h.off_values) // 2


def _packed(t: torch.Tensor | None, h, buf: torch.Tensor, name: str) -> tuple[torch.Tensor, int]:
    """A packed gradient, one fp16 entry for each entry of the values section, and its address.
    (That of a weight with nothing kept is empty, and an empty tensor has no address: the
    weight's buffer stands for it; nothing is written there.)"""
    n = _values_len(h)
    if t is None:
        t = torch.empty_strided((n,), (1,), dtype=torch.float16, device=buf.device)
    else:
        t = _half(t, name)
        if t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1) or t.numel() < n:
            raise ValueError(f"{name} must be 1-D and contiguous with at least {n} entries")
    return t, t.data_ptr() if t.numel() else buf.data_ptr()


def _ws_of(ws: torch.Tensor | None, need: int, like: torch.Tensor):
    """The caller's workspace, or one of `need` bytes: (tensor, address, bytes)."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=like.device)
        return ws, ws.data_ptr(), need
    return ws, ws.data_ptr(), _nbytes(ws)


def _epilogue(bias, act, residual, rows: int, N: int) -> spw_epilogue:
    ep = spw_epilogue(None, None, 0, _act(act))
    if bias is not None:
        b = _half(bias, "bias")
        if b.dim() != 1 or b.numel() != N or (N > 1 and b.stride(0) != 1):
            raise ValueError(f"bias must be 1-D and contiguous with {N} entries, got {tuple(b.shape)}")
        ep.bias = b.data_ptr()
    if residual is not None:
        r, _, ep.ldr = _mat(residual, rows, N, "residual")
        ep.residual = r.data_ptr()
    return ep


def spw_spmv_ep_path(hdr, B: int) -> int:
    """0 when spw_spmv_ep takes the CUDA-core decode for this weight and batch, 1 for the tensor
    cores, -1 for B outside 1..16."""
    return int(lib().spw_spmv_ep_path(ctypes.byref(_hdr(hdr)), int(B)))


def spw_spmv_ep_workspace_bytes(hdr, B: int) -> int:
    return int(lib().spw_spmv_ep_workspace_bytes(ctypes.byref(_hdr(hdr)), int(B)))


@_on_stream
def spw_spmv_ep(hdr, buf: torch.Tensor, x: torch.Tensor, threshold: float = 0.0,
                act_bits: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                act=SPW_ACT_NONE, residual: torch.Tensor | None = None,
                y: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Decode with an epilogue: y = act(W_masked . x~ + bias) + residual (B x N fp16, B <= 16).

    bias: N fp16; residual: B x N fp16 (it may be y itself); act: a name of ACTIVATIONS or its
    number; the rest as spw_spmv.  ws: a zero-initialised uint8 workspace of
    spw_spmv_ep_workspace_bytes(hdr, B) bytes (allocated here when needed and not given)."""
    h = _hdr(hdr)
    x2, B, ldx = _mat(x, None, h.K, "x")
    _same_device(x, buf, act_bits, bias, residual, y, ws)
    _whole("buf act_bits ws", buf, act_bits, ws)
    ep = _epilogue(bias, act, residual, B, h.N)
    _need_buf(buf, h)
    _need_words(act_bits, h.K)
    y, py, ldy = _out(y, B, h.N, x, "y")
    if ws is None:
        need = spw_spmv_ep_workspace_bytes(h, B)
        ws = torch.zeros(need, dtype=torch.uint8, device=x.device) if need else None
    pws, nws = (None, 0) if ws is None else (ws.data_ptr(), _nbytes(ws))
    _check("spw_spmv_ep", lib().spw_spmv_ep(
        ctypes.byref(h), buf.data_ptr(), x2.data_ptr(), B, ldx, float(threshold), _ptr(act_bits),
        ctypes.byref(ep), py, ldy, pws, nws, _stream()))
    return y


def spw_spmm_ep_workspace_bytes(hdr, M: int) -> int:
    return int(lib().spw_spmm_ep_workspace_bytes(ctypes.byref(_hdr(hdr)), int(M)))


@_on_stream
def spw_spmm_ep(hdr, buf: torch.Tensor, X: torch.Tensor, bias: torch.Tensor | None = None,
                act=SPW_ACT_NONE, residual: torch.Tensor | None = None,
                Y: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Prefill with an epilogue: Y = act(X . W_masked^T + bias) + residual (M x N fp16).

    bias, act and residual as spw_spmv_ep.  ws: spw_spmm_ep_workspace_bytes(hdr, M) bytes of
    any content (allocated here when not given)."""
    h = _hdr(hdr)
    X2, M, ldx = _mat(X, None, h.K, "X")
    _same_device(X, buf, bias, residual, Y, ws)
    _whole("buf ws", buf, ws)
    ep = _epilogue(bias, act, residual, M, h.N)
    _need_buf(buf, h)
    Y, pY, ldy = _out(Y, M, h.N, X, "Y")
    ws, pws, nws = _ws_of(ws, spw_spmm_ep_workspace_bytes(h, M), X)
    _check("spw_spmm_ep", lib().spw_spmm_ep(
        ctypes.byref(h), buf.data_ptr(), X2.data_ptr(), M, ldx, ctypes.byref(ep), pY, ldy, pws, nws,
        _stream()))
    return Y


def spw_spmm_ffn_workspace_bytes(hdr_gate, hdr_up, M: int) -> int:
    return int(lib().spw_spmm_ffn_workspace_bytes(ctypes.byref(_hdr(hdr_gate)),
                                                  ctypes.byref(_hdr(hdr_up)), int(M)))


@_on_stream
def spw_spmm_ffn(hdr_gate, buf_gate: torch.Tensor, hdr_up, buf_up: torch.Tensor, X: torch.Tensor,
                 act=SPW_ACT_SILU, save: bool = False, H: torch.Tensor | None = None,
                 G: torch.Tensor | None = None, U: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None):
    """Prefill of the gated block in one kernel: H = act(X . W_gate^T) * (X . W_up^T), M x N.

    Returns H, or (H, G, U) with the two projections when save is set or G and U are given
    (what spw_spmm_ffn_backward takes).  ws: spw_spmm_ffn_workspace_bytes(...) bytes."""
    hg, hu = _hdr(hdr_gate), _hdr(hdr_up)
    X2, M, ldx = _mat(X, None, hg.K, "X")
    if (G is None) != (U is None):
        raise ValueError("G and U go together")
    save = save or G is not None
    _same_device(X, buf_gate, buf_up, H, G, U, ws)
    _whole("buf_gate buf_up ws", buf_gate, buf_up, ws)
    _need_buf(buf_gate, hg, "buf_gate")
    _need_buf(buf_up, hu, "buf_up")
    H, pH, ldh = _out(H, M, hg.N, X, "H")
    pG = pU = None
    ldg = ldu = 0
    if save:
        G, pG, ldg = _out(G, M, hg.N, X, "G")
        U, pU, ldu = _out(U, M, hg.N, X, "U")
    ws, pws, nws = _ws_of(ws, spw_spmm_ffn_workspace_bytes(hg, hu, M), X)
    _check("spw_spmm_ffn", lib().spw_spmm_ffn(
        ctypes.byref(hg), buf_gate.data_ptr(), ctypes.byref(hu), buf_up.data_ptr(), X2.data_ptr(), M, ldx, _act(act),
        pH, ldh, pG, ldg, pU, ldu, pws, nws, _stream()))
    return (H, G, U) if save else H


def spw_spmm_ffn_backward_workspace_bytes(hdr_gate, hdr_up, M: int) -> int:
    return int(lib().spw_spmm_ffn_backward_workspace_bytes(
        ctypes.byref(_hdr(hdr_gate)), ctypes.byref(_hdr(hdr_up)), int(M)))


@_on_stream
def spw_spmm_ffn_backward(hdr_gate, buf_gate: torch.Tensor, hdr_up, buf_up: torch.Tensor,
                          X: torch.Tensor | None, G: torch.Tensor, U: torch.Tensor, dH: torch.Tensor,
                          act=SPW_ACT_SILU, need_dx: bool = True, need_dv: bool = True,
                          dX: torch.Tensor | None = None, dV_gate: torch.Tensor | None = None,
                          dV_up: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Gradients of spw_spmm_ffn, the patterns held fixed: (dX, dV_gate, dV_up).

    dV_*: the kept weights' gradients in the order of the buffers' values sections (1-D fp16).
    need_dx / need_dv False leaves that part out (None in its place; X may then be None for
    need_dv False).  ws: spw_spmm_ffn_backward_workspace_bytes(...) bytes."""
    hg, hu = _hdr(hdr_gate), _hdr(hdr_up)
    G2, M, ldg = _mat(G, None, hg.N, "G")
    U2, _, ldu = _mat(U, M, hg.N, "U")
    dH2, _, lddh = _mat(dH, M, hg.N, "dH")
    if need_dv and X is None:
        raise ValueError("the weights' gradients need X")
    pX, ldx = None, 0
    if X is not None:
        X2, _, ldx = _mat(X, M, hg.K, "X")
        pX = X2.data_ptr()
    _same_device(G, U, dH, X, buf_gate, buf_up, dX, dV_gate, dV_up, ws)
    _whole("buf_gate buf_up ws", buf_gate, buf_up, ws)
    _need_buf(buf_gate, hg, "buf_gate")
    _need_buf(buf_up, hu, "buf_up")
    pdX, lddx = None, 0
    if need_dx:
        dX, pdX, lddx = _out(dX, M, hg.K, G, "dX")
    else:
        dX = None
    dV_gate, pVg = _packed(dV_gate, hg, buf_gate, "dV_gate") if need_dv else (None, None)
    dV_up, pVu = _packed(dV_up, hu, buf_up, "dV_up") if need_dv else (None, None)
    ws, pws, nws = _ws_of(ws, spw_spmm_ffn_backward_workspace_bytes(hg, hu, M), G)
    _check("spw_spmm_ffn_backward", lib().spw_spmm_ffn_backward(
        ctypes.byref(hg), buf_gate.data_ptr(), ctypes.byref(hu), buf_up.data_ptr(), pX, M, ldx, _act(act),
        G2.data_ptr(), ldg, U2.data_ptr(), ldu, dH2.data_ptr(), lddh, pdX, lddx, pVg,
        pVu, pws, nws, _stream()))
    return dX, dV_gate, dV_up


def spw_spmm_backward_workspace_bytes(hdr, M: int) -> int:
    return int(lib().spw_spmm_backward_workspace_bytes(ctypes.byref(_hdr(hdr)), int(M)))


@_on_stream
def spw_spmm_backward(hdr, buf: torch.Tensor, X: torch.Tensor | None, dY: torch.Tensor,
                      need_dx: bool = True, need_dv: bool = True, dX: torch.Tensor | None = None,
                      dV: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Gradients of Y = X . W_masked^T, the pattern held fixed: (dX, dV); dV, need_* and X as
    spw_spmm_ffn_backward.  ws: spw_spmm_backward_workspace_bytes(hdr, M) bytes."""
    h = _hdr(hdr)
    dY2, M, lddy = _mat(dY, None, h.N, "dY")
    if need_dv and X is None:
        raise ValueError("the weight's gradient needs X")
    pX, ldx = None, 0
    if X is not None:
        X2, _, ldx = _mat(X, M, h.K, "X")
        pX = X2.data_ptr()
    _same_device(dY, X, buf, dX, dV, ws)
    _whole("buf ws", buf, ws)
    _need_buf(buf, h)
    pdX, lddx = None, 0
    if need_dx:
        dX, pdX, lddx = _out(dX, M, h.K, dY, "dX")
    else:
        dX = None
    dV, pV = _packed(dV, h, buf, "dV") if need_dv else (None, None)
    ws, pws, nws = _ws_of(ws, spw_spmm_backward_workspace_bytes(h, M), dY)
    _check("spw_spmm_backward", lib().spw_spmm_backward(
        ctypes.byref(h), buf.data_ptr(), pX, M, ldx, dY2.data_ptr(), lddy, pdX, lddx,
        pV, pws, nws, _stream()))
    return dX, dV


class _Workspaces:
    """A holder's zeroed decode workspaces: one for each kind of call, batch and stream, so that
    calls on two streams can overlap.  A captured call gets its own (cleared by the graph): one
    that the graph shared with eager calls or with another graph would be in use twice when they
    run at once, and before the first replay it would not be cleared.  After a reported timeout,
    which leaves counters undefined, all are made anew."""

    def __init__(self, device):
        self._device, self._held, self._timeouts = device, {}, _timeouts

    def get(self, kind: str, B: int, size) -> torch.Tensor | None:
        """For a call on the current stream; size() gives the bytes (None for 0)."""
        if torch.cuda.is_current_stream_capturing():
            return self._new(size())
        if self._timeouts != _timeouts:
            self._held, self._timeouts = {}, _timeouts
        key = kind, B, _stream().value
        if key not in self._held:
            self._held[key] = self._new(size())
        return self._held[key]

    def _new(self, need: int):
        return torch.zeros(need, dtype=torch.uint8, device=self._device) if need else None


class SparseLinear24:
    """A weight held as its 2:4 part (sparse tensor cores) plus a TCB residual: a holder
    for spw_split24, spw_compress and spw_spmm24 (it adds no arithmetic)."""

    def __init__(self, W: torch.Tensor, mask: torch.Tensor, stream=None):
        self.N, self.K = W.shape
        self.s24, self.mask_r = spw_split24(W, mask, stream)
        self.buf_r, self.hdr_r = spw_compress(W, self.mask_r, stream=stream)

    def spmm(self, X, Y=None, ws=None, stream=None):
        return spw_spmm24(self.hdr_r, self.buf_r, self.s24, X, Y, ws, stream)


class SparseLinear:
    """A compressed weight with its header and decode workspaces (a holder for the calls above;
    it adds no arithmetic)."""

    def __init__(self, W: torch.Tensor, mask: torch.Tensor, stream=None):
        self.N, self.K = W.shape
        self.buf, self.hdr = spw_compress(W, mask, stream=stream)
        self._ws = {}
        self._workspaces = _Workspaces(self.buf.device)

    def workspace(self, B: int) -> torch.Tensor:
        """A workspace of spw_spmv for this batch, for callers that pass their own (the methods
        below hold others)."""
        if B not in self._ws:
            self._ws[B] = torch.zeros(max(spw_spmv_workspace_bytes(self.hdr, B), 16),
                                      dtype=torch.uint8, device=self.buf.device)
        return self._ws[B]

    @_on_stream
    def spmv(self, x, threshold=0.0, act_bits=None, y=None):
        x2 = x if x.dim() == 2 else x.unsqueeze(0)
        B = x2.shape[0]
        ws = self._workspaces.get("spmv", B, lambda: max(spw_spmv_workspace_bytes(self.hdr, B), 16))
        return spw_spmv(self.hdr, self.buf, x2, threshold, act_bits, y, ws)

    @_on_stream
    def spmv_auto(self, x, threshold=0.0, act_bits=None, y=None):
        x2 = x if x.dim() == 2 else x.unsqueeze(0)
        B = x2.shape[0]
        ws = self._workspaces.get("auto", B, lambda: max(spw_spmv_auto_workspace_bytes(self.hdr, B), 16))
        return spw_spmv_auto(self.hdr, self.buf, x2, threshold, act_bits, y, ws)

    def spmm(self, X, Y=None, stream=None):
        return spw_spmm(self.hdr, self.buf, X, Y, stream=stream)

    def spmm_tokens(self, X, threshold=0.0, Y=None, ws=None, stream=None):
        return spw_spmm_tokens(self.hdr, self.buf, X, threshold, Y, ws, stream=stream)

    @_on_stream
    def spmv_ep(self, x, threshold=0.0, act_bits=None, bias=None, act=SPW_ACT_NONE, residual=None,
                y=None):
        x2 = x if x.dim() == 2 else x.unsqueeze(0)
        B = x2.shape[0]
        ws = self._workspaces.get("ep", B, lambda: spw_spmv_ep_workspace_bytes(self.hdr, B))
        return spw_spmv_ep(self.hdr, self.buf, x2, threshold, act_bits, bias, act, residual, y, ws)

    def spmm_ep(self, X, bias=None, act=SPW_ACT_NONE, residual=None, Y=None, ws=None, stream=None):
        return spw_spmm_ep(self.hdr, self.buf, X, bias, act, residual, Y, ws, stream=stream)

    def spmm_backward(self, X, dY, need_dx=True, need_dv=True, ws=None, stream=None):
        return spw_spmm_backward(self.hdr, self.buf, X, dY, need_dx, need_dv, ws=ws, stream=stream)

    def values(self) -> torch.Tensor:
        """The kept weights as they stand in the buffer (fp16 view of the values section, the
        order of a packed gradient; a tile's filling must stay zero).  With launch overlap on
        (spw_set_launch_overlap) a kernel other than a decode, or a synchronisation, has to come
        between one that writes here and a decode of this layer."""
        return self.buf[self.hdr.off_values:self.hdr.bytes_total].view(torch.float16)

    def decompress(self, out=None, stream=None):
        return spw_decompress(self.hdr, self.buf, out, stream)


class SparseFFN:
    """The gate and up projections of a gated block with its activation (a holder for the
    calls above; it adds no arithmetic): spmv for 1 to 16 tokens, spmm for more, backward."""

    def __init__(self, gate: SparseLinear, up: SparseLinear, act=SPW_ACT_SILU):
        if (gate.N, gate.K) != (up.N, up.K):
            raise ValueError(f"gate is {gate.N} x {gate.K}, up {up.N} x {up.K}")
        self.gate, self.up, self.act = gate, up, _act(act)
        self._workspaces = _Workspaces(gate.buf.device)

    @_on_stream
    def spmv(self, x, threshold=0.0, h=None, act_bits=None):
        """(h, column-set words) of the decode's fused step (SiLU only)."""
        if self.act != SPW_ACT_SILU:
            raise ValueError("the decode form computes SiLU")
        x2 = x if x.dim() == 2 else x.unsqueeze(0)
        B = x2.shape[0]
        ws = self._workspaces.get("ffn", B, lambda: max(spw_spmv_ffn_workspace_bytes(self.gate.hdr, self.up.hdr, B), 16))
        return spw_spmv_ffn(self.gate.hdr, self.gate.buf, self.up.hdr, self.up.buf, x2, threshold, h,
                            act_bits, ws)

    def spmm(self, X, save=False, H=None, G=None, U=None, ws=None, stream=None):
        return spw_spmm_ffn(self.gate.hdr, self.gate.buf, self.up.hdr, self.up.buf, X, self.act, save,
                            H, G, U, ws, stream=stream)

    def backward(self, X, G, U, dH, need_dx=True, need_dv=True, ws=None, stream=None):
        return spw_spmm_ffn_backward(self.gate.hdr, self.gate.buf, self.up.hdr, self.up.buf, X, G, U, dH,
                                     self.act, need_dx, need_dv, ws=ws, stream=stream)
