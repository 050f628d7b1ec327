"""ctypes binding of libmx.so (include/mx.h): argument marshalling only.

Every step of the MX path runs in the library's HIP kernels; torch only
provides device memory and the current HIP stream.  Importing this module
without a built library raises immediately: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmx.so")

E4M3, E5M2, E2M3, E3M2, E2M1, INT8 = range(6)
FMT_NAMES = ("e4m3", "e5m2", "e2m3", "e3m2", "e2m1", "int8")
FORMATS = {"e4m3": E4M3, "e5m2": E5M2, "e2m3": E2M3, "e3m2": E3M2, "e2m1": E2M1, "int8": INT8}
BITS = {E4M3: 8, E5M2: 8, E2M3: 6, E3M2: 6, E2M1: 4, INT8: 8}
SRC_F32, SRC_BF16 = 0, 1
RNE, SR = 0, 1
LAYOUT_ROW, LAYOUT_COLT = 1, 2
FLAG_HADAMARD32 = 1
MX_OK, MX_ERR_ARG, MX_ERR_SHAPE, MX_ERR_ALIGN, MX_ERR_UNSUPPORTED, MX_ERR_HIP = 0, -1, -2, -3, -4, -5


class QuantParams(ctypes.Structure):
    _fields_ = [("src", ctypes.c_int32), ("fmt", ctypes.c_int32), ("layouts", ctypes.c_uint32),
                ("round", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("hadamard_signs", ctypes.c_uint32), ("seed", ctypes.c_uint64),
                ("counter_offset", ctypes.c_uint64)]


class Cache(ctypes.Structure):
    _fields_ = [("k_q", ctypes.c_void_p), ("k_s", ctypes.c_void_p), ("v_q", ctypes.c_void_p),
                ("v_s", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("dim", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class MXError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)} ({status})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run microscaling_block_scaled_amd.build")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.mx_quantize.restype = ctypes.c_int
    lib.mx_quantize.argtypes = [P, i64, i64, i64, ctypes.POINTER(QuantParams), P, P, P, P, P]
    lib.mx_dequantize.restype = ctypes.c_int
    lib.mx_dequantize.argtypes = [P, P, i32, i64, i64, P, P]
    lib.mx_gemm.restype = ctypes.c_int
    lib.mx_gemm.argtypes = [P, P, i32, P, P, i32, i64, i64, i64, P, i64, P]
    lib.mx_gemm_bf16.restype = ctypes.c_int
    lib.mx_gemm_bf16.argtypes = [P, P, i32, P, P, i32, i64, i64, i64, P, i64, P]
    lib.mx_gemm_mx.restype = ctypes.c_int
    lib.mx_gemm_mx.argtypes = [P, P, i32, P, P, i32, i64, i64, i64, i32, P, P, P]
    f32 = ctypes.c_float
    lib.mx_rmsnorm_quantize.restype = ctypes.c_int
    lib.mx_rmsnorm_quantize.argtypes = [P, i64, P, i64, P, i64, i64, i32, i32, f32, P, i64, P, i64, P, P, P, P]
    lib.mx_rmsnorm_backward.restype = ctypes.c_int
    lib.mx_rmsnorm_backward.argtypes = [P, i64, P, i64, P, P, P, i64, i64, i64, i32, P, i64, P, P, i64, P]
    lib.mx_rmsnorm_backward_workspace.restype = i64
    lib.mx_rmsnorm_backward_workspace.argtypes = [i64, i64, i32]
    for gemv_ in (lib.mx_gemv, lib.mx_gemv_bf16):
        gemv_.restype = ctypes.c_int
        gemv_.argtypes = [P, i64, P, P, i32, i64, i64, i64, P, i64, P]
    lib.mx_cache_write.restype = ctypes.c_int
    lib.mx_cache_write.argtypes = [ctypes.POINTER(Cache), P, i64, i64, P, i64, i64, i32, i64, P, P]
    lib.mx_attention.restype = ctypes.c_int
    lib.mx_attention.argtypes = [ctypes.POINTER(Cache), P, i64, P, i64, P, i64, i64, i64, f32, i64, P, i64, P, P,
                                 i64, P]
    lib.mx_attention_workspace.restype = i64
    lib.mx_attention_workspace.argtypes = [i64] * 6
    lib.mx_packed_bytes.restype = i64
    lib.mx_packed_bytes.argtypes = [i32, i64, i64]
    lib.mx_scale_bytes.restype = i64
    lib.mx_scale_bytes.argtypes = [i64, i64]
    lib.mx_status_str.restype = ctypes.c_char_p
    lib.mx_status_str.argtypes = [ctypes.c_int]
    lib.mx_version.restype = ctypes.c_char_p
    lib.mx_version.argtypes = []
    return lib


lib = _load()

# every symbol include/mx.h declares
EXPORTS = ("mx_quantize", "mx_dequantize", "mx_gemm", "mx_gemm_bf16", "mx_gemm_mx",
           "mx_rmsnorm_quantize", "mx_rmsnorm_backward", "mx_rmsnorm_backward_workspace", "mx_gemv",
           "mx_gemv_bf16", "mx_cache_write", "mx_attention", "mx_attention_workspace", "mx_packed_bytes", "mx_scale_bytes", "mx_status_str", "mx_version")


def status_str(status: int) -> str:
    return lib.mx_status_str(status).decode()


def version() -> str:
    return lib.mx_version().decode()


def packed_bytes(fmt: int, rows: int, cols: int) -> int:
    return int(lib.mx_packed_bytes(fmt, rows, cols))


def scale_bytes(rows: int, cols: int) -> int:
    return int(lib.mx_scale_bytes(rows, cols))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, what: str):
    if status != MX_OK:
        raise MXError(status, what)


def quantize(x: torch.Tensor, fmt: int, layouts: int = LAYOUT_ROW, round_mode: int = RNE,
             hadamard: bool = False, hadamard_signs: int = 0, seed: int = 0,
             counter_offset: int = 0, out: dict | None = None, stream=None) -> dict:
    """MX-quantize a 2-D fp32/bf16 device tensor.  Returns uint8 device tensors
    q_row [rows, packed cols], s_row [rows, blocks of cols] and/or q_colt [cols,
    packed rows], s_colt [cols, blocks of rows]; a short last block is padded
    with zeros to 32 elements.  ``out`` may supply them preallocated."""
    if x.dim() != 2 or x.dtype not in (torch.float32, torch.bfloat16) or not x.is_cuda:
        raise ValueError("x must be a 2-D fp32/bf16 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    rows, cols = x.shape
    src = SRC_F32 if x.dtype == torch.float32 else SRC_BF16
    o = dict(out or {})
    dev = x.device
    if layouts & LAYOUT_ROW and "q_row" not in o:
        o["q_row"] = torch.empty((rows, packed_bytes(fmt, 1, cols)), dtype=torch.uint8, device=dev)
        o["s_row"] = torch.empty((rows, scale_bytes(1, cols)), dtype=torch.uint8, device=dev)
    if layouts & LAYOUT_COLT and "q_colt" not in o:
        o["q_colt"] = torch.empty((cols, packed_bytes(fmt, 1, rows)), dtype=torch.uint8, device=dev)
        o["s_colt"] = torch.empty((cols, scale_bytes(1, rows)), dtype=torch.uint8, device=dev)
    p = QuantParams(src, fmt, layouts, round_mode, FLAG_HADAMARD32 if hadamard else 0,
                    hadamard_signs & 0xFFFFFFFF, seed, counter_offset)
    st = lib.mx_quantize(_ptr(x), rows, cols, x.stride(0), ctypes.byref(p),
                         _ptr(o.get("q_row")) if layouts & LAYOUT_ROW else None,
                         _ptr(o.get("s_row")) if layouts & LAYOUT_ROW else None,
                         _ptr(o.get("q_colt")) if layouts & LAYOUT_COLT else None,
                         _ptr(o.get("s_colt")) if layouts & LAYOUT_COLT else None,
                         _stream(stream))
    _check(st, "mx_quantize")
    return o


def dequantize(q: torch.Tensor, s: torch.Tensor, fmt: int, rows: int, cols: int,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    y = out if out is not None else torch.empty((rows, cols), dtype=torch.float32, device=q.device)
    _check(lib.mx_dequantize(_ptr(q), _ptr(s), fmt, rows, cols, _ptr(y), _stream(stream)),
           "mx_dequantize")
    return y


def gemm(a_q: torch.Tensor, a_s: torch.Tensor, a_fmt: int, b_q: torch.Tensor, b_s: torch.Tensor,
         b_fmt: int, M: int, N: int, K: int, c: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """C[M, N] fp32 = A[M, K] (row-wise MX) x B where B is given as B^T[N, K]
    (row-wise MX)."""
    if c is None:
        c = torch.empty((M, N), dtype=torch.float32, device=a_q.device)
    _check(lib.mx_gemm(_ptr(a_q), _ptr(a_s), a_fmt, _ptr(b_q), _ptr(b_s), b_fmt, M, N, K,
                       _ptr(c), c.stride(0), _stream(stream)), "mx_gemm")
    return c


def gemm_bf16(a_q: torch.Tensor, a_s: torch.Tensor, a_fmt: int, b_q: torch.Tensor,
              b_s: torch.Tensor, b_fmt: int, M: int, N: int, K: int,
              c: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``gemm`` with C rounded to bf16 (nearest even) in the kernel."""
    if c is None:
        c = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    if c.dtype != torch.bfloat16 or (c.dim() == 2 and c.shape[0] > 0 and c.stride(1) != 1):
        raise ValueError("c must be a bf16 tensor with unit column stride")
    _check(lib.mx_gemm_bf16(_ptr(a_q), _ptr(a_s), a_fmt, _ptr(b_q), _ptr(b_s), b_fmt, M, N, K,
                            _ptr(c), c.stride(0), _stream(stream)), "mx_gemm_bf16")
    return c


def gemm_mx(a_q: torch.Tensor, a_s: torch.Tensor, a_fmt: int, b_q: torch.Tensor,
            b_s: torch.Tensor, b_fmt: int, M: int, N: int, K: int, c_fmt: int,
            out: dict | None = None, stream=None) -> dict:
    """The product of ``gemm`` quantized row-wise (blocks of 32 along N, round to
    nearest even) into format ``c_fmt`` inside the GEMM.  Returns uint8 device
    tensors q_row [M, packed N] and s_row [M, blocks of N] (a short last block
    padded); ``out`` may supply them preallocated."""
    o = dict(out or {})
    dev = a_q.device
    if "q_row" not in o:
        o["q_row"] = torch.empty((M, packed_bytes(c_fmt, 1, N)), dtype=torch.uint8, device=dev)
        o["s_row"] = torch.empty((M, scale_bytes(1, N)), dtype=torch.uint8, device=dev)
    _check(lib.mx_gemm_mx(_ptr(a_q), _ptr(a_s), a_fmt, _ptr(b_q), _ptr(b_s), b_fmt, M, N, K,
                          c_fmt, _ptr(o["q_row"]), _ptr(o["s_row"]), _stream(stream)),
           "mx_gemm_mx")
    return o


# ---------------------------------------------------------------------------
# decoder-layer operators
# ---------------------------------------------------------------------------
_SRC = {torch.float32: SRC_F32, torch.bfloat16: SRC_BF16}


def _on(stream, t):
    """The HIP stream handle of a call whose first tensor is t, which must lie on
    the current device; and that device's number."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors must be on the current CUDA device, got {t.device}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream, dev


def _empty(dtype, device, stream, *shape):
    """A new tensor whose memory belongs to the stream that the call runs on.  (Sizes go
    to torch one by one: it takes a quarter longer over a tuple.)"""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _rows(t, shape, dtype, dev, what):
    """Checks a row-major matrix; its address and pitch.  The pitch of a single row
    says nothing: one that is allowed is given."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{what} must be a {tuple(shape)} {dtype} tensor on device {dev}")
    pitch, unit = t.stride()
    if unit != 1 and shape[1] > 1:
        raise ValueError(f"{what} must have unit column stride")
    return t.data_ptr(), pitch if shape[0] > 1 else -(-shape[1] // 8) * 8


def _flat(t, shape, dtype, dev, what):
    """Checks a contiguous tensor; its address."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} {dtype} tensor on device {dev}")
    return t.data_ptr()


def _out(o, name, shape, dtype, dev, device, stream):
    """The address of output `name`, a contiguous tensor: the caller's, or a new one."""
    t = o.get(name)
    if t is not None:
        return _flat(t, shape, dtype, dev, name)
    t = o[name] = _empty(dtype, device, stream, *shape)
    return t.data_ptr()


def _out_rows(o, name, shape, dtype, dev, device, stream):
    """The address and pitch of output `name`, a row-major matrix: the caller's, or a new
    one whose rows start on 16 bytes."""
    t = o.get(name)
    if t is not None:
        return _rows(t, shape, dtype, dev, name)
    rows, cols = shape
    per = 8 if dtype == torch.bfloat16 else 4
    pitch = -(-cols // per) * per
    t = _empty(dtype, device, stream, rows, pitch)
    o[name] = t if pitch == cols else t[:, :cols]
    return t.data_ptr(), pitch


def _work(t, dev):
    if t is None:
        return None, 0
    if t.dtype != torch.uint8 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on device {dev}")
    return t.data_ptr(), t.numel()


def rmsnorm_quantize(x: torch.Tensor, w: torch.Tensor, fmt: int, eps: float = 1e-5,
                     residual: torch.Tensor | None = None, want_y: bool = False,
                     out: dict | None = None, stream=None) -> dict:
    """Root-mean-square norm of h = x + residual (fp32 or bf16 rows) times w,
    quantized row-wise to MX.  Returns q_row and s_row as ``quantize`` does, rstd
    [rows] fp32 (NaN for rows of no columns), h where a residual is given, and y in
    x's type where ``want_y`` is set; ``out`` may supply any of them preallocated (h
    may be x or the residual)."""
    shape, dtype, device = x.shape, x.dtype, x.device
    if len(shape) != 2 or dtype not in _SRC or fmt not in BITS:
        raise ValueError("x must be a 2-D fp32/bf16 CUDA tensor, fmt a format")
    handle, dev = _on(stream, x)
    rows, cols = shape
    px, ld_x = _rows(x, shape, dtype, dev, "x")
    pr, ld_r = (None, 0) if residual is None else _rows(residual, shape, dtype, dev, "residual")
    pw = _flat(w, (cols,), dtype, dev, "w")
    o = dict(out) if out else {}
    nblk = (cols + 31) // 32
    packed = nblk * 4 * BITS[fmt]
    u8 = torch.uint8
    pq = _out(o, "q_row", (rows, packed), u8, dev, device, stream)
    ps = _out(o, "s_row", (rows, nblk), u8, dev, device, stream)
    prstd = _out(o, "rstd", (rows,), torch.float32, dev, device, stream)
    ph, ld_h = py, ld_y = None, 0
    if residual is not None or o.get("h") is not None:
        ph, ld_h = _out_rows(o, "h", shape, dtype, dev, device, stream)
    if want_y or o.get("y") is not None:
        py, ld_y = _out_rows(o, "y", shape, dtype, dev, device, stream)
    _check(lib.mx_rmsnorm_quantize(px, ld_x, pr, ld_r, pw, rows, cols, _SRC[dtype], fmt, eps, ph, ld_h, py, ld_y,
                                   pq, ps, prstd, handle),
           "mx_rmsnorm_quantize")
    if cols == 0 and rows > 0:  # the mean of nothing, which the library does not write
        with torch.cuda.stream(stream):
            o["rstd"].fill_(float("nan"))
    return o


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor,
                     dh: torch.Tensor | None = None, out: dict | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of ``rmsnorm_quantize`` for the gradient dy of y: dx, that of h
    (and so of x and the residual), in h's type, with dh, what reaches h another
    way, added; and dw in fp32.  ``out`` and ``workspace`` (a uint8 tensor) may
    be supplied."""
    shape, dtype, device = h.shape, h.dtype, h.device
    if len(shape) != 2 or dtype not in _SRC:
        raise ValueError("h must be a 2-D fp32/bf16 CUDA tensor")
    handle, dev = _on(stream, h)
    rows, cols = shape
    src = _SRC[dtype]
    pdy, ld_dy = _rows(dy, shape, dtype, dev, "dy")
    ph, ld_h = _rows(h, shape, dtype, dev, "h")
    pdh, ld_dh = (None, 0) if dh is None else _rows(dh, shape, dtype, dev, "dh")
    o = dict(out) if out else {}
    pdx, ld_dx = _out_rows(o, "dx", shape, dtype, dev, device, stream)
    pdw = _out(o, "dw", (cols,), torch.float32, dev, device, stream)
    if workspace is None:
        need = lib.mx_rmsnorm_backward_workspace(rows, cols, src)
        if need > 0:
            workspace = _empty(torch.uint8, device, stream, need)
    _check(lib.mx_rmsnorm_backward(pdy, ld_dy, ph, ld_h, _flat(w, (cols,), dtype, dev, "w"),
                                   _flat(rstd, (rows,), torch.float32, dev, "rstd"), pdh, ld_dh, rows, cols, src,
                                   pdx, ld_dx, pdw, *_work(workspace, dev), handle), "mx_rmsnorm_backward")
    return o


def _gemv(call, dtype, what, x, w_q, w_s, w_fmt, M, N, K, y, stream):
    handle, dev = _on(stream, x)
    if w_fmt not in BITS:
        raise ValueError("w_fmt must be a format")
    if x.shape != (M, K) or x.dtype != torch.bfloat16 or (K > 1 and x.stride(1) != 1):
        raise ValueError("x must be a bf16 [M, K] tensor with unit column stride")
    nblk = (K + 31) // 32
    pw = _flat(w_q, (N, nblk * 4 * BITS[w_fmt]), torch.uint8, dev, "w_q")
    ps = _flat(w_s, (N, nblk), torch.uint8, dev, "w_s")
    if y is None:
        y = _empty(dtype, x.device, stream, M, N)
        ld_y = N
    else:
        if y.shape != (M, N) or y.dtype != dtype or y.get_device() != dev or (N > 1 and y.stride(1) != 1):
            raise ValueError(f"y must be a {dtype} [M, N] tensor with unit column stride")
        ld_y = y.stride(0) if M > 1 else N
    _check(call(x.data_ptr(), x.stride(0) if M > 1 else K, pw, ps, w_fmt, M, N, K, y.data_ptr(), ld_y, handle), what)
    return y


def gemv(x: torch.Tensor, w_q: torch.Tensor, w_s: torch.Tensor, w_fmt: int, M: int, N: int, K: int,
         y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[M, N] fp32 = x[M, K] (bf16, a few tokens) x W^T for W [N, K] in 4-bit
    row-wise MX (E2M1)."""
    return _gemv(lib.mx_gemv, torch.float32, "mx_gemv", x, w_q, w_s, w_fmt, M, N, K, y, stream)


def gemv_bf16(x: torch.Tensor, w_q: torch.Tensor, w_s: torch.Tensor, w_fmt: int, M: int, N: int, K: int,
              y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``gemv`` with y rounded to bf16 (nearest even) in the kernel."""
    return _gemv(lib.mx_gemv_bf16, torch.bfloat16, "mx_gemv_bf16", x, w_q, w_s, w_fmt, M, N, K, y, stream)


def kv_cache(pages: int, heads: int, page: int, dim: int, device="cuda") -> dict:
    """A new paged 8-bit MX key/value cache: uint8 tensors k_q, v_q [pages, heads,
    page, dim] and k_s, v_s [pages, heads, page, dim / 32]."""
    e = lambda n: torch.zeros((pages, heads, page, n), dtype=torch.uint8, device=device)
    return {"k_q": e(dim), "k_s": e(dim // 32), "v_q": e(dim), "v_s": e(dim // 32)}


def _cache(c, fmt, dev):
    kq, u8 = c["k_q"], torch.uint8
    if kq.dim() != 4:
        raise ValueError("k_q must be [pages, heads, page, dim]")
    shape = kq.shape
    pages, heads, page, dim = shape
    scales = (pages, heads, page, dim // 32)
    return Cache(_flat(kq, shape, u8, dev, "k_q"), _flat(c["k_s"], scales, u8, dev, "k_s"),
                 _flat(c["v_q"], shape, u8, dev, "v_q"), _flat(c["v_s"], scales, u8, dev, "v_s"),
                 pages, heads, page, dim, fmt)


def cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: dict, fmt: int, stream=None) -> None:
    """Quantizes the keys and values of some tokens (fp32 or bf16 [tokens, heads,
    dim]) into a cache (``kv_cache``): token t goes to place slots[t] % page of
    page slots[t] // page; a slot outside the cache (-1) is not written."""
    handle, dev = _on(stream, k)
    c = _cache(cache, fmt, dev)
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3 or dtype not in _SRC or v.dtype != dtype or v.shape != shape or v.get_device() != dev:
        raise ValueError("k and v must be fp32/bf16 [tokens, heads, dim] tensors of one type")
    tokens = shape[0]
    if shape[1:] != (c.heads, c.dim):
        raise ValueError(f"k must be [tokens, {c.heads}, {c.dim}]")
    (ld_k, hs_k, unit_k), (ld_v, hs_v, unit_v) = k.stride(), v.stride()
    if unit_k != 1 or unit_v != 1:
        raise ValueError("k and v must have unit stride along dim")
    if tokens <= 1:  # the stride of a single token or head says nothing
        ld_k = ld_v = 0
    if c.heads <= 1:
        hs_k = hs_v = c.dim
    _check(lib.mx_cache_write(c, k.data_ptr(), ld_k, hs_k, v.data_ptr(), ld_v, hs_v, _SRC[dtype], tokens,
                              _flat(slots, (tokens,), torch.int64, dev, "slots"), handle), "mx_cache_write")


def attention(q: torch.Tensor, cache: dict, fmt: int, table: torch.Tensor, lens: torch.Tensor,
              scale: float | None = None, max_len: int | None = None, out: dict | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Attention of the last Lq tokens of B requests (q bf16 [B, Lq, query heads,
    dim]) over the requests' cached tokens: lens [B] int32 of them, the queries'
    own included, in the pages table [B, n] int32.  Query i sees the tokens before
    lens - Lq + i + 1.  Returns o like q and lse [B, Lq, query heads] fp32.
    ``max_len``: a bound of lens (default: what the table holds, which is slow where
    that is far more than the longest request has, as the work is cut by it); ``scale``:
    default 1 / sqrt(dim); ``out`` and ``workspace`` may be supplied."""
    handle, dev = _on(stream, q)
    c = _cache(cache, fmt, dev)
    shape, dim = q.shape, c.dim
    if len(shape) != 4 or q.dtype != torch.bfloat16 or shape[3] != dim:
        raise ValueError(f"q must be a bf16 [B, Lq, query heads, {dim}] tensor")
    B, Lq, heads_q, _ = shape
    sq = q.stride()
    if sq[3] != 1 or (sq[2] != dim and heads_q > 1) or (sq[0] != Lq * sq[1] and B > 1 and Lq > 1):
        raise ValueError("q must have contiguous heads and evenly spaced tokens")
    ld_q = sq[1] if Lq > 1 else sq[0] if B > 1 else heads_q * dim
    if table.dim() != 2 or table.dtype != torch.int32 or table.get_device() != dev or table.shape[0] != B or \
            (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be an int32 [B, pages] tensor with unit column stride")
    per = table.shape[1]
    if max_len is None:
        max_len = per * c.page
    elif max_len > per * c.page:  # whatever the distance of the table's rows is
        raise MXError(MX_ERR_SHAPE, "mx_attention")
    o = dict(out) if out else {}
    device = q.device
    po = _out(o, "o", shape, torch.bfloat16, dev, device, stream)
    plse = _out(o, "lse", (B, Lq, heads_q), torch.float32, dev, device, stream)
    if workspace is None:
        need = lib.mx_attention_workspace(B, Lq, heads_q, c.heads, dim, max_len)
        if need > 0:
            workspace = _empty(torch.uint8, device, stream, need)
    _check(lib.mx_attention(c, q.data_ptr(), ld_q, table.data_ptr(), table.stride(0) if B > 1 else per,
                            _flat(lens, (B,), torch.int32, dev, "lens"), B, Lq, heads_q,
                            dim ** -0.5 if scale is None else scale, max_len,
                            po, heads_q * dim, plse, *_work(workspace, dev), handle), "mx_attention")
    return o
