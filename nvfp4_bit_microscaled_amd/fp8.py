"""Python binding of the library's 8-bit operators (include/nvfp4_amd_fp8.h): E4M3
codes with one power-of-two scale per block of 128, the norm and the gated
feed-forward block on them.  Argument marshalling only, as the rest of the package:
the C names and the C argument order, with workspaces and streams as keywords.
"""
import ctypes

import torch

from . import _check, _dtype, _ws, load

BLOCK = 128
GEMM_FAST = 1 << 0

# every symbol nvfp4_amd_fp8.h declares
FP8_EXPORTS = ("fp8_tensor_bytes", "fp8_quantize", "fp8_rms_norm", "fp8_rms_norm_backward", "fp8_rms_norm_ws_bytes",
               "fp8_gemm", "fp8_gemm_ws_bytes", "fp8_ffn_fprop", "fp8_ffn_fprop_flags", "fp8_ffn_backward",
               "fp8_ffn_backward_flags", "fp8_ffn_ws_bytes", "fp8_ffn_fprop_ws_bytes", "fp8_ffn_backward_ws_bytes")


class fp8_tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("two_d", ctypes.c_int32)]


class fp8_ffn_buffers(ctypes.Structure):
    _fields_ = [("dgq", fp8_tensor), ("duq", fp8_tensor), ("dgq_t", fp8_tensor), ("duq_t", fp8_tensor),
                ("hq_t", fp8_tensor)]


_declared = None


def lib():
    """The loaded library with the 8-bit entry points' argument types."""
    global _declared
    if _declared is None:
        L = load()
        vp, i64, i32, f32, szv = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        tp, sz = ctypes.POINTER(fp8_tensor), ctypes.POINTER(ctypes.c_size_t)
        sigs = {
            "fp8_tensor_bytes": [i64, i64, i32, sz, sz],
            "fp8_quantize": [vp, i32, i64, i64, i64, tp, tp, vp],
            "fp8_rms_norm": [vp, i64, vp, i64, i32, i64, i64, vp, f32, vp, i64, tp, tp, vp, vp],
            "fp8_rms_norm_backward": [vp, vp, vp, i32, i64, i64, vp, vp, vp, vp, vp, szv, vp],
            "fp8_rms_norm_ws_bytes": [i64, i64, sz],
            "fp8_gemm": [tp, tp, vp, i32, i64, ctypes.c_uint32, vp, szv, vp],
            "fp8_gemm_ws_bytes": [i64, i64, i64, sz],
            "fp8_ffn_fprop": [tp, tp, tp, tp, tp, vp, vp, vp, i64, vp, szv, vp],
            "fp8_ffn_backward": [tp, tp, tp, tp, tp, tp, vp, vp, ctypes.POINTER(fp8_ffn_buffers), vp, vp, vp, vp, vp,
                                 szv, vp],
            "fp8_ffn_fprop_flags": [tp, tp, tp, tp, tp, vp, vp, vp, i64, ctypes.c_uint32, vp, szv, vp],
            "fp8_ffn_backward_flags": [tp, tp, tp, tp, tp, tp, vp, vp, ctypes.POINTER(fp8_ffn_buffers), vp, vp, vp, vp,
                                       ctypes.c_uint32, vp, szv, vp],
            "fp8_ffn_ws_bytes": [i64, i64, i64, sz],
            "fp8_ffn_fprop_ws_bytes": [i64, i64, i64, i32, ctypes.c_uint32, sz],
            "fp8_ffn_backward_ws_bytes": [i64, i64, i64, ctypes.c_uint32, sz],
        }
        for name, args in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        _declared = L
    return _declared


def _stream(stream=None):
    """The raw handle of `stream`, or of the current stream by the short way: a call on few
    tokens takes less time on the GPU than torch.cuda.current_stream() does on the host."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _bytes(name, *sizes):
    n = ctypes.c_size_t()
    _check(name, getattr(lib(), name)(*sizes, ctypes.byref(n)))
    return n.value


def fp8_tensor_bytes(rows: int, cols: int, two_d: bool = False):
    nc, ns = ctypes.c_size_t(), ctypes.c_size_t()
    _check("fp8_tensor_bytes",
           lib().fp8_tensor_bytes(rows, cols, int(two_d), ctypes.byref(nc), ctypes.byref(ns)))
    return nc.value, ns.value


class Fp8Tensor:
    """One quantized logical tensor [rows][cols], blocked along cols: `codes`, E4M3
    bytes [rows][cols padded to 128], and `scales`, E8M0 bytes [blocks along cols][rows
    padded to 16], or [blocks along cols][blocks along rows] with two_d."""

    def __init__(self, rows: int, cols: int, two_d: bool = False, device="cuda"):
        nc, ns = fp8_tensor_bytes(rows, cols, two_d)
        kb = -(-cols // BLOCK)
        self._set(torch.empty(nc, dtype=torch.uint8, device=device).view(rows, kb * BLOCK),
                  torch.empty(ns, dtype=torch.uint8, device=device).view(kb, ns // kb if kb else 0),
                  rows, cols, two_d)

    @classmethod
    def wrap(cls, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, two_d: bool = False):
        """A descriptor of codes and scales that the caller holds (contiguous, in the
        layout above, any 1-byte type)."""
        nc, ns = fp8_tensor_bytes(rows, cols, two_d)
        for t, n in ((codes, nc), (scales, ns)):
            if t.element_size() != 1 or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"contiguous 1-byte tensors of {nc} codes and {ns} scales expected")
        q = cls.__new__(cls)
        q._set(codes, scales, rows, cols, two_d)
        return q

    def _set(self, codes, scales, rows, cols, two_d):
        self.codes, self.scales, self.rows, self.cols, self.two_d = codes, scales, rows, cols, bool(two_d)
        self._desc = fp8_tensor(codes.data_ptr(), scales.data_ptr(), rows, cols, int(self.two_d))
        self.desc = ctypes.byref(self._desc)


def _q(q):
    return q.desc if q is not None else None


def _p(t):
    return t.data_ptr() if t is not None else None


def _ld(t):
    """The row stride of a 2D tensor whose rows are contiguous; of a single row (one token
    of a transposed or expanded tensor) torch gives any."""
    (rows, cols), (ld, one) = t.shape, t.stride()
    if one != 1 and cols > 1:
        raise ValueError("2D row-major tensor expected")
    return ld if rows > 1 else max(ld, cols)


def fp8_quantize(x: torch.Tensor, q: Fp8Tensor = None, q_t: Fp8Tensor = None, stream=None):
    """x [rows][cols] (bf16 or fp32, any row stride) into q and, transposed, q_t, in one
    read; either may be None."""
    _check("fp8_quantize", lib().fp8_quantize(x.data_ptr(), _dtype(x), x.shape[0], x.shape[1], _ld(x), _q(q), _q(q_t),
                                              _stream(stream)))


def fp8_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, yq: Fp8Tensor, residual: torch.Tensor = None,
                 h: torch.Tensor = None, yq_t: Fp8Tensor = None, rstd: torch.Tensor = None, stream=None):
    """h = x + residual; yq (and yq_t, transposed) = h / rms(h) * weight, quantized.
    h and residual go together; rstd [rows] fp32 is kept for the backward pass."""
    rows, cols = shape = x.shape
    _dense(weight, (cols,), torch.float32)
    if residual is not None:
        _like(residual, shape, x.dtype)
    if h is not None:
        _like(h, shape, x.dtype)
    if rstd is not None:
        _dense(rstd, (rows,), torch.float32)
    code = lib().fp8_rms_norm(
        x.data_ptr(), _ld(x), None if residual is None else residual.data_ptr(),
        cols if residual is None else _ld(residual), _dtype(x), rows, cols, weight.data_ptr(), eps,
        None if h is None else h.data_ptr(), cols if h is None else _ld(h), yq.desc,
        None if yq_t is None else yq_t.desc, None if rstd is None else rstd.data_ptr(), _stream(stream))
    if code:
        _check("fp8_rms_norm", code)


def fp8_rms_norm_ws_bytes(rows: int, cols: int) -> int:
    return _bytes("fp8_rms_norm_ws_bytes", rows, cols)


def fp8_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          dx: torch.Tensor, dweight: torch.Tensor, ws: torch.Tensor, dh: torch.Tensor = None,
                          stream=None):
    """dx and dweight of fp8_rms_norm from dy (the gradient of y) and dh (the residual
    stream's own gradient, optional).  ws: fp8_rms_norm_ws_bytes device bytes."""
    rows, cols = h.shape
    for t in (dy, h, dx, dh):
        if t is not None:
            _dense(t, (rows, cols), h.dtype)
    _dense(weight, (cols,), torch.float32)
    _dense(rstd, (rows,), torch.float32)
    _dense(dweight, (cols,), torch.float32)
    wp, wb = _ws(ws)
    _check("fp8_rms_norm_backward", lib().fp8_rms_norm_backward(
        dy.data_ptr(), h.data_ptr(), _p(dh), _dtype(h), rows, cols, weight.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
        dweight.data_ptr(), wp, wb, _stream(stream)))


def fp8_gemm_ws_bytes(M: int, N: int, K: int) -> int:
    return _bytes("fp8_gemm_ws_bytes", M, N, K)


def fp8_gemm(a: Fp8Tensor, b: Fp8Tensor, c: torch.Tensor, ws: torch.Tensor = None, fast: bool = False, stream=None):
    """c [a.rows][b.rows] (bf16 or fp32, any row stride) = deq(a) deq(b)^T, summed in
    binary32; fast: by the 8-bit matrix instruction, at twice the rate, with a relative
    error of about 2e-5 (see the header)."""
    if c.shape != (a.rows, b.rows):
        raise ValueError(f"c is {tuple(c.shape)}, the product {(a.rows, b.rows)}")
    wp, wb = _ws(ws)
    _check("fp8_gemm", lib().fp8_gemm(a.desc, b.desc, c.data_ptr(), _dtype(c), _ld(c), GEMM_FAST if fast else 0, wp, wb,
                                      _stream(stream)))


def fp8_ffn_ws_bytes(M: int, K: int, F: int) -> int:
    """Enough for the forward and the backward call."""
    return _bytes("fp8_ffn_ws_bytes", M, K, F)


def fp8_ffn_fprop_ws_bytes(M: int, K: int, F: int, keep: bool = False, fast: bool = False) -> int:
    """The forward call's own; keep: it is given g and u."""
    return _bytes("fp8_ffn_fprop_ws_bytes", M, K, F, int(keep), GEMM_FAST if fast else 0)


def fp8_ffn_backward_ws_bytes(M: int, K: int, F: int, fast: bool = False) -> int:
    """The backward call's own, for g and u aligned to 16 bytes."""
    return _bytes("fp8_ffn_backward_ws_bytes", M, K, F, GEMM_FAST if fast else 0)


def fp8_ffn_fprop(xq: Fp8Tensor, wg: Fp8Tensor, wu: Fp8Tensor, wd: Fp8Tensor, hq: Fp8Tensor, y: torch.Tensor,
                  g: torch.Tensor = None, u: torch.Tensor = None, ws: torch.Tensor = None, stream=None,
                  fast: bool = False):
    """y = (silu(x wg^T) * (x wu^T)) wd^T; g and u (bf16 [M][F], both or neither) keep
    the projections for fp8_ffn_backward.  ws: fp8_ffn_fprop_ws_bytes device bytes.  fast:
    as for fp8_gemm, for all of the block's products (the header says what it costs)."""
    for t in (g, u):
        if t is not None:
            _dense(t, (xq.rows, wg.rows), torch.bfloat16)
    if y.dtype != torch.bfloat16 or y.shape != (xq.rows, xq.cols):
        raise ValueError("y: bf16, one row per token")
    wp, wb = _ws(ws)
    _check("fp8_ffn_fprop", lib().fp8_ffn_fprop_flags(
        xq.desc, wg.desc, wu.desc, wd.desc, hq.desc, _p(g), _p(u), y.data_ptr(), _ld(y), GEMM_FAST if fast else 0, wp,
        wb, _stream(stream)))


class FfnBuffers:
    """Caller-owned quantized intermediates of fp8_ffn_backward for M tokens, width K
    and inner width F."""

    def __init__(self, M: int, K: int, F: int, device="cuda"):
        self.dgq, self.duq = Fp8Tensor(M, F, device=device), Fp8Tensor(M, F, device=device)
        self.dgq_t, self.duq_t = Fp8Tensor(F, M, device=device), Fp8Tensor(F, M, device=device)
        self.hq_t = Fp8Tensor(F, M, device=device)
        self._s = fp8_ffn_buffers(self.dgq._desc, self.duq._desc, self.dgq_t._desc, self.duq_t._desc, self.hq_t._desc)


def fp8_ffn_backward(dyq: Fp8Tensor, dyq_t: Fp8Tensor, xq_t: Fp8Tensor, wg_t: Fp8Tensor, wu_t: Fp8Tensor,
                     wd_t: Fp8Tensor, g: torch.Tensor, u: torch.Tensor, bufs: FfnBuffers, dx: torch.Tensor,
                     dwg: torch.Tensor, dwu: torch.Tensor, dwd: torch.Tensor, ws: torch.Tensor = None, stream=None,
                     fast: bool = False):
    """The block's gradients (bf16) from dy in both layouts, x^T, the transposed weights
    and the forward call's g and u.  ws: fp8_ffn_backward_ws_bytes device bytes; fast as
    for the forward call."""
    M, K, F = dyq.rows, dyq.cols, wd_t.rows
    for t, shape in ((g, (M, F)), (u, (M, F)), (dx, (M, K)), (dwg, (F, K)), (dwu, (F, K)), (dwd, (K, F))):
        _dense(t, shape, torch.bfloat16)
    wp, wb = _ws(ws)
    _check("fp8_ffn_backward", lib().fp8_ffn_backward_flags(
        dyq.desc, dyq_t.desc, xq_t.desc, wg_t.desc, wu_t.desc, wd_t.desc, g.data_ptr(), u.data_ptr(),
        ctypes.byref(bufs._s), dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), dwd.data_ptr(),
        GEMM_FAST if fast else 0, wp, wb, _stream(stream)))


def _dense(t, shape, dtype):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"contiguous {dtype} tensor {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")


def _like(t, shape, dtype):
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{dtype} tensor {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
