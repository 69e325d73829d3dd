"""Python binding of the library's 8-bit operators (include/nvfp4_amd_fp8.h): E4M3
codes with one power-of-two scale per block of 128, the norm and the gated
feed-forward block on them, dropout, and low-rank adapters beside a projection.
Argument marshalling only, as the rest of the package: the C names and the C argument
order, with workspaces and streams as keywords.
"""
import ctypes

import torch

from . import _check, _dtype, _ws, load

BLOCK = 128
GEMM_FAST = 1 << 0
LORA_MIXED = 1 << 3

# every symbol nvfp4_amd_fp8.h declares
FP8_EXPORTS = ("fp8_tensor_bytes", "fp8_quantize", "fp8_rms_norm", "fp8_rms_norm_backward", "fp8_rms_norm_ws_bytes",
               "fp8_gemm", "fp8_gemm_ws_bytes", "fp8_ffn_fprop", "fp8_ffn_fprop_flags", "fp8_ffn_backward",
               "fp8_ffn_backward_flags", "fp8_ffn_ws_bytes", "fp8_ffn_fprop_ws_bytes", "fp8_ffn_backward_ws_bytes",
               "fp8_dropout", "fp8_dropout_rms_norm", "fp8_dropout_rms_norm_backward", "fp8_lora_fprop",
               "fp8_lora_fprop_ws_bytes", "fp8_lora_backward", "fp8_lora_backward_ws_bytes")


class fp8_tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("two_d", ctypes.c_int32)]


class fp8_ffn_buffers(ctypes.Structure):
    _fields_ = [("dgq", fp8_tensor), ("duq", fp8_tensor), ("dgq_t", fp8_tensor), ("duq_t", fp8_tensor),
                ("hq_t", fp8_tensor)]


class fp8_dropout_config(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("step", ctypes.c_void_p)]


class fp8_lora(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("count", ctypes.c_int32), ("rank", ctypes.c_int32)]


_declared = None


def lib():
    """The loaded library with the 8-bit entry points' argument types."""
    global _declared
    if _declared is None:
        L = load()
        vp, i64, i32, f32, szv = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        tp, sz = ctypes.POINTER(fp8_tensor), ctypes.POINTER(ctypes.c_size_t)
        dp, lp, u32 = ctypes.POINTER(fp8_dropout_config), ctypes.POINTER(fp8_lora), ctypes.c_uint32
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
            "fp8_dropout": [vp, i64, vp, i64, i32, i64, i64, dp, vp, i64, vp],
            "fp8_dropout_rms_norm": [vp, i64, vp, i64, i32, i64, i64, dp, vp, f32, vp, i64, tp, tp, vp, vp],
            "fp8_dropout_rms_norm_backward": [vp, vp, vp, i32, i64, i64, dp, vp, vp, vp, vp, vp, vp, szv, vp],
            "fp8_lora_fprop": [tp, tp, lp, vp, dp, vp, i64, u32, vp, szv, vp],
            "fp8_lora_fprop_ws_bytes": [i64, i64, i64, i32, u32, sz],
            "fp8_lora_backward": [tp, tp, tp, lp, vp, dp, vp, i64, vp, vp, u32, vp, szv, vp],
            "fp8_lora_backward_ws_bytes": [i64, i64, i64, i32, i32, u32, sz],
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
        if codes.device != scales.device:  # a call looks at the codes' device
            raise ValueError(f"codes on {codes.device}, scales on {scales.device}")
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


class Dropout:
    """One dropout's probability and place in the generator: `seed` and `offset` are the
    caller's, `step` (optional, one int64 or uint64 on the device) is added to offset when
    the kernels run.  Calls with the same four and a tensor of the same shape use the same
    mask; a layer and step of a run take an offset of their own: offset + step is one number,
    so layers' offsets belong further apart than a run's steps (layer << 40).  Stochastic
    rounding draws the same bits of the same seed and offset: give it others."""

    def __init__(self, p: float, seed: int, offset: int = 0, step: torch.Tensor = None):
        if not 0 <= p < 1:
            raise ValueError(f"a probability in [0, 1) expected, got {p}")
        if step is not None and (step.dtype not in (torch.int64, torch.uint64) or step.numel() != 1):
            raise ValueError("step: one 64-bit integer")
        self.p, self.seed, self.offset, self.step = p, seed, offset, step
        self._s = fp8_dropout_config(p, seed & (2 ** 64 - 1), offset & (2 ** 64 - 1), _p(step))
        self.desc = ctypes.byref(self._s)


def fp8_dropout(x: torch.Tensor, drop: Dropout, y: torch.Tensor, residual: torch.Tensor = None, stream=None):
    """y = residual + dropout(x) (bf16 or fp32, any row strides); without a residual also the
    gradient, from dy.  y may be x or the residual."""
    _like(y, x.shape, x.dtype)
    if residual is not None:
        _like(residual, x.shape, x.dtype)
    rows, cols = x.shape
    _on_one_device(x, y, residual, drop.step)
    code = lib().fp8_dropout(x.data_ptr(), _ld(x), _p(residual), cols if residual is None else _ld(residual), _dtype(x),
                             rows, cols, drop.desc, y.data_ptr(), _ld(y), _stream(stream))
    if code:
        _check("fp8_dropout", code)


def fp8_dropout_rms_norm(x: torch.Tensor, drop: Dropout, weight: torch.Tensor, eps: float, yq: Fp8Tensor,
                         residual: torch.Tensor, h: torch.Tensor, yq_t: Fp8Tensor = None, rstd: torch.Tensor = None,
                         stream=None):
    """h = residual + dropout(x); yq (and yq_t, transposed) = h / rms(h) * weight, quantized:
    fp8_rms_norm behind a dropped-out branch."""
    rows, cols = shape = x.shape
    _dense(weight, (cols,), torch.float32)
    _like(residual, shape, x.dtype)
    _like(h, shape, x.dtype)
    if rstd is not None:
        _dense(rstd, (rows,), torch.float32)
    _on_one_device(x, residual, h, weight, rstd, drop.step, yq.codes, None if yq_t is None else yq_t.codes)
    _check("fp8_dropout_rms_norm", lib().fp8_dropout_rms_norm(
        x.data_ptr(), _ld(x), residual.data_ptr(), _ld(residual), _dtype(x), rows, cols, drop.desc, weight.data_ptr(),
        eps, h.data_ptr(), _ld(h), yq.desc, _q(yq_t), _p(rstd), _stream(stream)))


def fp8_dropout_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                                  drop: Dropout, dx: torch.Tensor, dresidual: torch.Tensor, dweight: torch.Tensor,
                                  ws: torch.Tensor, dh: torch.Tensor = None, stream=None):
    """dx (of the dropped-out branch), dresidual and dweight of fp8_dropout_rms_norm from dy
    and dh (the residual stream's own gradient, optional).  ws: fp8_rms_norm_ws_bytes."""
    rows, cols = h.shape
    for t in (dy, h, dx, dresidual, dh):
        if t is not None:
            _dense(t, (rows, cols), h.dtype)
    _dense(weight, (cols,), torch.float32)
    _dense(rstd, (rows,), torch.float32)
    _dense(dweight, (cols,), torch.float32)
    _on_one_device(dy, h, dx, dresidual, dh, weight, rstd, dweight, ws, drop.step)
    wp, wb = _ws(ws)
    _check("fp8_dropout_rms_norm_backward", lib().fp8_dropout_rms_norm_backward(
        dy.data_ptr(), h.data_ptr(), _p(dh), _dtype(h), rows, cols, drop.desc, weight.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), dresidual.data_ptr(), dweight.data_ptr(), wp, wb, _stream(stream)))


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


class LoraAdapters:
    """`count` low-rank adapters of a projection from `cols` to `rows` features: `a` [count]
    [rank][cols padded to 8] and `b` [count][rows][rank], bf16, and `scale` [count] fp32
    (alpha / rank).  rank is a multiple of 8 up to 128: one in between is stored with zeros
    in a's further rows and b's further columns.  New ones have b = 0 and add nothing."""

    def __init__(self, count: int, rank: int, rows: int, cols: int, device="cuda"):
        z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=device)  # noqa: E731
        self._set(z(count, rank, -(-cols // 8) * 8), z(count, rows, rank), torch.ones(count, device=device), cols)

    @classmethod
    def wrap(cls, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor, cols: int):
        """A descriptor of adapters that the caller holds, in the layout above."""
        l = cls.__new__(cls)
        l._set(a, b, scale, cols)
        return l

    def _set(self, a, b, scale, cols):
        count, rank, lda = a.shape
        if rank % 8 or not 8 <= rank <= 128 or lda % 8 or lda < cols or count < 1:
            raise ValueError(f"a: [count][rank][lda] expected, rank and lda multiples of 8, rank at most 128 and lda at "
                             f"least {cols}, got {tuple(a.shape)}")
        _dense(a, (count, rank, lda), torch.bfloat16)
        _dense(b, (count, b.shape[1], rank), torch.bfloat16)
        _dense(scale, (count,), torch.float32)
        self.a, self.b, self.scale = a, b, scale
        self.count, self.rank, self.rows, self.cols = count, rank, b.shape[1], cols
        self._s = fp8_lora(a.data_ptr(), b.data_ptr(), scale.data_ptr(), lda, count, rank)
        self.desc = ctypes.byref(self._s)


def _lora_flags(fast, mixed):
    return (GEMM_FAST if fast else 0) | (LORA_MIXED if mixed else 0)


def fp8_lora_fprop_ws_bytes(M: int, N: int, K: int, rank: int, fast: bool = False, mixed: bool = False) -> int:
    return _bytes("fp8_lora_fprop_ws_bytes", M, N, K, rank, _lora_flags(fast, mixed))


def fp8_lora_backward_ws_bytes(M: int, N: int, K: int, rank: int, count: int, fast: bool = False,
                               mixed: bool = False) -> int:
    return _bytes("fp8_lora_backward_ws_bytes", M, N, K, rank, count, _lora_flags(fast, mixed))


def fp8_lora_fprop(xq: Fp8Tensor, wq: Fp8Tensor, lora: LoraAdapters, y: torch.Tensor, index: torch.Tensor = None,
                   drop: Dropout = None, ws: torch.Tensor = None, fast: bool = False, stream=None, mixed: bool = False):
    """y[m] (bf16, any row stride) = x[m] W^T + scale_i (dropout(x)[m] a_i^T) b_i^T, i =
    index[m] (int32; outside [0, count): no adapter; None: all tokens have adapter 0).  ws:
    fp8_lora_fprop_ws_bytes device bytes; fast: as for fp8_gemm, for the product with W; mixed:
    neighbouring tokens have different adapters (of 65 to 512 tokens: what takes less time then)."""
    _lora_shapes(lora, wq.rows, wq.cols, xq.rows, index)
    _like(y, (xq.rows, wq.rows), torch.bfloat16)
    _on_one_device(y, xq.codes, wq.codes, lora.a, lora.b, lora.scale, index, ws, None if drop is None else drop.step)
    wp, wb = _ws(ws)
    code = lib().fp8_lora_fprop(xq.desc, wq.desc, lora.desc, _p(index), _q(drop), y.data_ptr(), _ld(y),
                                _lora_flags(fast, mixed), wp, wb, _stream(stream))
    if code:
        _check("fp8_lora_fprop", code)


def fp8_lora_backward(dyq: Fp8Tensor, wq_t: Fp8Tensor, xq: Fp8Tensor, lora: LoraAdapters, dx: torch.Tensor,
                      da: torch.Tensor, db: torch.Tensor, ws: torch.Tensor, index: torch.Tensor = None,
                      drop: Dropout = None, fast: bool = False, stream=None, mixed: bool = False):
    """dx (bf16, any row stride), da and db (fp32, a's and b's layouts) from dy, the transposed
    weight, x, and the forward call's adapters, index and drop; fast and mixed as there.  ws:
    fp8_lora_backward_ws_bytes device bytes."""
    _lora_shapes(lora, wq_t.cols, wq_t.rows, xq.rows, index)
    _like(dx, (xq.rows, xq.cols), torch.bfloat16)
    _dense(da, lora.a.shape, torch.float32)
    _dense(db, lora.b.shape, torch.float32)
    _on_one_device(dx, dyq.codes, wq_t.codes, xq.codes, lora.a, lora.b, lora.scale, da, db, index, ws,
                   None if drop is None else drop.step)
    wp, wb = _ws(ws)
    _check("fp8_lora_backward", lib().fp8_lora_backward(
        dyq.desc, wq_t.desc, xq.desc, lora.desc, _p(index), _q(drop), dx.data_ptr(), _ld(dx), da.data_ptr(),
        db.data_ptr(), _lora_flags(fast, mixed), wp, wb, _stream(stream)))


def _lora_shapes(lora, rows, cols, tokens, index):
    if (lora.rows, lora.cols) != (rows, cols):
        raise ValueError(f"adapters of a {(lora.rows, lora.cols)} projection, the weight is {(rows, cols)}")
    if index is not None:
        _dense(index, (tokens,), torch.int32)


def _on_one_device(first, *others):
    """Every tensor is on the current GPU, whose stream and kernels the call uses."""
    d = first.device
    for t in others:
        if t is not None and t.device != d:
            raise ValueError(f"tensors on {d} and {t.device}")
    if d.type != "cuda":
        raise ValueError(f"tensors on a GPU expected, got {d}")
    if d.index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {d}, which is not the current device")


def _dense(t, shape, dtype):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"contiguous {dtype} tensor {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")


def _like(t, shape, dtype):
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{dtype} tensor {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
