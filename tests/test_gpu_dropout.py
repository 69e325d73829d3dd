"""GPU: dropout alone, in front of the norm, and in its gradient.

Tolerances, fixed before the first run: fp8_dropout takes two binary32 operations (the
product with the gain, the sum) and one rounding, which torch repeats on the CPU: equal.
The norm's outputs equal those of fp8_dropout and then fp8_rms_norm, which do the same
operations.  dresidual equals fp8_rms_norm_backward's dx; dx is dropout of it before its own
rounding: equal in binary32 (there is none); in bf16 two roundings lie between dx and the
dropout of the rounded one, 2^-8 of the value each."""
import pytest
import torch

import drop_ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SHAPES = [(1, 1), (1, 7), (3, 8), (1, 5120), (8, 5120), (5, 513), (130, 520), (33, 2501), (7, 8200), (2, 16385), (300, 1000)]


def make(rows, cols, dtype, seed, extra=0):
    """A tensor with rows cols + extra apart."""
    gen = torch.Generator().manual_seed(seed)
    t = torch.randn(rows, cols + extra, generator=gen).to(DT[dtype]).cuda()
    return t[:, :cols]


def want(x, residual, p, mask):
    y = drop_ref.dropout(x.cpu(), p, mask)
    return (y if residual is None else residual.cpu().float() + y).to(x.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dropout(fp4, rows, cols, dtype):
    for i, (p, extra, has_res) in enumerate(((0.1, 0, True), (0.5, 0, False), (0.3, 3, True), (0.25, 8, False),
                                             (0.0, 0, True), (0.99, 8, True))):
        x, r = make(rows, cols, dtype, i, extra), make(rows, cols, dtype, 50 + i, extra) if has_res else None
        buf = torch.full((rows, cols + extra), 7.0, dtype=x.dtype, device="cuda")
        y = buf[:, :cols]
        step = torch.tensor([3 + i], dtype=torch.int64, device="cuda")
        fp4.fp8_dropout(x, fp4.Dropout(p, 0x123456789ABCDEF0 + i, 2 ** 33 + 1, step if i % 2 else None), y, residual=r)
        mask = drop_ref.keep(rows, cols, p, 0x123456789ABCDEF0 + i, 2 ** 33 + 1, 3 + i if i % 2 else 0)
        assert torch.equal(y.cpu(), want(x, r, p, mask)), (p, extra, has_res)
        assert (buf[:, cols:] == 7.0).all()  # what lies between the rows is left as it is


def test_gradient_is_the_formulas_and_the_differences(fp4):
    """dropout is linear with the same mask: its gradient's call on dy, and the central
    difference of sum(dropout(x) * dy) along v, which is exact here but for the sums'
    rounding (binary64 sums of binary32 values of one rounding each: 2^-23 of sum |.|)."""
    p, d = 0.3, fp4.Dropout(0.3, 5, 6)
    x, dy, v = (make(40, 100, "fp32", s) for s in (1, 2, 3))
    out = [torch.empty_like(x) for _ in range(3)]
    fp4.fp8_dropout(dy, d, out[0])
    assert torch.equal(out[0].cpu(), want(dy, None, p, drop_ref.keep(40, 100, p, 5, 6)))
    fp4.fp8_dropout(x + v, d, out[1])
    fp4.fp8_dropout(x - v, d, out[2])
    diff = ((out[1].double() - out[2].double()) * dy.double() / 2).sum()
    scale = ((out[1].double().abs() + out[2].double().abs()) * dy.double().abs()).sum()
    assert abs(float(diff - (out[0].double() * v.double()).sum())) <= 2.0 ** -22 * float(scale)


@pytest.mark.parametrize("rows,cols", [(4, 64), (5, 77)])
def test_in_place_and_nonfinite(fp4, rows, cols):
    """y in x's or the residual's place; a dropped infinity or NaN counts as 0."""
    d, mask = fp4.Dropout(0.4, 11), drop_ref.keep(rows, cols, 0.4, 11)
    x, r = make(rows, cols, "bf16", 1), make(rows, cols, "bf16", 2)
    x[0, :] = float("nan")
    x[1, :] = float("inf")
    ref = want(x, r, 0.4, mask)
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        fp4.fp8_dropout(a, d, (a, b)[which], residual=b)
        got = (a, b)[which].cpu()
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.nan_to_num(9.0), ref.nan_to_num(9.0))
    assert torch.equal(ref[0].isnan(), mask[0])


def test_refused_and_empty(fp4):
    x = make(4, 16, "bf16", 1)
    with pytest.raises(ValueError):
        fp4.fp8_dropout(x, fp4.Dropout(0.1, 1, step=torch.zeros(1, dtype=torch.int64)), torch.empty_like(x))
    with pytest.raises(ValueError):
        fp4.fp8_dropout(x.t(), fp4.Dropout(0.1, 1), torch.empty_like(x.t()))
    with pytest.raises(fp4.Fp4Error):
        fp4.fp8_dropout(x, fp4.Dropout(1 - 2.0 ** -18, 1), torch.empty_like(x))
    e = torch.empty(0, 16, device="cuda")
    fp4.fp8_dropout(e, fp4.Dropout(0.1, 1), e)


def test_another_stream(fp4):
    x, d = make(64, 1024, "bf16", 1), fp4.Dropout(0.2, 3)
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fp4.fp8_dropout(x, d, y, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y.cpu(), want(x, None, 0.2, drop_ref.keep(64, 1024, 0.2, 3)))


def test_captured_graph_draws_anew(fp4):
    """A graph whose step is advanced in it: each replay's mask is the next step's."""
    x = make(16, 264, "bf16", 1)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    y, d = torch.empty_like(x), fp4.Dropout(0.5, 21, 100, step)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fp4.fp8_dropout(x, d, y)  # before the capture
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp4.fp8_dropout(x, d, y)
        step.add_(1)
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(x)
        fp4.fp8_dropout(x, fp4.Dropout(0.5, 21, 100 + i), eager)
        assert torch.equal(y, eager)
        assert torch.equal(eager.cpu(), want(x, None, 0.5, drop_ref.keep(16, 264, 0.5, 21, 100 + i)))


NORM_SHAPES = [(1, 64), (9, 500), (5, 777), (6, 1024), (4, 1500), (3, 2501), (130, 3000), (5, 4095), (7, 5120), (2, 6145), (3, 8192),
               (2, 9001), (2, 10240)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_equals_dropout_then_norm(fp4, rows, cols, dtype):
    p = 0.2
    d = fp4.Dropout(p, 9, 1, torch.tensor([4], device="cuda"))
    for extra in (0, 5):
        x, r = make(rows, cols, dtype, 1, extra), make(rows, cols, dtype, 2, extra)
        w = 1 + 0.1 * make(1, cols, "fp32", 3)[0].contiguous()
        h, h2 = torch.empty_like(x), torch.empty(rows, cols, dtype=x.dtype, device="cuda")
        q, qt, q2, qt2 = (fp4.Fp8Tensor(*s) for s in ((rows, cols), (cols, rows)) * 2)
        rs, rs2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        fp4.fp8_dropout_rms_norm(x, d, w, 1e-6, q, r, h, yq_t=qt, rstd=rs)
        fp4.fp8_dropout(x, d, h2, residual=r)
        fp4.fp8_rms_norm(h2, w, 1e-6, q2, yq_t=qt2, rstd=rs2)
        assert torch.equal(h, h2) and torch.equal(rs, rs2)
        assert torch.equal(h.cpu(), want(x, r, p, drop_ref.keep(rows, cols, p, 9, 5)))
        for a, b in ((q, q2), (qt, qt2)):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales[:, :a.rows], b.scales[:, :b.rows])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_gradient(fp4, rows, cols, dtype):
    p = 0.3
    d, mask = fp4.Dropout(p, 31, 2), drop_ref.keep(rows, cols, p, 31, 2)
    h, dy, dh = (make(rows, cols, dtype, s).contiguous() for s in (1, 2, 3))
    w = 1 + 0.1 * make(1, cols, "fp32", 4)[0].contiguous()
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-6).float()
    ws = torch.empty(max(fp4.fp8_rms_norm_ws_bytes(rows, cols), 16), dtype=torch.uint8, device="cuda")
    for use_dh in (dh, None):
        dx, dres, ref = (torch.empty_like(h) for _ in range(3))
        dw, dw_ref = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        fp4.fp8_dropout_rms_norm_backward(dy, h, w, rstd, d, dx, dres, dw, ws, dh=use_dh)
        fp4.fp8_rms_norm_backward(dy, h, w, rstd, ref, dw_ref, ws, dh=use_dh)
        assert torch.equal(dres, ref) and torch.equal(dw, dw_ref)
        drop = drop_ref.dropout(dres.cpu(), p, mask)
        if dtype == "fp32":
            assert torch.equal(dx.cpu(), drop)
        else:
            assert ((dx.cpu().float() - drop).abs() <= 2.02 * 2.0 ** -8 * drop.abs()).all()
    # dx and dresidual in dh's and dy's places
    a, b = dh.clone(), dy.clone()
    fp4.fp8_dropout_rms_norm_backward(dy, h, w, rstd, d, dx, dres, dw, ws, dh=dh)
    fp4.fp8_dropout_rms_norm_backward(b, h, w, rstd, d, b, a, dw_ref, ws, dh=a)
    assert torch.equal(a, dres) and torch.equal(b, dx) and torch.equal(dw, dw_ref)


def test_norm_gradient_of_no_rows(fp4):
    e = torch.empty(0, 64, device="cuda")
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), 5.0, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    fp4.fp8_dropout_rms_norm_backward(e, e, w, torch.empty(0, device="cuda"), fp4.Dropout(0.1, 1), e, e, dw, ws)
    assert (dw == 0).all()


def test_offsets_past_32_bits(fp4):
    """The last rows of a tensor of more than 2^31 elements, bf16."""
    rows, cols = 262145, 8200
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = 1
    fp4.fp8_dropout(x, fp4.Dropout(0.5, 8), x)
    groups = cols // 8
    first = (rows - 3) * groups
    import numpy as np
    g = np.arange(first, rows * groups, dtype=np.uint64)
    zero = np.zeros_like(g)
    words = drop_ref.philox(g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), zero, zero, 8, 0)
    half = np.stack([v for w in words for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
    keep = torch.from_numpy(half.reshape(3, cols) >= 32768)
    assert torch.equal(x[-3:].cpu().float(), keep.float() * 2)
    assert int((x[:-3] != 0).sum()) == 0
