"""GPU parity of the 8-bit operators' large and split paths at the sizes of fp8_paths.py
(test_fp8_plan.py checks that they get there), on sampled rows of each result: both sides
of tiles', launches' and the tensor's ends.  Tolerances as in test_gpu_fp8_block.py."""
import pytest
import torch

import fp8_paths as paths
import fp8_ref as ref
from test_gpu_fp8 import BF16, FP32, act_rel, full, rnd, rows_of
from test_gpu_fp8_block import check

pytestmark = pytest.mark.gpu


def sample(m):
    """Rows on both sides of multiples of 64 that matter, spread over m rows."""
    at = {0, 64, 128, 256, m // 2 // 256 * 256, (m - 1) // 256 * 256, (m - 1) // 128 * 128, 16384, m}
    return sorted({r for a in at for r in range(a - 3, a + 4) if 0 <= r < m})


def some(q):
    """(rows, the tensor of those rows on the CPU)"""
    r = sample(q.rows)
    return r, rows_of(q, r)


def on_cpu(fp4, q):
    t = fp4.Fp8Tensor(q.rows, q.cols, q.two_d, device="cpu")
    t.codes.copy_(q.codes)
    t.scales.copy_(q.scales)
    return t


def quantized(fp4, x, two_d=False):
    """The library's quantization (test_quantize holds it to the definition), which is
    quicker than the reference's at these sizes."""
    q = fp4.Fp8Tensor(*x.shape, two_d)
    fp4.fp8_quantize(x, q)
    return q


def weights(fp4, K, F):
    """wg, wu, wd and their transposes"""
    w = [rnd(F, K, seed=5, std=K ** -0.5), rnd(F, K, seed=6, std=K ** -0.5), rnd(K, F, seed=7, std=F ** -0.5)]
    q, t = [fp4.Fp8Tensor(*x.shape, True) for x in w], [fp4.Fp8Tensor(x.shape[1], x.shape[0], True) for x in w]
    for x, a, b in zip(w, q, t):
        fp4.fp8_quantize(x.cuda(), a, b)
    return q, t


def both(fp4, x):
    """x and x^T, quantized"""
    q, t = fp4.Fp8Tensor(*x.shape), fp4.Fp8Tensor(x.shape[1], x.shape[0])
    fp4.fp8_quantize(x.cuda(), q, t)
    return q, t


def nans(*shape):
    return torch.full(shape, float("nan"), dtype=BF16, device="cuda")


@pytest.mark.parametrize("name", paths.PRODUCTS)
def test_products(fp4, name):
    (M, N, K, fast), _ = paths.PRODUCTS[name]
    a, b = quantized(fp4, rnd(M, K, std=0.5).cuda()), quantized(fp4, rnd(N, K, seed=1, std=0.02).cuda())
    ws = torch.empty(max(fp4.fp8_gemm_ws_bytes(M, N, K), 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    rows, part = some(a)
    cols = rows_of(b, list(range(N)))
    for dtype in (FP32, BF16):
        c = torch.full((M + 1, N), -7.0, dtype=dtype, device="cuda")
        fp4.fp8_gemm(a, b, c[:M], ws, fast=fast)
        check(c[rows], part, cols, fast, f"{dtype}", bf16=dtype == BF16)
        assert (c[M] == -7.0).all(), "past the last row"
        assert not (c[:M] == -7.0).all(1).any(), "a row that no launch wrote"


def as_rows(fp4, q, rows):
    """Rows of a tile-scaled tensor as a 1 x 128-scaled one on the CPU (the same values)."""
    t = fp4.Fp8Tensor(len(rows), q.cols, device="cpu")
    t.codes.copy_(q.codes[rows])
    t.scales.fill_(127)
    t.scales[:, :len(rows)] = q.scales.cpu()[:, torch.tensor(rows) // 128]
    return t


@pytest.mark.parametrize("kinds", [(False, True), (True, False), (True, True)], ids=["1d2d", "2d1d", "2d2d"])
@pytest.mark.parametrize("name", [n for n in paths.PRODUCTS if "256" in n or "128x" in n])
def test_products_of_tile_scales(fp4, name, kinds):
    (M, N, K, fast), _ = paths.PRODUCTS[name]
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    x, w = (torch.randn(r, K, generator=gen, device="cuda") for r in (M, N))
    for t in (x, w):  # blocks of many magnitudes, so that a wrong tile's scale shows
        t *= torch.exp2(torch.randint(-6, 7, (-(-t.shape[0] // 128), -(-K // 128)), generator=gen, device="cuda").float()
                        ).repeat_interleave(128, 0)[:t.shape[0]].repeat_interleave(128, 1)[:, :K]
    a, b = quantized(fp4, x, kinds[0]), quantized(fp4, w, kinds[1])
    ws = torch.empty(max(fp4.fp8_gemm_ws_bytes(M, N, K), 16), dtype=torch.uint8, device="cuda")
    c = torch.empty(M, N, device="cuda")
    fp4.fp8_gemm(a, b, c, ws, fast=fast)
    rows, cols = sample(M), sample(N)
    part = [as_rows(fp4, q, r) if q.two_d else rows_of(q, r) for q, r in ((a, rows), (b, cols))]
    check(c[rows][:, cols], *part, fast, name, bf16=False)


@pytest.mark.parametrize("fast", [False, True], ids=["binary32", "fast"])
@pytest.mark.parametrize("shape", [(300, 1, 257), (1, 300, 1), (5000, 3, 1000), (2, 5000, 100), (129, 1, 1), (64, 65, 127),
                                   (70000, 17, 130)], ids=str)
def test_thin_products(fp4, shape, fast):
    M, N, K = shape
    a, b = quantized(fp4, rnd(M, K).cuda()), quantized(fp4, rnd(N, K, seed=1).cuda())
    ws = torch.empty(max(fp4.fp8_gemm_ws_bytes(M, N, K), 16), dtype=torch.uint8, device="cuda")
    for dtype in (FP32, BF16):
        c = torch.full((M, N + 1), -7.0, dtype=dtype, device="cuda")
        fp4.fp8_gemm(a, b, c[:, :N], ws, fast=fast)
        check(c[:, :N], rows_of(a, list(range(M))), rows_of(b, list(range(N))), fast, str(dtype), bf16=dtype == BF16)
        assert (c[:, N] == -7.0).all()


@pytest.mark.parametrize("name", paths.FORWARD)
def test_forward(fp4, name):
    (M, K, F, fast), _ = paths.FORWARD[name]
    (wg, wu, wd), _ = weights(fp4, K, F)
    x = quantized(fp4, rnd(M, K, seed=8).cuda())
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda").fill_(0xFF)
    hq, y, g, u = full(fp4.Fp8Tensor(M, F)), nans(M, K), nans(M, F), nans(M, F)
    fp4.fp8_ffn_fprop(x, wg, wu, wd, hq, y, g=g, u=u, ws=ws, fast=fast)
    rows, part = some(x)
    check(g[rows], part, on_cpu(fp4, wg), fast, "g")
    check(u[rows], part, on_cpu(fp4, wu), fast, "u")
    gd, ud = g[rows].cpu().double(), u[rows].cpu().double()
    h = ref.silu(gd) * ud
    ref.assert_near(rows_of(hq, rows), h, h.abs() * act_rel(gd), "h")
    check(y[rows], rows_of(hq, rows), on_cpu(fp4, wd), fast, "y")
    assert y.isfinite().all() and g.isfinite().all() and u.isfinite().all()


@pytest.mark.parametrize("name", paths.BACKWARD)
def test_backward(fp4, name):
    """The products' results, each against its own operands (test_gpu_fp8_block.py covers
    the step between them)."""
    (M, K, F, fast), *_ = paths.BACKWARD[name]
    _, (wg_t, wu_t, wd_t) = weights(fp4, K, F)
    dyq, dyq_t = both(fp4, rnd(M, K, seed=9, std=1e-3))
    _, x_t = both(fp4, rnd(M, K, seed=8))
    g, u = rnd(M, F, seed=10, std=2.0), rnd(M, F, seed=11)
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda").fill_(0xFF)
    bufs = fp4.FfnBuffers(M, K, F)
    dx, dwg, dwu, dwd = nans(M, K), nans(F, K), nans(F, K), nans(K, F)
    fp4.fp8_ffn_backward(dyq, dyq_t, x_t, wg_t, wu_t, wd_t, g.cuda(), u.cuda(), bufs, dx, dwg, dwu, dwd, ws=ws, fast=fast)
    rows = sample(M)
    dh, bound = ref.product(rows_of(dyq, rows), on_cpu(fp4, wd_t))
    off = 1e-5 * bound + (ref.cut(rows_of(dyq, rows), on_cpu(fp4, wd_t)) if fast else 0)
    gd = g[rows].double()
    ref.assert_near(rows_of(bufs.duq, rows), dh * ref.silu(gd), ref.silu(gd).abs() * (off + dh.abs() * act_rel(gd)), "du")
    check(dx[rows], rows_of(bufs.dgq, rows), on_cpu(fp4, wg_t), fast, "dx", (rows_of(bufs.duq, rows), on_cpu(fp4, wu_t)))
    inner, across = sample(F), list(range(K))
    check(dwg[inner], rows_of(bufs.dgq_t, inner), rows_of(x_t, across), fast, "dwg")
    check(dwu[inner], rows_of(bufs.duq_t, inner), rows_of(x_t, across), fast, "dwu")
    across = sample(K)
    check(dwd[across], rows_of(dyq_t, across), rows_of(bufs.hq_t, list(range(F))), fast, "dwd")
    assert all(t.isfinite().all() for t in (dx, dwg, dwu, dwd))
