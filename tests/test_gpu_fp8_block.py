"""GPU parity of the gated block by kind of sums: binary32 ones within the framework's
tolerance for products (1e-5 sum |a b| and half a bf16 step, parity.check_gemm), and the
8-bit matrix instruction's within what it cuts off besides (fp8_ref.check_fast)."""
import pytest
import torch

import fp8_ref as ref
from parity import check_gemm
from test_gpu_fp8 import BF16, FSHAPES, act_rel, full, rnd, weights

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("fast", [False, True], ids=["binary32", "fast"])


def check(c, a, b, fast, what, more=None, bf16=True):
    if fast:
        return ref.check_fast(c, a, b, what, more)
    want, bound = (sum(t) for t in zip(*(ref.product(*p) for p in [(a, b)] + ([more] if more else []))))
    check_gemm(c.float().cpu().numpy(), want.numpy(), bound.numpy(), bf16, what)


@KINDS
@pytest.mark.parametrize("shape", FSHAPES, ids=str)
def test_fprop(fp4, shape, fast):
    M, K, F = shape
    wg, wu, wd = weights(fp4, K, F)
    x = ref.put(fp4, rnd(M, K, seed=8))
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda").fill_(0xFF)
    hq, y = full(fp4.Fp8Tensor(M, F)), torch.full((M, K + 3), -7.0, dtype=BF16, device="cuda")
    g, u = (torch.full((M, F), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    fp4.fp8_ffn_fprop(x, wg, wu, wd, hq, y[:, :K], g=g, u=u, ws=ws, **({"fast": True} if fast else {}))
    check(g, x, wg, fast, "g")
    check(u, x, wu, fast, "u")
    gd, ud = g.cpu().double(), u.cpu().double()
    h = ref.silu(gd) * ud
    ref.assert_near(hq, h, h.abs() * act_rel(gd), "h")
    check(y[:, :K], hq, wd, fast, "y")
    assert (y[:, K:] == -7.0).all()
    h2, y2 = full(fp4.Fp8Tensor(M, F)), torch.empty(M, K, dtype=BF16, device="cuda")
    fp4.fp8_ffn_fprop(x, wg, wu, wd, h2, y2, ws=ws.fill_(0xFF), **({"fast": True} if fast else {}))
    assert torch.equal(h2.codes, hq.codes) and torch.equal(y2, y[:, :K]), "without g and u"


@KINDS
@pytest.mark.parametrize("shape", FSHAPES, ids=str)
def test_backward(fp4, shape, fast):
    """Each step against its own operands; dh's error is that of its product."""
    M, K, F = shape
    wg_t, wu_t, wd_t = (ref.transposed(fp4, w) for w in weights(fp4, K, F))
    dy, x = rnd(M, K, seed=9, std=1e-3), rnd(M, K, seed=8)
    dyq, dyq_t, x_t = ref.put(fp4, dy), ref.put(fp4, dy.t()), ref.put(fp4, x.t())
    g, u = rnd(M, F, seed=10, std=2.0), rnd(M, F, seed=11)
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda").fill_(0xFF)
    bufs = fp4.FfnBuffers(M, K, F)
    for q in (bufs.dgq, bufs.duq, bufs.dgq_t, bufs.duq_t, bufs.hq_t):
        full(q)
    dx, dwg, dwu, dwd = (torch.full(s, float("nan"), dtype=BF16, device="cuda") for s in ((M, K), (F, K), (F, K), (K, F)))
    fp4.fp8_ffn_backward(dyq, dyq_t, x_t, wg_t, wu_t, wd_t, g.cuda(), u.cuda(), bufs, dx, dwg, dwu, dwd, ws=ws,
                         **({"fast": True} if fast else {}))
    dh, bound = ref.product(dyq, wd_t)
    gd, ud = g.double(), u.double()
    s = torch.sigmoid(gd)
    rel, off = act_rel(gd), 1e-5 * bound + (ref.cut(dyq, wd_t) if fast else 0)
    du, dg, h = dh * ref.silu(gd), dh * ud * ref.dsilu(gd), ref.silu(gd) * ud
    e_du = ref.silu(gd).abs() * (off + dh.abs() * rel)
    e_dg = ud.abs() * (ref.dsilu(gd).abs() * off + (dh.abs() + off) * s * (1 + gd.abs() * (1 - s)) * rel)
    for q, v, e, name in ((bufs.dgq, dg, e_dg, "dg"), (bufs.duq, du, e_du, "du"), (bufs.dgq_t, dg.t(), e_dg.t(), "dg_t"),
                          (bufs.duq_t, du.t(), e_du.t(), "du_t"), (bufs.hq_t, h.t(), (h.abs() * rel).t(), "h_t")):
        ref.assert_near(q, v, e, name)
    check(dx, bufs.dgq, wg_t, fast, "dx", (bufs.duq, wu_t))
    check(dwg, bufs.dgq_t, x_t, fast, "dwg")
    check(dwu, bufs.duq_t, x_t, fast, "dwu")
    check(dwd, dyq_t, bufs.hq_t, fast, "dwd")


@pytest.mark.parametrize("M", [8, 300, 2500])
def test_sums_keep_small_products(fp4, M):
    """Groups of eight products, one of +-256 (the groups' signs alternate) beside seven of
    2^-6: binary32 holds every partial sum, and the sum is 112 * 2^-6 for every 128 of K.
    Cut off at 2^-13 of the largest of a group it would be 0."""
    K, F = 256, 4096
    row = torch.full((K,), 2.0 ** -6)
    row[::16], row[8::16] = 256.0, -256.0
    x = ref.put(fp4, row.repeat(M, 1))
    one = lambda *s: ref.put(fp4, torch.ones(*s), True)  # noqa: E731
    e = lambda *s: torch.full(s, float("nan"), dtype=BF16, device="cuda")  # noqa: E731
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda")
    g, u, y = e(M, F), e(M, F), e(M, K)
    fp4.fp8_ffn_fprop(x, one(F, K), one(F, K), one(K, F), fp4.Fp8Tensor(M, F), y, g=g, u=u, ws=ws)
    assert (g == 3.5).all() and (u == 3.5).all()
    # dh = 3.5 everywhere; with g large silu(g) = g, silu'(g) = 1
    g, u = torch.full((M, F), 64.0, dtype=BF16, device="cuda"), torch.ones(M, F, dtype=BF16, device="cuda")
    bufs = fp4.FfnBuffers(M, K, F)
    xt = ref.put(fp4, row.repeat(M, 1).t())
    fp4.fp8_ffn_backward(x, xt, xt, one(K, F), one(K, F), one(F, K), g, u, bufs, e(M, K), e(F, K), e(F, K), e(K, F), ws=ws)
    assert (ref.values(bufs.dgq) == 3.5).all() and (ref.values(bufs.duq) == 224.0).all()


def test_fast_block_in_a_graph(fp4):
    """Forward and backward through the fused kernels, captured: every replay gives the eager
    call's bits."""
    M, K, F = 2500, 256, 4096
    w = weights(fp4, K, F)
    tw = [ref.transposed(fp4, q) for q in w]
    x, dy = rnd(M, K), rnd(M, K, seed=2)
    xq, xt, dyq, dyt = ref.put(fp4, x), ref.put(fp4, x.t()), ref.put(fp4, dy), ref.put(fp4, dy.t())
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    hq, bufs = fp4.Fp8Tensor(M, F), fp4.FfnBuffers(M, K, F)
    y, g, u, dx, dwg, dwu, dwd = e(M, K), e(M, F), e(M, F), e(M, K), e(F, K), e(F, K), e(K, F)
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda")

    def step():
        fp4.fp8_ffn_fprop(xq, *w, hq, y, g=g, u=u, ws=ws, fast=True)
        fp4.fp8_ffn_backward(dyq, dyt, xt, *tw, g, u, bufs, dx, dwg, dwu, dwd, ws=ws, fast=True)

    step()
    outs = [y, dx, dwg, dwu, dwd, hq.codes, bufs.hq_t.codes]
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        step()
