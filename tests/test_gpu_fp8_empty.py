"""Empty sums: every output that has elements is written, with what a sum of nothing gives."""
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import BF16, full, rnd

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("fast", [False, True], ids=["binary32", "fast"])


def e(*s):
    return torch.full(s, 7.0, dtype=BF16, device="cuda")


@KINDS
@pytest.mark.parametrize("M,F", [(5, 300), (70, 300), (2500, 4096), (2500, 4001), (0, 300), (70, 0)])
def test_block_of_no_width(fp4, M, F, fast):
    """K = 0: g, u and h are zeros, as products of no terms; there is no y."""
    Q = fp4.Fp8Tensor
    hq, g, u = full(Q(M, F)), e(M, F), e(M, F)
    ws = torch.empty(max(fp4.fp8_ffn_ws_bytes(M, 0, F), 16), dtype=torch.uint8, device="cuda")
    w = Q(F, 0, True), Q(F, 0, True), Q(0, F, True)
    fp4.fp8_ffn_fprop(Q(M, 0), *w, hq, e(M, 0), g=g, u=u, ws=ws, fast=fast)
    assert (g == 0).all() and (u == 0).all() and (hq.codes & 0x7F == 0).all()
    assert (hq.scales[:, :M] == 127).all()
    h2 = full(Q(M, F))
    fp4.fp8_ffn_fprop(Q(M, 0), *w, h2, e(M, 0), ws=ws, fast=fast)
    assert (h2.codes & 0x7F == 0).all()


@KINDS
def test_backward_of_no_width(fp4, fast):
    M, F = 70, 304
    Q = fp4.Fp8Tensor
    g, u = rnd(M, F), rnd(M, F, seed=1)
    bufs = fp4.FfnBuffers(M, 0, F)
    for n in ("dgq", "duq", "dgq_t", "duq_t", "hq_t"):
        full(getattr(bufs, n))
    ws = torch.empty(max(fp4.fp8_ffn_ws_bytes(M, 0, F), 16), dtype=torch.uint8, device="cuda")
    fp4.fp8_ffn_backward(Q(M, 0), Q(0, M), Q(0, M), Q(0, F, True), Q(0, F, True), Q(F, 0, True), g.cuda(), u.cuda(), bufs,
                         e(M, 0), e(F, 0), e(F, 0), e(0, F), ws=ws, fast=fast)
    for n in ("dgq", "duq", "dgq_t", "duq_t"):
        assert (getattr(bufs, n).codes & 0x7F == 0).all(), n
    gd, ud = g.double(), u.double()
    h = (ref.silu(gd) * ud).t()
    ref.assert_near(bufs.hq_t, h, h.abs() * ((1.5 * gd.abs() + 16) * 2.0 ** -24).t(), "h_t")


@KINDS
def test_block_of_no_inner_width(fp4, fast):
    M, K = 70, 200
    Q = fp4.Fp8Tensor
    ws = torch.empty(max(fp4.fp8_ffn_ws_bytes(M, K, 0), 16), dtype=torch.uint8, device="cuda")
    y = e(M, K)
    fp4.fp8_ffn_fprop(Q(M, K), Q(0, K, True), Q(0, K, True), Q(K, 0, True), Q(M, 0), y, ws=ws, fast=fast)
    assert (y == 0).all()
    dx = e(M, K)
    fp4.fp8_ffn_backward(Q(M, K), Q(K, M), Q(K, M), Q(K, 0, True), Q(K, 0, True), Q(0, K, True), e(M, 0), e(M, 0),
                         fp4.FfnBuffers(M, K, 0), dx, e(0, K), e(0, K), e(K, 0), ws=ws, fast=fast)
    assert (dx == 0).all()
