"""Products with less than fp8_gemm_ws_bytes of workspace: K is not split, so the result is
that without a workspace to the bit, and nothing is written there."""
import pytest
import torch

from test_gpu_fp8 import rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fast", [False, True], ids=["binary32", "fast"])
@pytest.mark.parametrize("shape", [(8, 5120, 20480), (64, 1024, 8192), (300, 520, 6000), (4300, 3900, 4000)], ids=str)
def test_short_workspace_is_none(fp4, shape, fast):
    M, N, K = shape
    a, b = fp4.Fp8Tensor(M, K), fp4.Fp8Tensor(N, K)
    fp4.fp8_quantize(rnd(M, K).cuda(), a)
    fp4.fp8_quantize(rnd(N, K, seed=1).cuda(), b)
    need = fp4.fp8_gemm_ws_bytes(M, N, K)
    none, c = (torch.empty(M, N, device="cuda") for _ in range(2))
    fp4.fp8_gemm(a, b, none, fast=fast)
    ws = torch.full((need + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    # the size covers both kinds of sums; neither plan of these shapes fits in half of it
    for part in (16, need // 32 * 16, need // 64 * 16):
        fp4.fp8_gemm(a, b, c, ws[:part], fast=fast)
        assert torch.equal(c, none), f"{part} of {need} bytes"
        assert (ws == 0xA5).all(), f"{part} of {need} bytes"
    fp4.fp8_gemm(a, b, c, ws[:need], fast=fast)
    # the two orders of a sum of K normal products: fast ones are each off by 2.6e-5 of the
    # sum's deviation (K^1/2), and 15 of that are allowed between them
    assert (c - none).abs().max() <= 15 * 2.6e-5 * K ** 0.5 and (ws[need:] == 0xA5).all()


@pytest.mark.parametrize("fast", [False, True], ids=["binary32", "fast"])
@pytest.mark.parametrize("shape", [(8, 4096, 384), (40, 2000, 2600), (300, 300, 1100), (1900, 130, 2205), (2500, 136, 4008),
                                   (2500, 136, 4001), (4100, 1030, 6100)], ids=str)
def test_block_in_its_own_workspace(fp4, shape, fast):
    """Each call with exactly its own bytes gives the bits that it gives with plenty, and
    writes nothing past them."""
    M, K, F = shape
    q, t = fp4.Fp8Tensor, lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    w, wt = [q(F, K, True), q(F, K, True), q(K, F, True)], [q(K, F, True), q(K, F, True), q(F, K, True)]
    for i, (a, b) in enumerate(zip(w, wt)):
        fp4.fp8_quantize(rnd(a.rows, a.cols, seed=i, std=a.cols ** -0.5).cuda(), a, b)
    xq, xt, dyq, dyt = q(M, K), q(K, M), q(M, K), q(K, M)
    fp4.fp8_quantize(rnd(M, K, seed=4).cuda(), xq, xt)
    fp4.fp8_quantize(rnd(M, K, seed=5).cuda(), dyq, dyt)
    most = fp4.fp8_ffn_ws_bytes(M, K, F) + 4 * M * F + 4096
    ws = torch.empty(most, dtype=torch.uint8, device="cuda")

    def run(sizes):
        ws.fill_(0xA5)
        hq, y, h2, y2, g, u = q(M, F), t(M, K), q(M, F), t(M, K), t(M, F), t(M, F)
        bufs, grads = fp4.FfnBuffers(M, K, F), (t(M, K), t(F, K), t(F, K), t(K, F))
        calls = (lambda s: fp4.fp8_ffn_fprop(xq, *w, hq, y, g=g, u=u, ws=s, fast=fast),
                 lambda s: fp4.fp8_ffn_fprop(xq, *w, h2, y2, ws=s, fast=fast),
                 lambda s: fp4.fp8_ffn_backward(dyq, dyt, xt, *wt, g, u, bufs, *grads, ws=s, fast=fast))
        for call, n in zip(calls, sizes):
            ws.fill_(0xA5)
            call(ws[:n])
            assert (ws[n:] == 0xA5).all()
        assert torch.equal(y2, y) and torch.equal(h2.codes, hq.codes)
        return [y, hq.codes, g, u, *grads]

    own = (fp4.fp8_ffn_fprop_ws_bytes(M, K, F, True, fast), fp4.fp8_ffn_fprop_ws_bytes(M, K, F, False, fast),
           fp4.fp8_ffn_backward_ws_bytes(M, K, F, fast))
    assert all(torch.equal(a, b) for a, b in zip(run(own), run((most,) * 3)))
