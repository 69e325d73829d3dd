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
