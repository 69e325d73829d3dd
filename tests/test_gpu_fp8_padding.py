"""The padding of a tensor's scales (rows past the tensor's, up to a multiple of 16) is not
read for a result: any byte there, NaN's 0xFF among them, gives the same bits."""
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import BF16, FP32, rnd, weights
from test_gpu_fp8_nonfinite import F, K, M, NAMES, block, inputs  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("fast", [False, True], ids=["binary32", "fast"])
BYTES = pytest.mark.parametrize("byte", [0, 254, 255])


def pad(q, byte):
    q.scales[:, q.rows:] = byte
    return q


@KINDS
@BYTES
@pytest.mark.parametrize("shape", [(5, 300, 400), (20, 1000, 4100), (300, 700, 900), (1030, 260, 300), (3900, 3901, 300)],
                         ids=str)
def test_products(fp4, shape, byte, fast):
    m, n, k = shape
    x, w = rnd(m, k).cuda(), rnd(n, k, seed=1).cuda()
    a, b = fp4.Fp8Tensor(m, k), fp4.Fp8Tensor(n, k)
    fp4.fp8_quantize(x, a)
    fp4.fp8_quantize(w, b)
    ws = torch.empty(max(fp4.fp8_gemm_ws_bytes(m, n, k), 16), dtype=torch.uint8, device="cuda")
    for dtype in (FP32, BF16):
        want, got = (torch.empty(m, n, dtype=dtype, device="cuda") for _ in range(2))
        fp4.fp8_gemm(pad(a, 127), pad(b, 127), want, ws, fast=fast)
        fp4.fp8_gemm(pad(a, byte), pad(b, byte), got, ws, fast=fast)
        assert torch.equal(got, want)


@KINDS
@BYTES
@pytest.mark.parametrize("tokens", [5, 100, M])
def test_block_forward(fp4, tokens, byte, fast):
    w = weights(fp4, K, F)
    x = ref.put(fp4, rnd(tokens, K, seed=8))
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(tokens, K, F), dtype=torch.uint8, device="cuda")
    outs = []
    for b in (127, byte):
        hq, y = fp4.Fp8Tensor(tokens, F), torch.empty(tokens, K, dtype=BF16, device="cuda")
        fp4.fp8_ffn_fprop(pad(x, b), *w, hq, y, ws=ws, fast=fast)
        outs.append((hq.codes, hq.scales[:, :tokens], y))
    assert all(torch.equal(p, q) for p, q in zip(*outs))


@KINDS
@BYTES
def test_block_backward(block, byte, fast):  # noqa: F811
    assert M % 16 and K % 16
    base, want = block(*inputs(), fast)
    bufs, got = block(*inputs(), fast, lambda *qs: [pad(q, byte) for q in qs])
    for n in NAMES:
        a, b = getattr(bufs, n), getattr(base, n)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales[:, :a.rows], b.scales[:, :b.rows]), n
    assert all(torch.equal(p, q) for p, q in zip(got, want))
