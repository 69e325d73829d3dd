"""GPU: how many adapters are loaded says nothing about a token's results; that the caller says
the tokens' adapters are mixed changes the kernels and not the results' bounds (lora_ref.py)."""
import pytest
import torch

from lora_ref import Problem, check, product_tol

pytestmark = pytest.mark.gpu


def run(fp4, q, count, fast, mixed):
    """Both passes with the first `count` adapters loaded, in workspaces of their size."""
    l = fp4.LoraAdapters.wrap(q.a[:count].contiguous(), q.b[:count].contiguous(), q.scale[:count].contiguous(), q.K)
    y, dx = (torch.empty(q.M, n, dtype=torch.bfloat16, device="cuda") for n in (q.N, q.K))
    da, db = torch.empty(l.a.shape, device="cuda"), torch.empty(l.b.shape, device="cuda")
    how = dict(fast=fast, mixed=mixed)
    for n, call in ((fp4.fp8_lora_fprop_ws_bytes(q.M, q.N, q.K, q.rank, **how),
                     lambda ws: fp4.fp8_lora_fprop(q.x, q.w, l, y, index=q.index, drop=q.drop, ws=ws, **how)),
                    (fp4.fp8_lora_backward_ws_bytes(q.M, q.N, q.K, q.rank, count, **how),
                     lambda ws: fp4.fp8_lora_backward(q.dy, q.w_t, q.x, l, dx, da, db, ws, index=q.index, drop=q.drop,
                                                      **how))):
        buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        call(buf[:n])
        assert (buf[n:] == 0xA5).all()
    return y, dx, da[:, :, :q.K], db


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("M,N,K,rank", [(1, 520, 5120, 16), (8, 5120, 2600, 16), (64, 512, 5120, 64), (70, 300, 2600, 16),
                                        (128, 5120, 5120, 16), (130, 5120, 5120, 64), (256, 520, 2600, 8),
                                        (300, 600, 1030, 16), (512, 520, 2600, 64)])
def test_results_do_not_depend_on_the_adapters_loaded(fp4, M, N, K, rank, fast, mixed):
    """Tokens of the first two of 2 to 100 adapters: the same to the last bit."""
    q = Problem(fp4, M, N, K, rank, 100, "one", 0.1, seed=M)
    q.index[:] = (torch.arange(M, device="cuda") % 3).int() - 1
    first = run(fp4, q, 2, fast, mixed)
    for count in (15, 16, 100):
        for name, a, b in zip(("y", "dx", "da", "db"), first, run(fp4, q, count, fast, mixed)):
            assert torch.equal(a, b[:2] if name in ("da", "db") else b), (name, count)


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("M,N,K,rank,count,spread,p", [
    (65, 130, 100, 16, 3, "mixed", 0.0), (100, 300, 1001, 40, 30, "mixed", 0.25), (129, 64, 2000, 128, 2, "runs", 0.0),
    (300, 264, 1000, 16, 20, "mixed", 0.1), (511, 77, 300, 8, 200, "mixed", 0.0), (512, 520, 130, 24, 1, "one", 0.1),
    (513, 100, 260, 16, 40, "mixed", 0.1)])
def test_mixed(fp4, M, N, K, rank, count, spread, p, fast):
    q = Problem(fp4, M, N, K, rank, count, spread, p, seed=M)
    y, dx, da, db = run(fp4, q, count, fast, True)
    want, tol = q.forward()
    check(y, want, tol + product_tol(q.x, q.w, fast, want.device), "y")
    want, tol = q.backward()
    check(dx, want[0], tol[0] + product_tol(q.dy, q.w_t, fast, want[0].device), "dx")
    check(da, want[1], tol[1], "da")
    check(db, want[2], tol[2], "db")


def test_a_wide_result(fp4):
    """512 mixed tokens beside 8.4 million columns, more groups of 256 columns of a token than a
    launch has room for: y = t b with t = 1 and a b of few bits, W = 0."""
    M, N, K = 512, 8400000, 8
    x, w = fp4.Fp8Tensor(M, K), fp4.Fp8Tensor(N, K, True)
    for q in (x, w):
        q.codes.zero_()
        q.scales.fill_(127)
    x.codes[:, 0] = 0x38  # 1
    l = fp4.LoraAdapters(16, 8, N, K)
    l.a[:, 0, 0] = 1
    l.b[:, :, 0] = (torch.arange(N, device="cuda") % 251).bfloat16()
    index = (torch.arange(M, device="cuda") % 17).int()  # every seventeenth has none
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fp4.fp8_lora_fprop_ws_bytes(M, N, K, 8, mixed=True), dtype=torch.uint8, device="cuda")
    fp4.fp8_lora_fprop(x, w, l, y, index=index, ws=ws, mixed=True)
    assert (y[index == 16] == 0).all()
    for m in (0, 1, 255, 510):
        assert torch.equal(y[m], l.b[int(index[m]), :, 0])
