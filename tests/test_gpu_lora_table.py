"""GPU: how many adapters are loaded says nothing about a token's results."""
import pytest
import torch

from lora_ref import Problem, check, product_tol

pytestmark = pytest.mark.gpu


def run(fp4, q, count, fast):
    """Both passes with the first `count` adapters loaded."""
    l = fp4.LoraAdapters.wrap(q.a[:count].contiguous(), q.b[:count].contiguous(), q.scale[:count].contiguous(), q.K)
    y, dx = (torch.empty(q.M, n, dtype=torch.bfloat16, device="cuda") for n in (q.N, q.K))
    da, db = torch.empty(l.a.shape, device="cuda"), torch.empty(l.b.shape, device="cuda")
    ws = torch.empty(max(fp4.fp8_lora_fprop_ws_bytes(q.M, q.N, q.K, q.rank, fast=fast),
                         fp4.fp8_lora_backward_ws_bytes(q.M, q.N, q.K, q.rank, count, fast=fast)), dtype=torch.uint8,
                     device="cuda")
    fp4.fp8_lora_fprop(q.x, q.w, l, y, index=q.index, drop=q.drop, ws=ws, fast=fast)
    fp4.fp8_lora_backward(q.dy, q.w_t, q.x, l, dx, da, db, ws, index=q.index, drop=q.drop, fast=fast)
    return y, dx, da[:2, :, :q.K], db[:2]


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("M,N,K,rank", [(1, 520, 5120, 16), (8, 5120, 2600, 16), (64, 512, 5120, 64), (70, 300, 2600, 16),
                                        (128, 5120, 5120, 16), (130, 5120, 5120, 64), (256, 520, 2600, 8),
                                        (300, 600, 1030, 16), (512, 520, 2600, 64)])
def test_results_do_not_depend_on_the_adapters_loaded(fp4, M, N, K, rank, fast):
    """Tokens of the first two of 1 to 100 adapters: the same to the last bit."""
    q = Problem(fp4, M, N, K, rank, 100, "one", 0.1, seed=M)
    q.index[:] = (torch.arange(M, device="cuda") % 3).int() - 1
    first = run(fp4, q, 2, fast)
    for count in (15, 16, 100):
        for name, a, b in zip(("y", "dx", "da", "db"), first, run(fp4, q, count, fast)):
            assert torch.equal(a, b), (name, count)
