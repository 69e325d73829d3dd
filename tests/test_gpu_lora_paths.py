"""GPU: the product's kernels that begin with the adapters' part, each tile with and without K
parts, with several adapters and tokens without one, and with a dropout of dx's part; on the
same paths an adapter's infinities (the tolerances are derived in lora_ref.py)."""
import pytest
import torch

from lora_paths import PATHS
from lora_ref import Problem, check, product_tol
from test_gpu_lora import backward, fprop

pytestmark = pytest.mark.gpu

# adapters, which tokens have them, rank, dropout
BATCHES = [(3, "mixed", 16, 0.1), (4, "runs", 40, 0.1), (1, "one", 8, 0.3), (5, "mixed", 24, 0.0)]


def problem(fp4, name, back, batch, **kw):
    (M, out, contraction, fast), _ = PATHS[name]
    count, spread, rank, p = batch
    N, K = (contraction, out) if back else (out, contraction)
    return Problem(fp4, M, N, K, rank, count, spread, p, seed=M + count, **kw), fast


@pytest.mark.parametrize("batch", BATCHES, ids=str)
@pytest.mark.parametrize("name", PATHS)
def test_forward(fp4, name, batch):
    q, fast = problem(fp4, name, False, batch)
    y, (want, tol) = fprop(fp4, q, fast, extra=3), q.forward()
    check(y, want, tol + product_tol(q.x, q.w, fast, want.device), "y")


@pytest.mark.parametrize("batch", BATCHES, ids=str)
@pytest.mark.parametrize("name", PATHS)
def test_backward(fp4, name, batch):
    q, fast = problem(fp4, name, True, batch)
    got, (want, tol) = backward(fp4, q, fast, extra=3), q.backward()
    check(got[0], want[0], tol[0] + product_tol(q.dy, q.w_t, fast, want[0].device), "dx")
    check(got[1], want[1], tol[1], "da")
    check(got[2], want[2], tol[2], "db")


def nonfinite(t):
    return ~torch.isfinite(t.float())


@pytest.mark.parametrize("name", PATHS)
def test_an_infinity_of_b_stays_in_its_rows_and_columns(fp4, name):
    """Rows of adapter 1 have an infinity or NaN in every column whose b has one, and everything
    else is the same to the last bit."""
    q, fast = problem(fp4, name, False, (3, "mixed", 16, 0.0))
    clean = fprop(fp4, q, fast)
    q.b[1, 3::5, 2], q.b[1, 8::10, 9] = float("inf"), float("nan")
    y, hit = fprop(fp4, q, fast), torch.zeros(q.M, q.N, dtype=torch.bool, device="cuda")
    hit[:, 3::5] = (q.index == 1)[:, None]
    assert torch.equal(nonfinite(y), hit) and torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("name", PATHS)
def test_an_infinity_of_a_stays_in_its_rows_and_columns(fp4, name, p):
    """The same of a in dx; what the dropout takes has nothing of it."""
    import drop_ref
    q, fast = problem(fp4, name, True, (3, "mixed", 16, p))
    clean = backward(fp4, q, fast)
    q.a[1, 2, 3:q.K:5], q.a[1, 9, 8:q.K:10] = float("inf"), float("nan")
    dx, da, db = backward(fp4, q, fast)
    hit = torch.zeros(q.M, q.K, dtype=torch.bool, device="cuda")
    hit[:, 3::5] = (q.index == 1)[:, None]
    if p:
        hit &= drop_ref.keep(q.M, q.K, p, q.seed, q.offset).cuda()
    assert torch.equal(nonfinite(dx), hit) and torch.equal(dx[~hit], clean[0][~hit])
    assert torch.equal(da, clean[1])  # of dt and x alone
    assert torch.equal(db[0], clean[2][0]) and torch.equal(db[2], clean[2][2]) and nonfinite(db[1]).any()
