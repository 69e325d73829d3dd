"""GPU: low-rank adapters beside a projection, forward and gradients, against binary64 (the
tolerances are derived in lora_ref.py)."""
import pytest
import torch

from fp8_paths import PRODUCTS
from lora_ref import Problem, check, product_tol

pytestmark = pytest.mark.gpu


def ws_of(n):
    """A workspace of exactly n bytes with a fence behind it."""
    buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[:n], buf[n:]


def fprop(fp4, q, fast, extra=0, index=True):
    buf = torch.full((q.M, q.N + extra), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:, :q.N]
    ws, fence = ws_of(fp4.fp8_lora_fprop_ws_bytes(q.M, q.N, q.K, q.rank, fast=fast))
    fp4.fp8_lora_fprop(q.x, q.w, q.lora, y, index=q.index if index else None, drop=q.drop, ws=ws, fast=fast)
    assert (fence == 0xA5).all() and (buf[:, q.N:] == 7.0).all()
    return y


def backward(fp4, q, fast, extra=0, index=True):
    buf = torch.full((q.M, q.K + extra), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = buf[:, :q.K]
    da, db = torch.full(q.a.shape, 9.0, device="cuda"), torch.full(q.b.shape, 9.0, device="cuda")
    ws, fence = ws_of(fp4.fp8_lora_backward_ws_bytes(q.M, q.N, q.K, q.rank, q.count, fast=fast))
    fp4.fp8_lora_backward(q.dy, q.w_t, q.x, q.lora, dx, da, db, ws, index=q.index if index else None, drop=q.drop,
                          fast=fast)
    assert (fence == 0xA5).all() and (buf[:, q.K:] == 7.0).all()
    assert (da[:, :, q.K:] == 0).all()
    return dx, da[:, :, :q.K], db


def check_forward(fp4, q, fast, **kw):
    y, (want, tol) = fprop(fp4, q, fast, **kw), q.forward()
    check(y, want, tol + product_tol(q.x, q.w, fast, want.device), "y")


def check_backward(fp4, q, fast, **kw):
    got, (want, tol) = backward(fp4, q, fast, **kw), q.backward()
    check(got[0], want[0], tol[0] + product_tol(q.dy, q.w_t, fast, want[0].device), "dx")
    check(got[1], want[1], tol[1], "da")
    check(got[2], want[2], tol[2], "db")


# M, N, K, rank, adapters, which tokens have them, dropout
CASES = [(1, 64, 128, 8, 1, "one", 0.0), (1, 130, 100, 16, 3, "mixed", 0.0), (1, 1, 1, 8, 2, "one", 0.5),
         (5, 77, 300, 8, 4, "mixed", 0.0), (8, 520, 2600, 16, 8, "mixed", 0.0), (16, 64, 64, 128, 16, "mixed", 0.2),
         (17, 129, 640, 24, 5, "mixed", 0.0), (33, 257, 1001, 40, 16, "mixed", 0.1), (64, 512, 1024, 64, 100, "mixed", 0.0),
         (130, 300, 333, 56, 2, "runs", 0.0), (200, 100, 129, 8, 1, "none", 0.3), (300, 264, 1000, 16, 7, "runs", 0.0),
         (300, 265, 1003, 96, 7, "runs", 0.25), (513, 700, 520, 32, 1, "one", 0.05), (700, 130, 200, 120, 3, "mixed", 0.0),
         (1000, 257, 1001, 8, 40, "mixed", 0.4), (300, 264, 1000, 16, 20, "mixed", 0.1), (500, 77, 300, 128, 16, "runs", 0.0)]


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("M,N,K,rank,count,spread,p", CASES)
def test_fprop(fp4, M, N, K, rank, count, spread, p, fast):
    q = Problem(fp4, M, N, K, rank, count, spread, p, seed=M)
    check_forward(fp4, q, fast, extra=(0, 3, 8)[M % 3])


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("M,N,K,rank,count,spread,p", CASES)
def test_backward(fp4, M, N, K, rank, count, spread, p, fast):
    q = Problem(fp4, M, N, K, rank, count, spread, p, seed=M)
    check_backward(fp4, q, fast, extra=(0, 3, 8)[M % 3])


@pytest.mark.parametrize("name", PRODUCTS)
def test_fprop_on_every_path_of_the_product(fp4, name):
    M, N, K, fast = PRODUCTS[name][0]
    k = list(PRODUCTS).index(name)
    spread, p = ("one", "runs", "mixed")[k % 3], (0.0, 0.1)[k % 2]
    q = Problem(fp4, M, N, K, (16, 8, 40)[k % 3], 1 if spread == "one" else 3, spread, p, seed=k)
    check_forward(fp4, q, fast)


@pytest.mark.parametrize("name", PRODUCTS)
def test_backward_on_every_path_of_the_product(fp4, name):
    M, K, N, fast = PRODUCTS[name][0]  # dx's contraction is the projection's width
    k = list(PRODUCTS).index(name)
    spread, p = ("one", "runs", "mixed")[(k + 1) % 3], (0.0, 0.1)[k % 2]
    q = Problem(fp4, M, N, K, (16, 8, 40)[k % 3], 1 if spread == "one" else 3, spread, p, seed=k)
    check_backward(fp4, q, fast)


@pytest.mark.parametrize("fast", [False, True])
def test_without_an_index_every_token_has_the_first(fp4, fast):
    q = Problem(fp4, 70, 200, 300, 16, 2, "one", 0.1)
    q.index.zero_()
    check_forward(fp4, q, fast, index=False)
    check_backward(fp4, q, fast, index=False)


def test_new_adapters_add_nothing(fp4):
    q = Problem(fp4, 40, 200, 300, 16, 2)
    q.lora = fp4.LoraAdapters(2, 16, 200, 300)
    q.lora.a.normal_()
    plain = torch.empty(40, 200, dtype=torch.bfloat16, device="cuda")
    fp4.fp8_gemm(q.x, q.w, plain, torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
    assert torch.equal(fprop(fp4, q, False), plain)


@pytest.mark.parametrize("M,N,K,fast", [(20, 130, 300, False), (300, 260, 400, True), (2100, 2050, 300, True),
                                        (3900, 3896, 600, False)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_infinities_and_nans_stay_with_their_tokens(fp4, M, N, K, fast, p):
    """One adapter and one token of another hold NaNs and infinities: the other tokens' rows
    are the same to the last bit, and so are the other adapters' gradients."""
    q = Problem(fp4, M, N, K, 16, 3, "mixed", p, seed=1, dev64="cpu")
    clean = fprop(fp4, q, fast), *backward(fp4, q, fast)
    token = int((q.index == 1).nonzero()[0, 0])
    q.a[0, :, ::7] = float("nan")
    q.b[0, ::5] = float("inf")
    q.x.codes[token, :K] = 0x7F
    q.dy.codes[token, :N] = 0x7F
    y, dx, da, db = fprop(fp4, q, fast), *backward(fp4, q, fast)
    others = (q.index != 0)
    others[token] = False
    assert torch.equal(y[others], clean[0][others]) and torch.equal(dx[others], clean[1][others])
    assert torch.equal(da[2], clean[2][2]) and torch.equal(db[2], clean[3][2])
    assert y[q.index == 0].isnan().any() and y[token].isnan().all() and db[1].isnan().all()


def test_results_are_the_same_again(fp4):
    for shape in ((8, 520, 2600, 16, 8, "mixed", 0.1), (777, 500, 600, 32, 5, "runs", 0.1)):
        q = Problem(fp4, *shape)
        first = fprop(fp4, q, True), *backward(fp4, q, True)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, (fprop(fp4, q, True), *backward(fp4, q, True))))


@pytest.mark.parametrize("M,N,K", [(0, 64, 128), (5, 0, 128), (5, 64, 0), (0, 0, 0), (70, 0, 128), (70, 64, 0), (600, 64, 0)])
def test_empty(fp4, M, N, K):
    """No tokens, no outputs, no inputs: zeros where there is something to write."""
    q = Problem(fp4, M, N, K, 8, 2, "one")
    assert (fprop(fp4, q, False) == 0).all()
    dx, da, db = backward(fp4, q, False)
    assert (dx == 0).all() and (da == 0).all() and (db == 0).all()


@pytest.mark.parametrize("rows", [8, 40, 70])
def test_the_last_rows_of_a_large_product(fp4, rows):
    """Binary32 sums of whole rounds of large tiles and a tail of few rows."""
    q = Problem(fp4, 16384 + rows, 4000, 700, 8, 2, "runs", 0.0, seed=3)
    check_forward(fp4, q, False)
    q = Problem(fp4, 16384 + rows, 700, 4000, 8, 2, "runs", 0.1, seed=4)
    check_backward(fp4, q, False)


@pytest.mark.parametrize("M,N,K,rank,count,spread", [(20000, 96, 160, 8, 300, "mixed"), (600, 200, 130, 16, 1000, "mixed"),
                                                     (20, 300, 200, 8, 3000, "mixed"), (9000, 130, 72, 24, 4, "runs")])
def test_many_tokens_and_adapters(fp4, M, N, K, rank, count, spread):
    q = Problem(fp4, M, N, K, rank, count, spread, 0.1, seed=2)
    check_forward(fp4, q, False)
    check_backward(fp4, q, False)


def test_adapters_far_behind_each_other(fp4):
    """Offsets past 2^31 elements: the last adapters of many, and the same among the last 20 (the
    number of adapters has a part in which kernels run, and at 20 and at 500 they are the same)."""
    N, K, rank, count = 20000, 17000, 128, 500
    a = torch.zeros(count, rank, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(count, N, rank, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    a[-2:].normal_(generator=gen)
    b[-2:].normal_(generator=gen)
    scale = torch.ones(count, device="cuda")
    for M in (3, 70, 600):
        index = torch.full((M,), count - 1, dtype=torch.int32, device="cuda")
        index[1] = count - 2
        xs = torch.randn(M, K, generator=gen, device="cuda")
        x, w = fp4.Fp8Tensor(M, K), fp4.Fp8Tensor(N, K, True)
        fp4.fp8_quantize(xs, x)
        w.codes.zero_()
        w.scales.fill_(127)
        y, z = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ws = torch.empty(fp4.fp8_lora_fprop_ws_bytes(M, N, K, rank), dtype=torch.uint8, device="cuda")
        fp4.fp8_lora_fprop(x, w, fp4.LoraAdapters.wrap(a, b, scale, K), y, index=index, ws=ws)
        near = fp4.LoraAdapters.wrap(a[-20:].contiguous(), b[-20:].contiguous(), scale[-20:].contiguous(), K)
        fp4.fp8_lora_fprop(x, w, near, z, index=index - (count - 20), ws=ws)
        assert torch.equal(y, z) and float(y.float().abs().mean()) > 1


def test_side_stream_and_graph(fp4):
    """On a stream of its own, and captured: replays follow the index, the adapters and the
    step as they are then, two graphs with workspaces of their own."""
    q = Problem(fp4, 24, 300, 500, 16, 4, "mixed", 0.1)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    q.drop = fp4.Dropout(0.1, q.seed, q.offset, step)
    outs = []
    for k in range(2):
        y, dx = (torch.empty(24, n, dtype=torch.bfloat16, device="cuda") for n in (300, 500))
        da, db = torch.empty(q.a.shape, device="cuda"), torch.empty(q.b.shape, device="cuda")
        wf = torch.empty(fp4.fp8_lora_fprop_ws_bytes(24, 300, 500, 16), dtype=torch.uint8, device="cuda")
        wb = torch.empty(fp4.fp8_lora_backward_ws_bytes(24, 300, 500, 16, 4), dtype=torch.uint8, device="cuda")

        def go():
            fp4.fp8_lora_fprop(q.x, q.w, q.lora, y, index=q.index, drop=q.drop, ws=wf)
            fp4.fp8_lora_backward(q.dy, q.w_t, q.x, q.lora, dx, da, db, wb, index=q.index, drop=q.drop)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            go()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go()
        outs.append((g, y, dx, da, db, wf, wb))
    for i in range(3):
        step.fill_(i)
        q.index.copy_(q.index.roll(1))
        q.b.mul_(0.5)
        for g, *_ in outs:
            g.replay()
        torch.cuda.synchronize()
        q.offset += 1 if i else 0
        eager = Problem.__new__(Problem)
        eager.__dict__.update(q.__dict__)
        eager.drop = fp4.Dropout(0.1, q.seed, q.offset)
        want = fprop(fp4, eager, False), *backward(fp4, eager, False)
        for _, y, dx, da, db, *_ in outs:
            for a, b in zip((y, dx, da[:, :, :500], db), want):
                assert torch.equal(a, b)
