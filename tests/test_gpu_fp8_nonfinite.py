"""The gated block's backward pass where a token or a few values are not finite: the
others' tensors are what they are without them, to the bit (no tolerance)."""
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import BF16, full, rnd, weights

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("fast", [False, True], ids=["binary32", "fast"])
# the last 128 columns and rows hold 40 and 68, and `fast` takes the fused kernel
M, K, F = 2500, 136, 4008
NAMES = ("dgq", "duq", "dgq_t", "duq_t", "hq_t")


@pytest.fixture(scope="module")
def block(fp4):
    w = [ref.transposed(fp4, q) for q in weights(fp4, K, F)]
    x_t = ref.put(fp4, rnd(M, K, seed=8).t())
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda")

    def run(dy, g, u, fast, edit=lambda *q: None):
        dyq, dyq_t = ref.put(fp4, dy.nan_to_num(0, 0, 0)), ref.put(fp4, dy.nan_to_num(0, 0, 0).t())
        dyq.codes[:, :K][~dy.isfinite().cuda()] = 0x7F
        edit(dyq, dyq_t)
        bufs = fp4.FfnBuffers(M, K, F)
        for n in NAMES:
            full(getattr(bufs, n))
        out = [torch.empty(s, dtype=BF16, device="cuda") for s in ((M, K), (F, K), (F, K), (K, F))]
        fp4.fp8_ffn_backward(dyq, dyq_t, x_t, *w, g.cuda(), u.cuda(), bufs, *out, ws=ws, fast=fast)
        return bufs, out

    return run


def inputs():
    return rnd(M, K, seed=9, std=1e-3), rnd(M, F, seed=10), rnd(M, F, seed=11)


@KINDS
@pytest.mark.parametrize("which", ["dy", "g", "u"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=str)
def test_a_token_leaves_the_others(block, which, value, fast):
    """Token 101: the padding stays zeros, and the other tokens' dg, du and dx their own."""
    dy, g, u = inputs()
    base, out = block(dy, g, u, fast)
    {"dy": dy, "g": g, "u": u}[which][101] = value
    bufs, got = block(dy, g, u, fast)
    keep = torch.arange(M, device="cuda") != 101
    for n in ("dgq", "duq"):
        a, b = getattr(bufs, n), getattr(base, n)
        assert (a.codes[:, F:] == 0).all(), f"{n}: padding"
        assert torch.equal(a.codes[keep], b.codes[keep]), n
        assert torch.equal(a.scales[:, :M][:, keep], b.scales[:, :M][:, keep]), n
    assert torch.equal(got[0][keep], out[0][keep])


@KINDS
@pytest.mark.parametrize("rows", [1, 4, 127], ids=["one", "four", "block"])
def test_nans_of_a_column_leave_its_blocks_other_tokens(block, rows, fast):
    """NaNs of u in tokens 128 .. of column 40 (four neighbours are one thread's share of the
    column) are NaN codes of dg and h there; every other code and every scale but that
    block's is what it was, and that block's is the other tokens' own."""
    dy, g, u = inputs()
    u[128:128 + rows, 40] = 0.0  # adds nothing to a block's maximum, as a NaN should
    base, _ = block(dy, g, u, fast)
    u[128:128 + rows, 40] = float("nan")
    bufs, _ = block(dy, g, u, fast)
    keep = torch.ones(M, F, dtype=torch.bool, device="cuda")
    keep[128:128 + rows, 40] = False
    for n in NAMES:
        a, b, k = getattr(bufs, n), getattr(base, n), keep if n in ("dgq", "duq") else keep.t()
        assert torch.equal(a.codes[:, :k.shape[1]][k], b.codes[:, :k.shape[1]][k]), n
        assert torch.equal(a.scales[:, :k.shape[0]], b.scales[:, :k.shape[0]]), n
        if n in ("dgq", "dgq_t", "hq_t"):
            assert (a.codes[:, :k.shape[1]][~k] & 0x7F == 0x7F).all(), n


@KINDS
@pytest.mark.parametrize("inner", [F, 4001, 3968], ids=str)
@pytest.mark.parametrize("tokens", [5, 100, M])
def test_forward_of_a_token_leaves_the_others(fp4, tokens, inner, fast):
    """A NaN in token 3: its y is NaN, h's padding stays zeros, the other tokens their own."""
    w = weights(fp4, K, inner)
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(tokens, K, inner), dtype=torch.uint8, device="cuda")
    x = ref.put(fp4, rnd(tokens, K, seed=8))
    runs = []
    for bad in (False, True):
        if bad:
            x.codes[3, 7] = 0x7F
        hq, y = full(fp4.Fp8Tensor(tokens, inner)), torch.empty(tokens, K, dtype=BF16, device="cuda")
        fp4.fp8_ffn_fprop(x, *w, hq, y, ws=ws, fast=fast)
        assert (hq.codes[:, inner:] & 0x7F == 0).all(), "padding"
        runs.append((hq.codes, hq.scales[:, :tokens].t(), y))
    keep = torch.arange(tokens, device="cuda") != 3
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(*runs))
    assert runs[1][2][3].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(6, 100), (200, 600), (131, 1000), (7, 2500), (5, 5000), (3, 8200)], ids=str)
def test_norm_of_a_token_leaves_the_padding(fp4, shape, dtype):
    """A NaN in the last token: its y is NaN, the padding of both layouts zeros, the other
    tokens their own."""
    m, n = shape
    x, w = rnd(m, n, dtype=dtype), torch.ones(n, device="cuda")
    runs = []
    for bad in (False, True):
        if bad:
            x[m - 1, 5] = float("nan")
        y, yt, rs = full(fp4.Fp8Tensor(m, n)), full(fp4.Fp8Tensor(n, m)), torch.empty(m, device="cuda")
        fp4.fp8_rms_norm(x.cuda(), w, 1e-6, y, yq_t=yt, rstd=rs)
        assert (y.codes[:, n:] & 0x7F == 0).all() and (yt.codes[:, m:] & 0x7F == 0).all(), "padding"
        runs.append((y.codes[:m - 1], y.scales[:, :m - 1], rs[:m - 1]))
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert (y.codes[m - 1, :n] & 0x7F == 0x7F).all()
