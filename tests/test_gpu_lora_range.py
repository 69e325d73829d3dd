"""GPU: adapters whose coefficients come to the end of binary32.

t, dt and their products with a factor are binary32 values that the matrix cores take as sums
of bf16.  The inputs below have few bits, so that the results are known: powers of two times
one number, and one rounding to bf16 where the output has it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ONE, NAN_CODE = 0x38, 0x7F  # E4M3


def ones(fp4, rows, cols, two_d=False, byte=127):
    q = fp4.Fp8Tensor(rows, cols, two_d)
    q.codes.zero_()
    q.codes[:, :cols] = ONE
    q.scales.fill_(byte)
    return q


def zeros(fp4, rows, cols):
    q = ones(fp4, rows, cols, True)
    q.codes.zero_()
    return q


def adapters(fp4, count, N, K):
    """Zeros, to be filled in, of rank 8."""
    return fp4.LoraAdapters.wrap(torch.zeros(count, 8, -(-K // 8) * 8, dtype=torch.bfloat16, device="cuda"),
                                 torch.zeros(count, N, 8, dtype=torch.bfloat16, device="cuda"),
                                 torch.ones(count, device="cuda"), K)


def fprop(fp4, x, w, l, index, fast, drop=None):
    y = torch.empty(x.rows, w.rows, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fp4.fp8_lora_fprop_ws_bytes(x.rows, w.rows, x.cols, l.rank, fast=fast), dtype=torch.uint8,
                     device="cuda")
    fp4.fp8_lora_fprop(x, w, l, y, index=index, drop=drop, ws=ws, fast=fast)
    return y.float()


def backward(fp4, dy, wt, x, l, index, fast, drop=None):
    dx = torch.empty(x.rows, x.cols, dtype=torch.bfloat16, device="cuda")
    da, db = torch.empty(l.a.shape, device="cuda"), torch.empty(l.b.shape, device="cuda")
    ws = torch.empty(fp4.fp8_lora_backward_ws_bytes(x.rows, dy.cols, x.cols, l.rank, l.count, fast=fast),
                     dtype=torch.uint8, device="cuda")
    fp4.fp8_lora_backward(dy, wt, x, l, dx, da, db, ws, index=index, drop=drop, fast=fast)
    return dx.float(), da, db


SIZES = [(20, 72, 136), (300, 200, 264), (700, 130, 200)]


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_large_coefficients(fp4, M, N, K, fast):
    """c t = 3.4e38, between the largest bf16 and the largest binary32 value, is finite; one
    past binary32 is an infinity of its sign, and a NaN nowhere."""
    big = float(torch.tensor(3.4e38))
    index = (torch.arange(M, device="cuda") % 4).int() - 1  # none, and three adapters
    for side in ("y", "dx"):
        l = adapters(fp4, 3, N, K)
        l.scale.fill_(big)
        t = torch.tensor([1.0, 4.0, -4.0], dtype=torch.bfloat16, device="cuda")
        if side == "y":
            l.a[:, 0, 0], l.b[:, :, 0] = t, 2.0 ** -20
            got = fprop(fp4, ones(fp4, M, K), zeros(fp4, N, K), l, index, fast)
        else:
            l.b[:, 0, 0], l.a[:, 0, :] = t, 2.0 ** -20
            got = backward(fp4, ones(fp4, M, N), zeros(fp4, K, N), ones(fp4, M, K), l, index, fast)[0]
        want = torch.tensor([0.0, big * 2.0 ** -20, float("inf"), float("-inf")], device="cuda").bfloat16().float()
        assert torch.equal(got, want[index.long() + 1][:, None].expand_as(got)), side


@pytest.mark.parametrize("M", [20, 700])
def test_large_sums_in_the_gradients(fp4, M):
    """dt and t past the largest bf16 are what da and db say; past binary32, infinities."""
    N, K = 130, 200
    index = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    index[3], index[M - 2] = 0, 1
    l = adapters(fp4, 2, N, K)
    l.scale.fill_(2.0 ** -10)
    f = float(2.0 ** 127 * 1.998046875)  # 2 - 2^-9: between the largest bf16 and binary32 values
    two = torch.tensor([1.984375, 0.013671875], dtype=torch.bfloat16, device="cuda")
    # dt by dy = 2^127, da = c dt x with x = 1
    l.b[0, :2, 0], l.b[1, :2, 0] = two, 4.0
    _, da, _ = backward(fp4, ones(fp4, M, N, byte=254), zeros(fp4, K, N), ones(fp4, M, K), l, index, False)
    assert (da[0, 0, :K] == f * 2.0 ** -10).all() and (da[1, 0, :K] == float("inf")).all()
    # t by x = 2^127, db = c dy t with dy = 1
    l.b.zero_()
    l.a[0, 0, :2], l.a[1, 0, :2] = two, -4.0
    _, _, db = backward(fp4, ones(fp4, M, N), zeros(fp4, K, N), ones(fp4, M, K, byte=254), l, index, False)
    assert (db[0, :, 0] == f * 2.0 ** -10).all() and (db[1, :, 0] == float("-inf")).all()


@pytest.mark.parametrize("M", [20, 700])
def test_a_nan_stays_in_its_column_of_the_gradients(fp4, M):
    """A block with a NaN has a large scale and zeros beside it: the zeros add nothing, however
    large the coefficient, and a dropped NaN nothing either."""
    import drop_ref
    N, K = 130, 200
    index = torch.zeros(M, dtype=torch.int32, device="cuda")
    l = adapters(fp4, 1, N, K)
    l.b[:, 0, 0], l.a[:, 0, 0] = 4096.0, 4096.0

    def spoiled(cols, at):
        q = ones(fp4, M, cols)
        q.codes[5, 128 * (at // 128):128 * (at // 128) + 128] = 0
        q.codes[5, at] = NAN_CODE
        q.scales[at // 128, 5] = 247  # 2^120, what the quantizer gives such a block
        return q

    _, da, _ = backward(fp4, ones(fp4, M, N), zeros(fp4, K, N), spoiled(K, 131), l, index, False)
    assert da[0, 0, 131].isnan()
    want = torch.full((K,), 4096.0 * M, device="cuda")
    want[128:] = 4096.0 * (M - 1)
    cols = torch.arange(K, device="cuda") != 131
    assert torch.equal(da[0, 0, :K][cols], want[cols])
    # with a dropout that takes the NaN away
    seed = next(s for s in range(50) if not drop_ref.keep(M, K, 0.5, s)[5, 131])
    mask = drop_ref.keep(M, K, 0.5, seed).float().cuda()
    _, da, _ = backward(fp4, ones(fp4, M, N), zeros(fp4, K, N), spoiled(K, 131), l, index, False,
                        fp4.Dropout(0.5, seed))
    mask[5, 128:] = 0
    assert torch.equal(da[0, 0, :K], mask.sum(0) * 2 * 4096.0)

    _, _, db = backward(fp4, spoiled(N, 129), zeros(fp4, K, N), ones(fp4, M, K), l, index, False)
    assert db[0, 129, 0].isnan()
    want = torch.full((N,), 4096.0 * M, device="cuda")
    want[128:] = 4096.0 * (M - 1)
    assert torch.equal(db[0, :129, 0], want[:129])
