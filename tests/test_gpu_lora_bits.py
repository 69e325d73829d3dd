"""GPU: with binary32 sums the adapters' coefficients keep all of binary32.

t = 1 + 2^-10 + 2^-20 has 21 bits; the product with the weight takes 1 + 2^-10 of it away again,
and what is left, 2^-20, is the coefficient's last bit.  All sums are exact in binary32."""
import pytest
import torch

import drop_ref

pytestmark = pytest.mark.gpu

SIZES = [(20, 70, 136), (65, 300, 4000), (300, 200, 264), (700, 130, 1030), (3900, 3896, 200)]
T = (1.0, 2.0 ** -10, 2.0 ** -20)


def tokens(fp4, rows, cols):
    """Ones in the first three columns."""
    q = fp4.Fp8Tensor(rows, cols)
    q.codes.zero_()
    q.codes[:, :3] = 0x38
    q.scales.fill_(127)
    return q


def weight(fp4, rows, cols, byte):
    """Every row -1, -2^-10, 0 ... times 2^(byte - 119)."""
    q = fp4.Fp8Tensor(rows, cols, True)
    q.codes.zero_()
    q.codes[:, 0], q.codes[:, 1] = 0xF8, 0xA8  # -256, -2^-2
    q.scales.fill_(byte)
    return q


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(fp4, M, N, K):
    a, b = bf16(1, 8, -(-K // 8) * 8), bf16(1, N, 8)
    a[0, 5, :3] = torch.tensor(T)
    b[0, :, 5] = 1
    y = bf16(M, N)
    ws = torch.empty(fp4.fp8_lora_fprop_ws_bytes(M, N, K, 8), dtype=torch.uint8, device="cuda")
    fp4.fp8_lora_fprop(tokens(fp4, M, K), weight(fp4, N, K, 119), fp4.LoraAdapters.wrap(a, b, torch.ones(1, device="cuda"), K),
                       y, ws=ws)
    assert (y == 2.0 ** -20).all()


@pytest.mark.parametrize("p", [0.0, 0.5])
@pytest.mark.parametrize("M,N,K", [(m, k, n) for m, n, k in SIZES])
def test_gradient(fp4, M, N, K, p):
    """With a dropout of a half what is kept of dt a is twice as large, and so is W here."""
    a, b = bf16(1, 8, -(-K // 8) * 8), bf16(1, N, 8)
    b[0, :3, 5] = torch.tensor(T)
    a[0, 5] = 1
    dx, da, db = bf16(M, K), torch.empty(a.shape, device="cuda"), torch.empty(b.shape, device="cuda")
    ws = torch.empty(fp4.fp8_lora_backward_ws_bytes(M, N, K, 8, 1), dtype=torch.uint8, device="cuda")
    fp4.fp8_lora_backward(tokens(fp4, M, N), weight(fp4, K, N, 120 if p else 119), tokens(fp4, M, K),
                          fp4.LoraAdapters.wrap(a, b, torch.ones(1, device="cuda"), K), dx, da, db, ws,
                          drop=fp4.Dropout(p, 3) if p else None)
    if p == 0:
        assert (dx == 2.0 ** -20).all()
        return
    keep = drop_ref.keep(M, K, p, 3).cuda()
    assert (dx[keep] == 2.0 ** -19).all() and (dx[~keep] == -2.0).all()  # -2 - 2^-9, rounded
