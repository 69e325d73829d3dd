"""CPU checks of the low-rank adapters' calls: refusals (none gets to the device), workspace
sizes, the binding's checks, and the tests' reference gradients against differences."""
import ctypes
import os

import pytest
import torch

OK, NULL, SHAPE, ALIGN, DTYPE, MODE, MISMATCH, WORKSPACE = 0, 1, 2, 3, 4, 5, 6, 8
P, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)
M, N, K, R, C = 40, 300, 100, 16, 3


@pytest.fixture(scope="module")
def m():
    import nvfp4_bit_microscaled_amd as m
    if not os.path.exists(m.LIB_PATH):
        from nvfp4_bit_microscaled_amd import build
        build.build()
    return m


@pytest.fixture(scope="module")
def lib(m):
    from nvfp4_bit_microscaled_amd import fp8
    return fp8.lib()


def T(rows, cols, two_d=0):
    from nvfp4_bit_microscaled_amd.fp8 import fp8_tensor
    return ctypes.byref(fp8_tensor(0x100000, 0x200000, rows, cols, two_d))


def L(a=0x30000, b=0x40000, scale=0x50000, lda=104, count=C, rank=R):
    from nvfp4_bit_microscaled_amd.fp8 import fp8_lora
    return ctypes.byref(fp8_lora(a, b, scale, lda, count, rank))


def D(p=0.1):
    from nvfp4_bit_microscaled_amd.fp8 import fp8_dropout_config
    return ctypes.byref(fp8_dropout_config(p, 1, 2, None))


LORA_REFUSALS = [(dict(a=None), NULL), (dict(b=None), NULL), (dict(scale=None), NULL), (dict(a=0x30008), ALIGN),
                 (dict(b=0x40008), ALIGN), (dict(scale=0x50002), ALIGN), (dict(lda=96), SHAPE), (dict(lda=108), SHAPE),
                 (dict(count=0), SHAPE), (dict(count=-1), SHAPE), (dict(count=65536), SHAPE), (dict(rank=0), SHAPE),
                 (dict(rank=12), SHAPE), (dict(rank=136), SHAPE), (dict(rank=-8), SHAPE)]


def test_fprop_refusals(lib, m):
    need = m.fp8_lora_fprop_ws_bytes(M, N, K, R)

    def f(x=None, w=None, lora=None, index=P, drop=None, y=P, ldy=N, flags=0, ws=P, n=need):
        return lib.fp8_lora_fprop(x or T(M, K), w or T(N, K, 1), lora or L(), index, drop, y, ldy, flags, ws, n, None)
    assert need > 0
    for bad, code in LORA_REFUSALS:
        assert f(lora=L(**bad)) == code, bad
    assert lib.fp8_lora_fprop(T(M, K), T(N, K, 1), None, P, None, P, N, 0, P, need, None) == NULL
    assert lib.fp8_lora_fprop(None, T(N, K, 1), L(), P, None, P, N, 0, P, need, None) == NULL
    assert f(x=T(M, K, 1)) == MISMATCH and f(w=T(N, K)) == MISMATCH and f(w=T(N, K + 1, 1)) == MISMATCH
    assert f(flags=2) == MODE
    assert f(drop=D(1.0)) == SHAPE
    assert f(index=ctypes.c_void_p(0x10002)) == ALIGN
    assert f(y=None) == NULL and f(y=ODD) == ALIGN and f(ldy=N - 1) == SHAPE
    assert f(n=need - 1) == WORKSPACE and f(ws=None) == NULL and f(ws=ctypes.c_void_p(0x10008)) == ALIGN


def test_backward_refusals(lib, m):
    need = m.fp8_lora_backward_ws_bytes(M, N, K, R, C)

    def f(dy=None, wt=None, x=None, lora=None, index=P, drop=None, dx=P, lddx=K, da=P, db=P, flags=0, ws=P, n=need):
        return lib.fp8_lora_backward(dy or T(M, N), wt or T(K, N, 1), x or T(M, K), lora or L(), index, drop, dx, lddx,
                                     da, db, flags, ws, n, None)
    for bad, code in LORA_REFUSALS:
        assert f(lora=L(**bad)) == code, bad
    assert f(dy=T(M, N, 1)) == MISMATCH and f(dy=T(M + 1, N)) == MISMATCH
    assert f(wt=T(K, N)) == MISMATCH and f(wt=T(N, K, 1)) == MISMATCH
    assert f(x=T(M, K, 1)) == MISMATCH
    assert f(flags=4) == MODE and f(drop=D(-1.0)) == SHAPE
    for name in ("dx", "da", "db", "ws"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: ODD}) == ALIGN, name
    assert f(lddx=K - 1) == SHAPE
    assert f(n=need - 1) == WORKSPACE


def test_ws_bytes(m):
    assert m.fp8_lora_fprop_ws_bytes(0, N, K, R) == 0
    for bad in ((-1, N, K, R), (M, N, K, 4), (M, N, K, 256), (1 << 25, N, K, R)):
        with pytest.raises(m.Fp4Error):
            m.fp8_lora_fprop_ws_bytes(*bad)
    for bad in ((M, N, K, R, 0), (M, N, K, 3, 1), (M, 1 << 22, 1 << 22, 128, 60000)):
        with pytest.raises(m.Fp4Error):
            m.fp8_lora_backward_ws_bytes(*bad)
    # many adapters and few tokens: no room for sums that no token has
    few, many = m.fp8_lora_backward_ws_bytes(8, 512, 512, 8, 8), m.fp8_lora_backward_ws_bytes(8, 512, 512, 8, 1000)
    assert many - few <= 1000 * (2 * 8 * 1024 + 4) + 64


def test_binding_refusals(m):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    good = (z(2, 8, 16), z(2, 5, 8), z(2, dt=torch.float32), 10)
    l = m.LoraAdapters.wrap(*good)
    for bad in ((z(2, 8, 12), *good[1:]), (z(2, 12, 16), z(2, 5, 12), *good[2:]), (z(2, 8, 8), *good[1:]),
                (good[0].float(), *good[1:]), (good[0], z(3, 5, 8), *good[2:]), (good[0], z(2, 5, 16), *good[2:]),
                (good[0], good[1], z(2), 10), (z(2, 136, 16), z(2, 5, 136), *good[2:])):
        with pytest.raises(ValueError):
            m.LoraAdapters.wrap(*bad)
    x, w = m.Fp8Tensor(4, 10, device="cpu"), m.Fp8Tensor(5, 10, True, device="cpu")
    y = z(4, 5)
    for kw in (dict(), dict(index=torch.zeros(3, dtype=torch.int32)), dict(index=torch.zeros(4, dtype=torch.int64))):
        with pytest.raises(ValueError):
            m.fp8_lora_fprop(x, w, l, y, **kw)
    with pytest.raises(ValueError):
        m.fp8_lora_fprop(x, w, l, z(4, 6))
    with pytest.raises(ValueError):
        m.fp8_lora_fprop(x, m.Fp8Tensor(6, 10, True, device="cpu"), l, z(4, 6))
    with pytest.raises(ValueError):
        m.fp8_lora_backward(m.Fp8Tensor(4, 5, device="cpu"), m.Fp8Tensor(10, 5, True, device="cpu"), x, l, z(4, 10),
                            torch.zeros(2, 8, 16), torch.zeros(2, 5, 7), None)
    new = m.LoraAdapters(3, 8, 20, 30, device="cpu")
    assert new.a.shape == (3, 8, 32) and new.b.shape == (3, 20, 8) and (new.b == 0).all()


def test_reference_gradients_against_differences(m):
    """sum(y * dy) along random directions of x, a and b, central differences of step 1e-5 in
    binary64: it is a polynomial of second degree in a step along one of them, so that the
    difference has no truncation error, and its rounding is about 1e-10 of values near 1."""
    from lora_ref import Problem
    for p in (0.0, 0.3):
        q = Problem(m, 9, 40, 50, 8, 3, p=p, device="cpu")
        x, w, dy, a, b, s, g = q.values()
        (dx, da, db), _ = q.backward()
        gen = torch.Generator().manual_seed(5)

        def loss(x, a, b):
            y = x @ w.t()
            for i in range(3):
                r = q.rows(i)
                y[r] += s[i] * (x[r] * g[r]) @ a[i].t() @ b[i].t()
            return (y * dy).sum()
        e = 1e-5
        for k, grad in enumerate((dx, da, db)):
            v = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
            lo, hi = [x, a, b], [x, a, b]
            hi[k], lo[k] = hi[k] + e * v, lo[k] - e * v
            assert abs((loss(*hi) - loss(*lo)) / (2 * e) - (grad * v).sum()) < 1e-8, (p, k)
