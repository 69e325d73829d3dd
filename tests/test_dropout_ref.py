"""CPU checks of dropout: refusals of the C calls (none of them gets to the device) and of
the binding, and the tests' own reference: the generator against the oracle's, the share it
keeps, its independence of the row's stride."""
import ctypes
import os

import numpy as np
import pytest
import torch

import drop_ref

OK, NULL, SHAPE, ALIGN, DTYPE, MODE, MISMATCH, WORKSPACE = 0, 1, 2, 3, 4, 5, 6, 8
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)


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


def D(p=0.1, step=None):
    from nvfp4_bit_microscaled_amd.fp8 import fp8_dropout_config
    return ctypes.byref(fp8_dropout_config(p, 1, 2, step))


def T(rows, cols, two_d=0):
    from nvfp4_bit_microscaled_amd.fp8 import fp8_tensor
    return ctypes.byref(fp8_tensor(0x100000, 0x200000, rows, cols, two_d))


def test_dropout_refusals(lib):
    def f(x=P, ldx=100, res=P, ldr=100, dt=0, rows=64, cols=100, drop=None, y=P, ldy=100, none=False):
        return lib.fp8_dropout(x, ldx, res, ldr, dt, rows, cols, None if none else drop or D(), y, ldy, None)
    assert f(dt=2) == DTYPE
    assert f(none=True) == NULL
    assert f(x=None) == NULL and f(y=None) == NULL
    for bad in (dict(ldx=99), dict(ldr=99), dict(ldy=99), dict(rows=-1), dict(cols=1 << 25)):
        assert f(**bad) == SHAPE, bad
    for p in (-0.1, 1.0, 1 - 2.0 ** -18, 1 - 2.0 ** -17, 2.0, float("nan"), float("inf")):
        assert f(drop=D(p)) == SHAPE, p
    for bad in ("x", "res", "y"):
        assert f(**{bad: ODD}) == ALIGN, bad
    assert f(drop=D(step=0x10004)) == ALIGN
    assert f(rows=0) == OK and f(cols=0, rows=3) == OK  # nothing to do
    assert f(x=None, res=None, y=None, rows=0) == OK


def test_dropout_norm_refusals(lib, m):
    def f(x=P, ldx=100, res=P, ldr=100, dt=0, drop=None, w=P, eps=1e-6, h=P, ldh=100, y=None, yt=None, rstd=P):
        return lib.fp8_dropout_rms_norm(x, ldx, res, ldr, dt, 64, 100, drop, w, eps, h, ldh, y or T(64, 100), yt, rstd,
                                        None)
    assert f() == NULL  # no dropout
    assert f(drop=D(), res=None, h=None) == NULL
    assert f(drop=D(), h=None) == NULL
    assert f(drop=D(1.0)) == SHAPE
    assert f(drop=D(), ldh=99) == SHAPE
    assert f(drop=D(), eps=0.0) == SHAPE
    assert f(drop=D(), dt=5) == DTYPE
    assert f(drop=D(), y=T(64, 100, 1)) == MODE
    assert f(drop=D(), yt=T(64, 100)) == MISMATCH
    assert f(drop=D(), yt=T(100, 64), rstd=None) == NULL
    need = m.fp8_rms_norm_ws_bytes(64, 100)

    def b(dy=P, h=P, dh=P, dt=0, rows=64, drop=None, w=P, rstd=P, dx=P, dres=P, dw=P, ws=P, n=need):
        return lib.fp8_dropout_rms_norm_backward(dy, h, dh, dt, rows, 100, drop or D(), w, rstd, dx, dres, dw, ws, n,
                                                 None)
    for name in ("dy", "h", "w", "rstd", "dx", "dres", "dw", "ws"):
        assert b(**{name: None}) == NULL, name
        assert b(**{name: ODD}) == ALIGN, name
    assert b(drop=D(1.5)) == SHAPE
    assert b(n=need - 1) == WORKSPACE
    assert b(dt=7) == DTYPE
    assert b(rows=-1) == SHAPE


def test_binding_refusals(m):
    x = torch.zeros(4, 16)
    for p in (-0.01, 1.0, float("nan")):
        with pytest.raises(ValueError):
            m.Dropout(p, 1)
    with pytest.raises(ValueError):
        m.Dropout(0.1, 1, step=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        m.Dropout(0.1, 1, step=torch.zeros(2, dtype=torch.int64))
    d = m.Dropout(0.1, 1)
    with pytest.raises(ValueError):
        m.fp8_dropout(x, d, x)  # not on a GPU
    with pytest.raises(ValueError):
        m.fp8_dropout(x, d, x[:2])
    with pytest.raises(ValueError):
        m.fp8_dropout(x, d, x.bfloat16())
    with pytest.raises(ValueError):
        m.fp8_dropout(x, d, x, residual=x[:, :8])
    with pytest.raises(ValueError):
        m.fp8_dropout_rms_norm(x, d, torch.zeros(15), 1e-6, m.Fp8Tensor(4, 16, device="cpu"), x, x)


def test_generator_against_the_oracles(oracle):
    """Philox of the reference equals the oracle's on counters of every word."""
    rng = np.random.default_rng(3)
    c = rng.integers(0, 2 ** 32, (50, 4), dtype=np.uint64)
    k = [int(v) for v in rng.integers(0, 2 ** 32, 2)]
    got = np.stack(drop_ref.philox(*(c[:, i].copy() for i in range(4)), *k), 1)
    for row, want in zip(got, c):
        assert [int(v) for v in row] == [int(v) for v in oracle.philox4x32_10([int(v) for v in want], k)]


@pytest.mark.parametrize("p", [0.0, 0.05, 0.5, 0.9])
def test_share_kept(p):
    """2^20 elements: the share kept is within 5 standard deviations of 1 - T / 2^16, and
    neighbouring offsets and seeds agree as often as independent masks do."""
    n = 1 << 20
    q = 1 - drop_ref.threshold(p) / 65536
    a = drop_ref.keep(1024, 1024, p, 77, 5).double()
    assert abs(float(a.mean()) - q) <= 5 * (q * (1 - q) / n) ** 0.5
    for other in (drop_ref.keep(1024, 1024, p, 77, 6), drop_ref.keep(1024, 1024, p, 78, 5)):
        both = q * q + (1 - q) ** 2
        agree = float((a == other.double()).double().mean())
        assert abs(agree - both) <= 5 * (both * (1 - both) / n) ** 0.5


def test_step_and_offset_add():
    assert torch.equal(drop_ref.keep(3, 20, 0.3, 9, 4, 3), drop_ref.keep(3, 20, 0.3, 9, 7))
    assert torch.equal(drop_ref.keep(3, 20, 0.3, 9, 2 ** 64 - 1, 3), drop_ref.keep(3, 20, 0.3, 9, 2))
