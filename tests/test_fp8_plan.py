"""The plan of the 8-bit products on the CPU: the sizes of the GPU tests reach the kernels
and splits that they are for, whatever the model's constants become."""
import ctypes
import os
import subprocess

import pytest

import fp8_paths as paths

HERE = os.path.dirname(os.path.abspath(__file__))
I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    out = tmp_path_factory.mktemp("plan") / "libfp8plan.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC",
                    os.path.join(HERE, "native", "fp8_plan_check.cpp"), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def blocks(k):
    return I64(-(-k // 128))


def product(plan, M, N, stages, fast):
    out = (I64 * 6)()
    plan.fp8_plan_product(I64(M), I64(N), stages, int(fast), 1, out)
    return tuple(out[:4]) + (bool(out[5]),)


@pytest.mark.parametrize("name", paths.PRODUCTS)
def test_products(plan, name):
    (M, N, K, fast), want = paths.PRODUCTS[name]
    assert product(plan, M, N, blocks(K), fast) == want


@pytest.mark.parametrize("name", paths.FORWARD)
def test_forward(plan, name):
    (M, K, F, fast), (kind, parts, *rows) = paths.FORWARD[name]
    out = (I64 * 6)()
    plan.fp8_plan_dual(I64(M), I64(F), blocks(K), int(fast), out)
    fused = fast and plan.fp8_plan_act_fused(I64(M), I64(F), blocks(K))
    apart = not fast and plan.fp8_plan_act_apart(I64(M), I64(F), blocks(K))
    assert (kind, parts) == (("fused", 1) if fused else ("apart", 1) if apart else ("dual", out[2]))
    assert not rows or rows == [out[0]]


@pytest.mark.parametrize("name", paths.BACKWARD)
def test_backward(plan, name):
    (M, K, F, fast), dx, dact, group = paths.BACKWARD[name]
    assert product(plan, M, K, I64(2 * -(-F // 128)), fast) == dx
    assert (fast and bool(plan.fp8_plan_dact_fused(I64(M), I64(F), blocks(K)))) == dact
    if group:
        whole = I64()
        plan.fp8_plan_group.restype = I64
        assert (plan.fp8_plan_group(I64(F), I64(K), blocks(M), ctypes.byref(whole)), whole.value) == group


def test_every_tile_is_reached(plan):
    """Each tile of the general kernel under both kinds of sums, by the sizes above or those
    of test_gpu_fp8.py."""
    import test_gpu_fp8 as t
    for fast in (False, True):
        shapes = [s[:3] for s, _ in paths.PRODUCTS.values() if s[3] == fast] + t.GSHAPES
        got = {product(plan, M, N, blocks(K), fast)[:2] for M, N, K in shapes}
        assert got == {(16, 64), (16, 128), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128), (256, 256)}, fast
    assert plan.fp8_plan_three_stages(I64(256)) and not plan.fp8_plan_three_stages(I64(257))
