"""CPU checks of the 8-bit operators' C ABI: exports, sizes, refusals (every call below
fails its host-side checks, so no device pointer is touched), the assembly's use of M0,
and the tests' own reference against its definition."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


def T(rows, cols, two_d=0, codes=0x100000, scales=0x200000):
    from nvfp4_bit_microscaled_amd.fp8 import fp8_tensor
    return ctypes.byref(fp8_tensor(codes, scales, rows, cols, two_d))


def test_header_binding_and_library_agree(m):
    with open(os.path.join(ROOT, "include", "nvfp4_amd_fp8.h")) as f:
        src = f.read()
    declared = sorted(set(re.findall(r"^\s*FP4_API\s+fp4_status\s+(fp8_\w+)\s*\(", src, re.M)))
    assert declared == sorted(m.FP8_EXPORTS)
    out = os.popen(f"nm -D --defined-only {m.LIB_PATH}").read()
    assert {n for n in (ln.split()[-1] for ln in out.splitlines() if " T " in ln) if n.startswith("fp8_")} \
        == set(m.FP8_EXPORTS)


def test_header_is_c(tmp_path):
    (tmp_path / "t.c").write_text('#include "nvfp4_amd_fp8.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    f"-I{ROOT}/include", "-c", str(tmp_path / "t.c"), "-o", str(tmp_path / "t.o")], check=True)


def test_tensor_bytes(m):
    assert m.fp8_tensor_bytes(10, 130) == (10 * 256, 2 * 16)
    assert m.fp8_tensor_bytes(129, 128, True) == (129 * 128, 2)
    assert m.fp8_tensor_bytes(0, 64) == (0, 0)
    for bad in ((-1, 4), (4, -1), (1 << 25, 4), (16776960, 16776960)):
        with pytest.raises(m.Fp4Error):
            m.fp8_tensor_bytes(*bad)


def test_quantize_refusals(lib):
    f = lib.fp8_quantize
    q, qt = T(64, 100), T(100, 64)
    assert f(P, 7, 64, 100, 100, q, qt, None) == DTYPE
    assert f(P, 0, 64, 100, 100, None, None, None) == NULL
    assert f(None, 0, 64, 100, 100, q, qt, None) == NULL
    assert f(P, 0, 64, 100, 99, q, qt, None) == SHAPE
    assert f(P, 0, -1, 100, 100, q, qt, None) == SHAPE
    assert f(ODD, 0, 64, 100, 100, q, qt, None) == ALIGN
    assert f(ctypes.c_void_p(0x10002), 1, 64, 100, 100, q, qt, None) == ALIGN
    assert f(P, 0, 64, 100, 100, T(64, 99), qt, None) == MISMATCH
    assert f(P, 0, 64, 100, 100, q, T(64, 100), None) == MISMATCH
    assert f(P, 0, 64, 100, 100, q, T(100, 64, 1), None) == MISMATCH  # scales of two kinds
    assert f(P, 0, 64, 100, 100, T(64, 100, 0, 0x100008), None, None) == ALIGN
    assert f(P, 0, 64, 100, 100, T(64, 100, 0, 0x100000, 0x200004), None, None) == ALIGN
    assert f(P, 0, 64, 100, 100, T(64, 100, 0, None), None, None) == NULL
    assert f(None, 0, 0, 100, 100, T(0, 100, 0, None, None), None, None) == OK  # nothing to do


def test_norm_refusals(lib):
    def f(x=P, ldx=100, res=P, ldr=100, dt=0, rows=64, cols=100, w=P, eps=1e-6, h=P, ldh=100, y=None, yt=None, rstd=P):
        return lib.fp8_rms_norm(x, ldx, res, ldr, dt, rows, cols, w, eps, h, ldh, y or T(64, 100), yt, rstd, None)
    assert f(dt=3) == DTYPE
    assert f(x=None) == NULL
    assert f(h=None) == NULL  # a residual without its sum
    assert f(res=None) == NULL
    assert f(w=None) == NULL
    assert f(yt=T(100, 64), rstd=None) == NULL  # the transposed output reads rstd
    for bad in (dict(ldx=99), dict(ldr=99), dict(ldh=99), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(rows=-1)):
        assert f(**bad) == SHAPE, bad
    assert f(x=ODD) == ALIGN
    assert f(w=ctypes.c_void_p(0x10002)) == ALIGN
    assert f(y=T(64, 101)) == MISMATCH
    assert f(yt=T(64, 100)) == MISMATCH
    assert f(y=T(64, 100, 1)) == MODE
    assert f(yt=T(100, 64, 1)) == MODE


def test_norm_backward_refusals(lib, m):
    need = m.fp8_rms_norm_ws_bytes(64, 100)

    def f(dy=P, h=P, dh=P, dt=0, rows=64, cols=100, w=P, rstd=P, dx=P, dw=P, ws=P, n=need):
        return lib.fp8_rms_norm_backward(dy, h, dh, dt, rows, cols, w, rstd, dx, dw, ws, n, None)
    assert need > 0
    assert f(dt=2) == DTYPE
    for name in ("dy", "h", "w", "rstd", "dx", "dw", "ws"):
        assert f(**{name: None}) == NULL, name
    for name in ("dy", "h", "dh", "w", "rstd", "dx", "dw", "ws"):
        assert f(**{name: ODD}) == ALIGN, name
    assert f(rows=-2) == SHAPE
    assert f(n=need - 1) == WORKSPACE


def test_gemm_refusals(lib, m):
    f = lib.fp8_gemm
    a, b = T(64, 100), T(32, 100, 1)
    assert f(a, T(32, 101), P, 1, 32, 0, None, 0, None) == MISMATCH
    assert f(a, b, P, 9, 32, 0, None, 0, None) == DTYPE
    assert f(a, b, P, 1, 31, 0, None, 0, None) == SHAPE
    assert f(a, b, None, 1, 32, 0, None, 0, None) == NULL
    assert f(a, b, P, 1, 32, 2, None, 0, None) == MODE
    assert f(None, b, P, 1, 32, 0, None, 0, None) == NULL
    assert f(a, b, ctypes.c_void_p(0x10002), 1, 32, 0, None, 0, None) == ALIGN
    assert f(a, b, P, 1, 32, 0, None, 64, None) == NULL
    assert f(a, b, P, 1, 32, 0, ctypes.c_void_p(0x10008), 64, None) == ALIGN
    assert f(T(64, 100, 0, 0x100001), b, P, 1, 32, 0, None, 0, None) == ALIGN
    assert f(T(64, 100, 0, None), b, P, 1, 32, 0, None, 0, None) == NULL
    assert f(T(0, 100, 0, None, None), b, None, 1, 32, 0, None, 0, None) == OK
    with pytest.raises(m.Fp4Error):
        m.fp8_gemm_ws_bytes(-1, 4, 4)


def test_ffn_refusals(lib, m):
    from nvfp4_bit_microscaled_amd.fp8 import fp8_ffn_buffers, fp8_tensor
    M, K, F = 40, 100, 260
    need = m.fp8_ffn_ws_bytes(M, K, F)

    def f(x=None, wg=None, wu=None, wd=None, hq=None, g=P, u=P, y=P, ldy=K, ws=P, n=need):
        return lib.fp8_ffn_fprop(x or T(M, K), wg or T(F, K, 1), wu or T(F, K, 1), wd or T(K, F, 1), hq or T(M, F), g,
                                 u, y, ldy, ws, n, None)
    assert f(x=T(M, K, 1)) == MISMATCH
    assert f(wg=T(F, K)) == MISMATCH
    assert f(wu=T(F + 1, K, 1)) == MISMATCH
    assert f(wd=T(F, K, 1)) == MISMATCH
    assert f(hq=T(M, K)) == MISMATCH
    assert f(g=None) == NULL
    assert f(u=None) == NULL
    assert f(y=None) == NULL
    assert f(u=ODD) == ALIGN
    assert f(ldy=K - 1) == SHAPE
    assert f(n=need - 1) == WORKSPACE
    assert f(ws=None) == NULL

    def b(bufs=None, dyq=None, wd_t=None, g=P, dwd=P, n=need):
        good = fp8_ffn_buffers(*(fp8_tensor(0x100000, 0x200000, r, c, 0)
                                 for r, c in ((M, F), (M, F), (F, M), (F, M), (F, M))))
        return lib.fp8_ffn_backward(dyq or T(M, K), T(K, M), T(K, M), T(K, F, 1), T(K, F, 1), wd_t or T(F, K, 1), g, P,
                                    ctypes.byref(bufs or good), P, P, P, dwd, P, n, None)
    assert b(dyq=T(M, K, 1)) == MISMATCH
    assert b(wd_t=T(F, K)) == MISMATCH
    assert b(g=None) == NULL
    assert b(dwd=ODD) == ALIGN
    assert b(n=need - 1) == WORKSPACE
    assert b(bufs=fp8_ffn_buffers()) == MISMATCH


def test_binding_refusals(m):
    q = m.Fp8Tensor(4, 100, device="cpu")
    with pytest.raises(ValueError):
        m.Fp8Tensor.wrap(q.codes[:, :64], q.scales, 4, 100)
    with pytest.raises(ValueError):
        m.Fp8Tensor.wrap(q.codes, q.scales.float(), 4, 100)
    with pytest.raises(ValueError):
        m.fp8_gemm(q, q, torch.empty(4, 5))
    with pytest.raises(TypeError):
        m.fp8_quantize(torch.zeros(4, 100, dtype=torch.float16), q, stream=_Stream())
    with pytest.raises(ValueError):
        m.fp8_rms_norm(torch.zeros(4, 100), torch.zeros(99), 1e-6, q, stream=_Stream())


class _Stream:
    cuda_stream = 0


def test_m0_is_only_written_by_the_dma_statements(tmp_path):
    """The LDS DMA statements set M0 in inline assembly, unseen by the compiler: every
    line of the assembly that names m0 is such a statement's own write, followed by one
    wait state and the load."""
    from nvfp4_bit_microscaled_amd import build
    out = tmp_path / "fp8_gemm.s"
    cmd = [build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, "fp8_gemm.hip"), "-o",
           str(out)]
    subprocess.run(cmd, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    lines = [ln.strip() for ln in out.read_text().splitlines()]
    uses = [i for i, ln in enumerate(lines) if re.search(r"\bm0\b", ln) and not ln.startswith(";")]
    assert uses, "the DMA statements are expected in the assembly"
    for i in uses:
        assert re.fullmatch(r"s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi|ttmp\d+)", lines[i]), lines[i]
        assert lines[i + 1] == "s_nop 0", lines[i + 1]
        assert re.fullmatch(r"buffer_load_(dwordx4|dword|ubyte) .* offen lds", lines[i + 2]), lines[i + 2]


def test_reference_scale_and_grid():
    """The reference's exponent is minimal, and its grid is the E4M3 type's."""
    a = torch.tensor([448.0, 448.0 * (1 + 2.0 ** -20), 1.75, 1.7500001, 1.0, 2.0 ** -140, 0.0, 3e38], dtype=torch.float64)
    e = ref.exponent(a)
    assert (a <= 448 * torch.exp2(e.double())).all()
    assert ((a > 448 * torch.exp2(e.double() - 1)) | (e == -126) | (a == 0)).all()
    v = torch.linspace(-448, 448, 300001, dtype=torch.float32)
    assert torch.equal(ref.grid(v.double()).float(), v.to(torch.float8_e4m3fn).float())


def test_reference_gradients_against_differences():
    """The formulas of the norm's and the activation's gradients against central
    differences in binary64 (step 1e-5: truncation 1e-10, rounding 1e-10 of values near
    1; bound 1e-7)."""
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, dy, vx, vw = rnd(3, 50), rnd(50), rnd(3, 50), rnd(3, 50), rnd(50)

    def loss(x, w):
        return (ref.norm(x, None, w, 1e-6)[2] * dy).sum()
    dx, dw = ref.norm_grad(dy, x, w, ref.norm(x, None, w, 1e-6)[1], None)
    e = 1e-5
    assert abs((loss(x + e * vx, w) - loss(x - e * vx, w)) / (2 * e) - (dx * vx).sum()) < 1e-7
    assert abs((loss(x, w + e * vw) - loss(x, w - e * vw)) / (2 * e) - (dw * vw).sum()) < 1e-7
    g = torch.linspace(-20, 20, 4001, dtype=torch.float64)
    assert ((ref.silu(g + e) - ref.silu(g - e)) / (2 * e) - ref.dsilu(g)).abs().max() < 1e-7
