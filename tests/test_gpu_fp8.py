"""GPU parity of the 8-bit operators with their definitions in binary64 (fp8_ref.py,
which also derives the tolerances): odd sizes and strides, blocks of zeros and of tiny
and huge values, one token to several tiles, both kinds of scales, both types."""
import pytest
import torch

import fp8_ref as ref
from parity import check_gemm

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
IDS = {BF16: "bf16", FP32: "fp32"}
EPS = 1e-6


def rnd(*shape, seed=0, std=1.0, dtype=BF16):
    gen = torch.Generator().manual_seed(seed + 1000 * shape[0] + shape[-1])
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def strided(x, ld, shift=0):
    """x on the GPU with row stride ld, `shift` elements into its allocation."""
    buf = torch.full((x.shape[0] * ld + shift + 64,), float("nan"), dtype=x.dtype, device="cuda")
    v = buf[shift:shift + x.shape[0] * ld].view(x.shape[0], ld)[:, :x.shape[1]]
    v.copy_(x)
    return v


def full(q):
    """Poison a tensor's buffers, so that what a call does not write is seen."""
    q.codes.fill_(0x7F)
    q.scales.fill_(0xFF)
    return q


# ------------------------------------------------------------------ quantization

QSHAPES = [(1, 1), (1, 128), (3, 130), (128, 128), (129, 257), (200, 64), (17, 1000), (384, 256), (513, 77)]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=IDS.get)
@pytest.mark.parametrize("two_d", [False, True], ids=["1d", "2d"])
@pytest.mark.parametrize("shape", QSHAPES, ids=str)
def test_quantize(fp4, shape, two_d, dtype):
    m, n = shape
    x = rnd(m, n, dtype=dtype, std=3.0)
    for xs in (x.cuda(), strided(x, n + 8, 8), strided(x, n + 3, 1)):
        q, qt = full(fp4.Fp8Tensor(m, n, two_d)), full(fp4.Fp8Tensor(n, m, two_d))
        fp4.fp8_quantize(xs, q, qt)
        ref.assert_quantized(q, x, "q")
        ref.assert_quantized(qt, x.t(), "q_t")
        q1, q2 = full(fp4.Fp8Tensor(m, n, two_d)), full(fp4.Fp8Tensor(n, m, two_d))
        fp4.fp8_quantize(xs, q1)
        fp4.fp8_quantize(xs, None, q2)
        assert torch.equal(q1.codes, q.codes) and torch.equal(q2.codes, qt.codes)
        assert torch.equal(ref.held(q1)[1], ref.held(q)[1]) and torch.equal(ref.held(q2)[1], ref.held(qt)[1])


def test_quantize_extremes(fp4):
    """Scales at both ends, borders of a power of two, zeros, subnormals and ties."""
    x = torch.zeros(12, 256)
    x[0, 0] = 3.4e38
    x[1, 5] = 448.0
    x[2, 5] = 448.0000305
    x[3, 5] = 1.75 * 2.0 ** -20
    x[4, 5] = 2.0 ** -126
    x[5, 5] = 2.0 ** -149
    x[6, :128] = torch.arange(128) * 3.5 + 0.5
    x[7, :128] = -1e-30
    x[8, 200] = -2.0 ** -133 * 1.75
    x[9] = torch.linspace(-448, 448, 256)
    x[10, :2] = torch.tensor([448.0, 2.0 ** -10])  # a tie of the smallest subnormal with zero
    q, qt = fp4.Fp8Tensor(12, 256), fp4.Fp8Tensor(256, 12)
    fp4.fp8_quantize(x.cuda(), q, qt)
    ref.assert_quantized(q, x)
    ref.assert_quantized(qt, x.t())


def test_quantize_keeps_other_blocks_of_a_nan(fp4):
    x = rnd(8, 384, dtype=FP32)
    y = x.clone()
    y[2, 130] = float("nan")
    y[5, 0] = float("inf")
    q, p = fp4.Fp8Tensor(8, 384), fp4.Fp8Tensor(8, 384)
    fp4.fp8_quantize(x.cuda(), p)
    fp4.fp8_quantize(y.cuda(), q)
    v, w = ref.values(q), ref.values(p)
    assert v[2, 130].isnan() and v[5, 0].isnan()
    keep = torch.ones(8, 384, dtype=torch.bool)
    keep[2, 128:256] = keep[5, :128] = False
    assert torch.equal(v[keep], w[keep])


# ---------------------------------------------------------------------------- norm

NSHAPES = [(1, 64), (1, 5120), (5, 100), (129, 511), (33, 1000), (130, 1024), (7, 2047), (4, 2501), (260, 4100),
           (3, 6144), (9, 7000), (2, 8193), (131, 9000)]


def sum_rel(cols):
    """Relative error of rstd: a thread's sums have at most max(32, cols / 256) terms,
    12 joining and final operations follow; the root halves what the sum is off by."""
    return (max(32, cols / 256) / 2 + 12) * 2.0 ** -24


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=IDS.get)
@pytest.mark.parametrize("shape", NSHAPES, ids=str)
def test_norm(fp4, shape, dtype):
    m, n = shape
    x, r = rnd(m, n, dtype=dtype), rnd(m, n, seed=1, std=2.0, dtype=dtype)
    w = 1 + rnd(n, seed=2, std=0.3, dtype=FP32)
    wc = w.cuda()
    for res, shift in ((r, 0), (None, 0), (r, 1)):
        xs = strided(x, n + 8 + shift, 8 + shift) if shift or n % 8 else x.cuda()
        h, rstd, y = ref.norm(x, res, w, EPS)
        err = y.abs() * (sum_rel(n) + 3 * 2.0 ** -24)
        yq, yt = full(fp4.Fp8Tensor(m, n)), full(fp4.Fp8Tensor(n, m))
        rs = torch.full((m,), float("nan"), device="cuda")
        hb = torch.full((m, n), float("nan"), dtype=dtype, device="cuda") if res is not None else None
        fp4.fp8_rms_norm(xs, wc, EPS, yq, residual=res.cuda() if res is not None else None, h=hb, yq_t=yt, rstd=rs)
        if res is not None:
            assert torch.equal(hb.cpu(), h)
        assert ((rs.cpu().double() - rstd).abs() <= rstd * sum_rel(n)).all()
        ref.assert_near(yq, y, err, "y")
        ref.assert_near(yt, y.t(), err.t(), "y_t")
        # without what only the backward pass reads: the same output
        y1 = full(fp4.Fp8Tensor(m, n))
        fp4.fp8_rms_norm(xs, wc, EPS, y1, residual=res.cuda() if res is not None else None, h=hb)
        assert torch.equal(y1.codes, yq.codes) and torch.equal(y1.scales[:, :m], yq.scales[:, :m])


@pytest.mark.parametrize("n", [640, 5120, 8200])
def test_norm_in_place_and_rows_of_zeros(fp4, n):
    """h over the residual; a row of zeros gives zeros, with rstd = eps^-1/2."""
    x, r = rnd(6, n), rnd(6, n, seed=3)
    x[2] = r[2] = 0
    w = torch.ones(n)
    h, rstd, y = ref.norm(x, r, w, EPS)
    buf, rs, yq = r.cuda(), torch.empty(6, device="cuda"), full(fp4.Fp8Tensor(6, n))
    fp4.fp8_rms_norm(x.cuda(), w.cuda(), EPS, yq, residual=buf, h=buf, rstd=rs)
    assert torch.equal(buf.cpu(), h)
    assert (ref.values(yq)[2] == 0).all()
    assert ((rs.cpu().double() - rstd).abs() <= rstd * sum_rel(n)).all()
    ref.assert_near(yq, y, y.abs() * (sum_rel(n) + 3 * 2.0 ** -24))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=IDS.get)
@pytest.mark.parametrize("shape", NSHAPES + [(0, 100), (1500, 300)], ids=str)
def test_norm_backward(fp4, shape, dtype):
    """dx: the row's mean is a binary32 sum of |v hhat| terms (bound: (max(32, cols / 256) +
    14) 2^-24 of the absolute sum), and six roundings follow; dweight: at most max(32,
    rows / 64) binary32 terms to a partial, joined in binary64, three roundings each."""
    m, n = shape
    h, dy, d = rnd(m, n, std=2.0, dtype=dtype), rnd(m, n, seed=1, dtype=dtype), rnd(m, n, seed=2, dtype=dtype)
    w = 1 + rnd(n, seed=3, std=0.3, dtype=FP32)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    for dh in (d, None):
        want, dw = ref.norm_grad(dy, h, w, rstd, dh)
        hhat = (h.double() * rstd.double()[:, None]).abs()
        v = (dy.double() * w.double()).abs()
        mean = (v * hhat).sum(1, keepdim=True) / n
        err = rstd.double()[:, None] * (v + hhat * mean) * (max(32, n / 256) + 20) * 2.0 ** -24
        half = torch.finfo(dtype).eps / 2
        dx, dwb = torch.empty(m, n, dtype=dtype, device="cuda"), torch.empty(n, device="cuda")
        ws = torch.empty(max(fp4.fp8_rms_norm_ws_bytes(m, n), 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
        hs, dys, ds = h.cuda(), dy.cuda(), d.cuda()
        fp4.fp8_rms_norm_backward(dys, hs, w.cuda(), rstd.cuda(), dx, dwb, ws, dh=ds if dh is not None else None)
        far = (dx.cpu().double() - want).abs() - (err * (1 + half) + half * (1 + 2.0 ** -8) * want.abs())
        assert (far <= 0).all(), float(far.max())
        bound = (dy.double().abs() * hhat).sum(0) * (max(32, m / 64) + 3) * 2.0 ** -24
        assert ((dwb.cpu().double() - dw).abs() <= bound + 2.0 ** -24 * dw.abs()).all()
        # in place over dy: the same bits
        fp4.fp8_rms_norm_backward(dys, hs, w.cuda(), rstd.cuda(), dys, dwb, ws, dh=ds if dh is not None else None)
        assert torch.equal(dys, dx)


# ---------------------------------------------------------------------------- product

GSHAPES = [(1, 1, 1), (1, 130, 128), (3, 257, 300), (4, 64, 1500), (16, 1000, 129), (17, 129, 640), (31, 300, 2000),
           (64, 256, 384), (65, 128, 100), (129, 131, 500), (256, 256, 256), (300, 700, 900), (257, 513, 1300),
           (512, 1024, 8192), (1000, 260, 4000), (1024, 768, 129), (5, 4100, 4090)]


def product_case(fp4, M, N, K, a2, b2):
    a = ref.put(fp4, rnd(M, K, std=0.5), a2)
    b = ref.put(fp4, rnd(N, K, seed=1, std=0.02), b2)
    return a, b


@pytest.mark.parametrize("kinds", [(False, True), (False, False), (True, True)], ids=["1d2d", "1d1d", "2d2d"])
@pytest.mark.parametrize("shape", GSHAPES, ids=str)
def test_gemm(fp4, shape, kinds):
    M, N, K = shape
    a, b = product_case(fp4, M, N, K, *kinds)
    want, bound = ref.product(a, b)
    ws = torch.empty(max(fp4.fp8_gemm_ws_bytes(M, N, K), 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    for dtype in (FP32, BF16):
        for ld, w in ((N, ws), (N, None), (N + 5, ws), (N + 24, None)):
            c = torch.full((M, ld), -7.0, dtype=dtype, device="cuda")
            fp4.fp8_gemm(a, b, c[:, :N], w)
            check_gemm(c[:, :N].float().cpu().numpy(), want.numpy(), bound.numpy(), dtype == BF16, f"{dtype} ld {ld}")
            assert (c[:, N:] == -7.0).all(), "past the row"


@pytest.mark.parametrize("kinds", [(False, True), (False, False), (True, True)], ids=["1d2d", "1d1d", "2d2d"])
@pytest.mark.parametrize("shape", GSHAPES, ids=str)
def test_fast_gemm(fp4, shape, kinds):
    M, N, K = shape
    ws = torch.empty(max(fp4.fp8_gemm_ws_bytes(M, N, K), 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    pairs = (product_case(fp4, M, N, K, *kinds),
             (ref.narrow(fp4, M, K, kinds[0], 1), ref.narrow(fp4, N, K, kinds[1], 2)))
    for dtype in (FP32, BF16):
        for ld, w in ((N, ws), (N, None), (N + 5, ws), (N + 24, None)):
            c = torch.full((M, ld), -7.0, dtype=dtype, device="cuda")
            fp4.fp8_gemm(*pairs[0], c[:, :N], w, fast=True)
            ref.check_fast(c[:, :N], *pairs[0], f"{dtype} ld {ld}")
            fp4.fp8_gemm(*pairs[1], c[:, :N], w, fast=True)
            want, bound = ref.product(*pairs[1])
            check_gemm(c[:, :N].float().cpu().numpy(), want.numpy(), bound.numpy(), dtype == BF16, f"narrow {dtype} {ld}")
            assert (c[:, N:] == -7.0).all(), "past the row"


def test_gemm_scales_are_applied_per_block(fp4):
    """Codes of ones with a power of two per block: every partial sum is a multiple of
    2^-4 below 2^14, exact in binary32 in any order, so the product is equal to the bit."""
    M, N, K = 150, 300, 640
    gen = torch.Generator().manual_seed(5)
    a, b = fp4.Fp8Tensor(M, K), fp4.Fp8Tensor(N, K, True)
    for q in (a, b):
        q.codes.fill_(0x38)  # 1.0
        q.scales.copy_(127 + torch.randint(-2, 3, tuple(q.scales.shape), generator=gen))
    want, _ = ref.product(a, b)
    for fast in (False, True):
        c = torch.empty(M, N, device="cuda")
        fp4.fp8_gemm(a, b, c, fast=fast)
        assert torch.equal(c.cpu().double(), want)


def rows_of(q, rows):
    """The rows of a 1 x 128-scaled library tensor as another one on the CPU."""
    import nvfp4_bit_microscaled_amd as m
    t = m.Fp8Tensor(len(rows), q.cols, device="cpu")
    t.codes.copy_(q.codes[rows].cpu())
    t.scales.fill_(127)
    t.scales[:, :len(rows)] = q.scales[:, rows].cpu()
    return t


# Large enough for the 256 x 256 kernel: whole rounds of tiles with ragged edges, rows of C
# that take no 16-byte stores, a last round in K parts (with and without a workspace)
@pytest.mark.parametrize("shape", [(3900, 3896, 1500), (3900, 3901, 1500), (4300, 3900, 4000)], ids=str)
def test_large_fast_gemm(fp4, shape):
    M, N, K = shape
    x, w = rnd(M, K, std=0.5).cuda(), rnd(N, K, seed=1, std=0.02).cuda()
    a, b = fp4.Fp8Tensor(M, K), fp4.Fp8Tensor(N, K)
    fp4.fp8_quantize(x, a)
    fp4.fp8_quantize(w, b)
    ws = torch.empty(max(fp4.fp8_gemm_ws_bytes(M, N, K), 16), dtype=torch.uint8, device="cuda").fill_(0xFF)
    rows = list(range(0, 9)) + list(range(250, 262)) + list(range(M - 270, M - 250)) + list(range(M - 9, M))
    part, cols = rows_of(a, rows), rows_of(b, list(range(N)))
    for dtype in (FP32, BF16):
        for space in (ws, None):
            c = torch.full((M + 1, N), -7.0, dtype=dtype, device="cuda")
            fp4.fp8_gemm(a, b, c[:M], space, fast=True)
            ref.check_fast(c[rows], part, cols, f"{dtype} ws {space is not None}")
            assert (c[M] == -7.0).all(), "past the last row"


# Large enough for the 256 x 256 tiles of the binary32 sums, aligned and odd rows of C
@pytest.mark.parametrize("shape", [(4200, 4000, 700), (4200, 4001, 700)], ids=str)
def test_large_gemm(fp4, shape):
    M, N, K = shape
    x, w = rnd(M, K, std=0.5).cuda(), rnd(N, K, seed=1, std=0.02).cuda()
    a, b = fp4.Fp8Tensor(M, K), fp4.Fp8Tensor(N, K)
    fp4.fp8_quantize(x, a)
    fp4.fp8_quantize(w, b)
    rows = list(range(0, 9)) + list(range(250, 262)) + list(range(M - 270, M - 250)) + list(range(4090, 4102)) + list(range(M - 9, M))
    want, bound = ref.product(rows_of(a, rows), rows_of(b, list(range(N))))
    for dtype in (FP32, BF16):
        c = torch.full((M + 1, N), -7.0, dtype=dtype, device="cuda")
        fp4.fp8_gemm(a, b, c[:M])
        check_gemm(c[rows].float().cpu().numpy(), want.numpy(), bound.numpy(), dtype == BF16, str(dtype))
        assert (c[M] == -7.0).all(), "past the last row"


def test_offsets_past_32_bits(fp4):
    """4.3e9 codes: the last rows of a quantization and of products that read it."""
    M, K, N = 262400, 16500, 136
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    for i in range(0, M, 26240):
        x[i:i + 26240] = torch.randn(26240, K, generator=gen, device="cuda")
    a, b = fp4.Fp8Tensor(M, K), ref.put(fp4, rnd(N, K, seed=1, std=0.02), True)
    assert a.codes.numel() > 2 ** 32
    fp4.fp8_quantize(x, a)
    rows = [0, 1, 130000, 259999] + list(range(M - 40, M))
    part = rows_of(a, rows)
    ref.assert_quantized(part, x[rows].cpu())
    del x
    cpu_b = fp4.Fp8Tensor(N, K, True, device="cpu")
    cpu_b.codes.copy_(b.codes)
    cpu_b.scales.copy_(b.scales)
    c = torch.empty(M, N, dtype=BF16, device="cuda")
    fp4.fp8_gemm(a, b, c, fast=True)
    ref.check_fast(c[rows], part, cpu_b)
    few = torch.empty(N, M, dtype=FP32, device="cuda")
    fp4.fp8_gemm(b, a, few)
    want, bound = ref.product(cpu_b, part)
    check_gemm(few[:, rows].cpu().numpy(), want.numpy(), bound.numpy(), False, "binary32 sums")


def test_gemm_of_no_k_is_zero(fp4):
    c = torch.full((5, 9), 3.0, device="cuda")
    fp4.fp8_gemm(fp4.Fp8Tensor(5, 0), fp4.Fp8Tensor(9, 0), c)
    assert (c == 0).all()


# -------------------------------------------------------------------------- gated block

FSHAPES = [(1, 64, 128), (3, 100, 300), (8, 384, 1000), (33, 257, 129), (130, 512, 640), (300, 300, 1100),
           (256, 1024, 768), (513, 256, 384), (300, 264, 1000), (700, 130, 200), (512, 1024, 2048),
           # enough tiles for the fused kernels: aligned rows of g and u, and rows that are not
           (2500, 130, 4000), (1900, 130, 2205)]


def weights(fp4, K, F):
    return (ref.put(fp4, rnd(F, K, seed=5, std=K ** -0.5), True), ref.put(fp4, rnd(F, K, seed=6, std=K ** -0.5), True),
            ref.put(fp4, rnd(K, F, seed=7, std=F ** -0.5), True))


def act_rel(g):
    """Relative error of silu(g) u, and of silu'(g)'s terms: exp(-g) is off by |g log2 e|
    2^-24 and three more roundings and one-ulp functions, with six products after it."""
    return (1.5 * g.abs() + 16) * 2.0 ** -24


@pytest.mark.parametrize("shape", FSHAPES, ids=str)
def test_ffn_fprop(fp4, shape):
    M, K, F = shape
    wg, wu, wd = weights(fp4, K, F)
    x = ref.put(fp4, rnd(M, K, seed=8))
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda").fill_(0xFF)
    hq, y = full(fp4.Fp8Tensor(M, F)), torch.full((M, K + 3), -7.0, dtype=BF16, device="cuda")
    g, u = (torch.full((M, F), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    fp4.fp8_ffn_fprop(x, wg, wu, wd, hq, y[:, :K], g=g, u=u, ws=ws)
    ref.check_fast(g, x, wg, "g")
    ref.check_fast(u, x, wu, "u")
    gd, ud = g.cpu().double(), u.cpu().double()
    h = ref.silu(gd) * ud
    ref.assert_near(hq, h, h.abs() * act_rel(gd), "h")
    ref.check_fast(y[:, :K], hq, wd, "y")
    assert (y[:, K:] == -7.0).all()
    # without g and u: the same h and y
    h2, y2 = full(fp4.Fp8Tensor(M, F)), torch.empty(M, K, dtype=BF16, device="cuda")
    fp4.fp8_ffn_fprop(x, wg, wu, wd, h2, y2, ws=ws)
    assert torch.equal(h2.codes, hq.codes) and torch.equal(y2, y[:, :K])


@pytest.mark.parametrize("shape", FSHAPES, ids=str)
def test_ffn_backward(fp4, shape):
    """Each step against its own operands; dh's error is that of a fast product."""
    M, K, F = shape
    wg_t, wu_t, wd_t = (ref.transposed(fp4, w) for w in weights(fp4, K, F))
    dy, x = rnd(M, K, seed=9, std=1e-3), rnd(M, K, seed=8)
    dyq, dyq_t, x_t = ref.put(fp4, dy), ref.put(fp4, dy.t()), ref.put(fp4, x.t())
    g, u = rnd(M, F, seed=10, std=2.0), rnd(M, F, seed=11)
    g[:, :4] = torch.tensor([-1.278, 0.0, 90.0, -100.0])  # silu's minimum, its middle and both ends
    ws = torch.empty(fp4.fp8_ffn_ws_bytes(M, K, F), dtype=torch.uint8, device="cuda").fill_(0xFF)
    bufs = fp4.FfnBuffers(M, K, F)
    for q in (bufs.dgq, bufs.duq, bufs.dgq_t, bufs.duq_t, bufs.hq_t):
        full(q)
    dx, dwg, dwu, dwd = (torch.full(s, float("nan"), dtype=BF16, device="cuda") for s in ((M, K), (F, K), (F, K), (K, F)))
    fp4.fp8_ffn_backward(dyq, dyq_t, x_t, wg_t, wu_t, wd_t, g.cuda(), u.cuda(), bufs, dx, dwg, dwu, dwd, ws=ws)
    dh, bound = ref.product(dyq, wd_t)
    gd, ud = g.double(), u.double()
    s = torch.sigmoid(gd)
    rel, off = act_rel(gd), 1e-5 * bound + ref.cut(dyq, wd_t)
    du = dh * ref.silu(gd)
    dg = dh * ud * ref.dsilu(gd)
    h = ref.silu(gd) * ud
    e_du = ref.silu(gd).abs() * (off + dh.abs() * rel)
    # silu' is a sum of two terms, which may cancel
    e_dg = ud.abs() * (ref.dsilu(gd).abs() * off + (dh.abs() + off) * s * (1 + gd.abs() * (1 - s)) * rel)
    for q, v, e, name in ((bufs.dgq, dg, e_dg, "dg"), (bufs.duq, du, e_du, "du"), (bufs.dgq_t, dg.t(), e_dg.t(), "dg_t"),
                          (bufs.duq_t, du.t(), e_du.t(), "du_t"), (bufs.hq_t, h.t(), (h.abs() * rel).t(), "h_t")):
        ref.assert_near(q, v, e, name)
    ref.check_fast(dx, bufs.dgq, wg_t, "dx", (bufs.duq, wu_t))
    ref.check_fast(dwg, bufs.dgq_t, x_t, "dwg")
    ref.check_fast(dwu, bufs.duq_t, x_t, "dwu")
    ref.check_fast(dwd, dyq_t, bufs.hq_t, "dwd")


def test_ffn_of_no_tokens(fp4):
    K, F = 256, 384
    wg, wu, wd = weights(fp4, K, F)
    ws = torch.empty(max(fp4.fp8_ffn_ws_bytes(0, K, F), 16), dtype=torch.uint8, device="cuda")
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    Q = fp4.Fp8Tensor
    fp4.fp8_ffn_fprop(Q(0, K), wg, wu, wd, Q(0, F), e(0, K), ws=ws)
    dwg, dwu, dwd = (torch.full(s, 3.0, dtype=BF16, device="cuda") for s in ((F, K), (F, K), (K, F)))
    fp4.fp8_ffn_backward(Q(0, K), Q(K, 0), Q(K, 0), *(ref.transposed(fp4, w) for w in (wg, wu, wd)), e(0, F), e(0, F),
                         fp4.FfnBuffers(0, K, F), e(0, K), dwg, dwu, dwd, ws=ws)
    assert (dwg == 0).all() and (dwu == 0).all() and (dwd == 0).all()


@pytest.mark.parametrize("size", [(24, 384, 640), (2500, 256, 4096)], ids=["few", "many"])
def test_on_a_side_stream_and_in_a_graph(fp4, size):
    """Norm, block and backward on a stream of its own, then captured and replayed: every
    replay gives the eager call's bits."""
    M, K, F = size
    wg, wu, wd = weights(fp4, K, F)
    tw = [ref.transposed(fp4, w) for w in (wg, wu, wd)]
    x, r, w, dy = rnd(M, K).cuda(), rnd(M, K, seed=1).cuda(), torch.ones(K, device="cuda"), rnd(M, K, seed=2).cuda()
    Q = fp4.Fp8Tensor
    e = lambda *s, d=BF16: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    xq, xt, hq, dyq, dyt = Q(M, K), Q(K, M), Q(M, F), Q(M, K), Q(K, M)
    h, rstd, y, g, u = e(M, K), e(M, d=FP32), e(M, K), e(M, F), e(M, F)
    dn, dx, dw, dwg, dwu, dwd = e(M, K), e(M, K), e(K, d=FP32), e(F, K), e(F, K), e(K, F)
    bufs = fp4.FfnBuffers(M, K, F)
    ws = e(max(fp4.fp8_ffn_ws_bytes(M, K, F), fp4.fp8_rms_norm_ws_bytes(M, K)), d=torch.uint8)

    def step():
        fp4.fp8_rms_norm(x, w, EPS, xq, residual=r, h=h, yq_t=xt, rstd=rstd)
        fp4.fp8_ffn_fprop(xq, wg, wu, wd, hq, y, g=g, u=u, ws=ws)
        fp4.fp8_quantize(dy, dyq, dyt)
        fp4.fp8_ffn_backward(dyq, dyt, xt, *tw, g, u, bufs, dn, dwg, dwu, dwd, ws=ws)
        fp4.fp8_rms_norm_backward(dn, h, w, rstd, dx, dw, ws, dh=dy)

    step()
    torch.cuda.synchronize()
    outs = [y, dx, dw, dwg, dwu, dwd, h, hq.codes, bufs.hq_t.codes]
    want = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        step()


def test_example_trains_and_decodes(fp4):
    """The example's block: plain gradient descent on a fixed batch lowers the loss in every
    step from the first to a fraction, and a token decoded alone is the batch's (its
    products may take another order of sums: a few bf16 steps of values of a few units)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_block.py")
    spec = importlib.util.spec_from_file_location("fp8_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, block, (x, r) = m.train(steps=12)
    assert losses[-1] < 0.9 * losses[0], losses
    full = block.forward(x, r).clone()
    for t in (0, 300):
        one = block.decode(x[t:t + 1].contiguous(), r[t:t + 1].contiguous())
        assert (one - full[t:t + 1]).abs().max() <= 2.0 ** -4
