"""Low-rank adapters beside a projection in binary64 (torch), for the tests: written from
include/nvfp4_amd_fp8.h and not from the library.

Tolerances, fixed before the first run.  A binary32 sum is within 1e-5 of its terms'
magnitudes, the products of bf16 and E4M3 values being exact.  With T the sum of
|dropout(x)| |a|, and c_i = scale_i gain of two roundings:
* y and dx: the adapters' part is within (1e-5 + 2^-17 + 1e-5 + 2^-23) |c| T |b| <= 3e-5 |c|
  T |b| (the sum t, its two bf16, the sum over the rank), added to the product's own 1e-5
  sum |x w| (and what a fast product cuts off), and half a step of the bf16 result;
* da and db: (1e-5 + 1e-5 + 2^-23) <= 2.1e-5 of |c| |dt|-magnitudes^T |x|, and 2^-24 of the
  binary32 result.
"""
import torch

import drop_ref
import fp8_ref as ref


class Problem:
    """Adapters, tokens and a mask: inputs on the device as the library takes them, and as
    binary64 values."""

    def __init__(self, fp4, M, N, K, rank, count, spread="mixed", p=0.0, seed=0, device="cuda", dev64=None):
        gen = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.M, self.N, self.K, self.rank, self.count, self.p = M, N, K, rank, count, p
        self.dev64 = dev64 or device
        self.x, self.w = self._held(fp4, rnd(M, K), False, device), self._held(fp4, 0.05 * rnd(N, K), True, device)
        self.w_t = ref.transposed(fp4, self.w) if N * K else fp4.Fp8Tensor(K, N, True, device=device)
        self.dy = self._held(fp4, 1e-3 * rnd(M, N), False, device)
        lda = -(-K // 8) * 8 + 8
        a = torch.full((count, rank, lda), float("nan"))
        a[:, :, :K] = rnd(count, rank, K) * max(K, 1) ** -0.5
        self.a, self.b = a.bfloat16().to(device), (0.1 * rnd(count, N, rank)).bfloat16().to(device)
        self.scale = (torch.rand(count, generator=gen) + 0.5).to(device)
        which = torch.randint(0, count, (M,), generator=gen)
        if spread == "one":
            which[:] = count - 1
        elif spread == "runs":
            which = which.sort().values
        elif spread == "none":
            which[:] = -1
        if spread in ("mixed", "runs") and M > 2:  # some without an adapter, by whatever number
            which[torch.rand(M, generator=gen) < 0.2] = -1
            which[M // 2] = count
            which[M // 3] = -2 ** 31
        self.index = which.int().to(device)
        self.seed, self.offset = 0xABCDEF0123456789 + seed, 2 ** 32 + 7 + seed
        self.drop = fp4.Dropout(p, self.seed, self.offset) if p else None
        self.lora = fp4.LoraAdapters.wrap(self.a, self.b, self.scale, K)

    @staticmethod
    def _held(fp4, v, two_d, device):
        """v quantized by the reference (by the library where that takes long)."""
        if v.numel() == 0:
            return fp4.Fp8Tensor(v.shape[0], v.shape[1], two_d, device=device)
        if v.numel() > 1 << 21:
            q = fp4.Fp8Tensor(v.shape[0], v.shape[1], two_d)
            fp4.fp8_quantize(v.cuda(), q)
            return q
        return ref.put(fp4, v.double(), two_d, device=device)

    def values(self):
        """x, w, dy, a, b, c (per adapter), mask times gain, in binary64."""
        d = self.dev64
        x, w, dy = (ref.values(q).to(d) for q in (self.x, self.w, self.dy))
        a, b = self.a[:, :, :self.K].double().to(d), self.b.double().to(d)
        g = torch.ones(self.M, self.K, dtype=torch.float64, device=d)
        if self.p:
            g = drop_ref.keep(self.M, self.K, self.p, self.seed, self.offset).double().to(d) \
                * (65536 / (65536 - drop_ref.threshold(self.p)))
        return x, w, dy, a, b, self.scale.double().to(d), g

    def rows(self, i):
        return (self.index.to(self.dev64) == i).nonzero()[:, 0]

    def forward(self):
        """(y, the adapters' part of the tolerance)."""
        x, w, _, a, b, s, g = self.values()
        y = x @ w.t().contiguous()
        tol = torch.zeros_like(y)
        for i in range(self.count):
            r = self.rows(i)
            xd, at, bt = x[r] * g[r], a[i].t().contiguous(), b[i].t().contiguous()
            y[r] += s[i] * (xd @ at) @ bt
            tol[r] = 3e-5 * s[i] * (xd.abs() @ at.abs()) @ bt.abs()
        return y, tol

    def backward(self):
        """dx, da, db and, of each, the adapters' part of the tolerance."""
        x, w, dy, a, b, s, g = self.values()
        dx, da, db = dy @ w, torch.zeros_like(a), torch.zeros_like(b)
        out = [torch.zeros_like(t) for t in (dx, da, db)]
        for i in range(self.count):
            r = self.rows(i)
            xd, dyr = x[r] * g[r], dy[r]
            t, dt = xd @ a[i].t().contiguous(), dyr @ b[i]
            ta, dta = xd.abs() @ a[i].abs().t().contiguous(), dyr.abs() @ b[i].abs()
            dx[r] += s[i] * g[r] * (dt @ a[i])
            out[0][r] = 3e-5 * s[i] * g[r] * (dta @ a[i].abs())
            da[i], db[i] = s[i] * dt.t().contiguous() @ xd, s[i] * dyr.t().contiguous() @ t
            out[1][i] = 2.1e-5 * s[i] * dta.t().contiguous() @ xd.abs()
            out[2][i] = 2.1e-5 * s[i] * dyr.abs().t().contiguous() @ ta
        return (dx, da, db), out


def product_tol(a, b, fast, device):
    """The tolerance of the product of two library tensors, [a.rows][b.rows]."""
    x, y = ref.values(a).to(device), ref.values(b).to(device)
    tol = 1e-5 * (x.abs() @ y.abs().t().contiguous())
    if fast:
        def top(v):
            return torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 8)).view(v.shape[0], -1, 8).amax(2)
        tol += 6 * 2.0 ** -13 * torch.sqrt(8 * (top(x).square() @ top(y).square().t().contiguous()))
    return tol


def check(got, want, tol, what=""):
    """|got - want| within tol, and half a step of got's type."""
    half = torch.finfo(got.dtype).eps / 2
    got = got.to(want.device).double()
    far = (got - want).abs() - (tol * (1 + half) + half * want.abs())
    assert not got.isnan().any(), f"{what}: NaN"
    assert (far <= 0).all(), f"{what}: {int((far > 0).sum())} of {far.numel()} out of tolerance, by {float(far.max())}"
