"""Cases, plain forms and exact values of the operators that fine-tune and serve a frozen
8-bit layer: a projection with low-rank adapters of many requests beside it, its
gradients, dropout whose mask is computed where it is needed, and the norm behind a
dropped-out branch, with its gradient.

Projection: y[m] = x[m] W^T + scale_i q (keep . x[m]) A_i^T B_i^T, i = index[m] (no second
term where index[m] is negative).  x [M][K] and W [N][K] are E4M3 with power-of-two scales
(1 x 128 blocks, 128 x 128 tiles: codes [rows][cols rounded up to 128], scale bytes
K-block-major), A_i [rank][K] and B_i [N][rank] are bf16.

keep, of element (r, c) of a [rows][cols] tensor: with g = r ceil(cols / 8) + c // 8, half-word
c % 8 of Philox4x32-10 with counter (g, offset + step) and key seed is at least T =
round(2^16 p); q = 2^16 / (2^16 - T).
"""
import math

import numpy as np
import torch

own = False  # True: run() calls the package's operators

EPS = 1e-6
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token of one request, its adapter among four
        {"name": "lora 1x5120x5120", "op": "lora", "m": 1, "n": 5120, "k": 5120, "rank": 16, "count": 4, "p": 0.0,
         "spread": "mixed", "fast": True},
        # eight requests decode through an up projection, each with an adapter of its own
        {"name": "lora 8x20480x5120", "op": "lora", "m": 8, "n": 20480, "k": 5120, "rank": 16, "count": 8, "p": 0.0,
         "spread": "mixed", "fast": True},
        # ragged prompts of several requests through an odd layer, some without an adapter
        {"name": "lora 333x4100x4090", "op": "lora", "m": 333, "n": 4100, "k": 4090, "rank": 24, "count": 5, "p": 0.0,
         "spread": "runs", "fast": False},
        # a training micro-batch of one adapter
        {"name": "lora train 4096x20480x5120", "op": "lora", "m": 4096, "n": 20480, "k": 5120, "rank": 64, "count": 1,
         "p": 0.05, "spread": "one", "fast": True},
        # a small layer's training step
        {"name": "lora grad 256x2048x512", "op": "lora_grad", "m": 256, "n": 2048, "k": 512, "rank": 8, "count": 1,
         "p": 0.0, "spread": "one", "fast": False},
        # several tenants' sequences in one batch, odd sizes
        {"name": "lora grad 777x2501x1030", "op": "lora_grad", "m": 777, "n": 2501, "k": 1030, "rank": 32, "count": 7,
         "p": 0.1, "spread": "runs", "fast": False},
        # the micro-batch's backward pass
        {"name": "lora grad 4096x20480x5120", "op": "lora_grad", "m": 4096, "n": 20480, "k": 5120, "rank": 16,
         "count": 1, "p": 0.05, "spread": "one", "fast": True},
        # the smallest call: launch latency
        {"name": "dropout 8x5120", "op": "dropout", "tokens": 8, "width": 5120, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # a micro-batch's branch back into the residual stream
        {"name": "dropout 16384x5120", "op": "dropout", "tokens": 16384, "width": 5120, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # the same in front of the next block's norm, both layouts of its output
        {"name": "dropout norm 16384x5120", "op": "norm", "tokens": 16384, "width": 5120, "dtype": "bf16", "p": 0.1,
         "train": True},
        # and its backward pass
        {"name": "dropout norm grad 16384x5120", "op": "norm_grad", "tokens": 16384, "width": 5120, "dtype": "bf16",
         "p": 0.1},
        # a width that is no multiple of a block or a vector, in fp32 (a debugging run of a small layer)
        {"name": "dropout norm grad 777x2501", "op": "norm_grad", "tokens": 777, "width": 2501, "dtype": "fp32",
         "p": 0.25},
    ]


def draw(rng):
    def size(lo, hi):
        """Spread over the logarithm; now and then a round number, most often not."""
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, v // 128 * 128) if v >= 256 and rng.random() < 0.5 else v

    op = rng.choice(["lora", "lora", "lora_grad", "lora_grad", "dropout", "norm", "norm_grad"])
    p = rng.choice([0.0, 0.05, 0.1, round(rng.uniform(0.01, 0.6), 3)])
    if op in ("lora", "lora_grad"):
        m = size(1, 4096)
        spread = rng.choice(["one", "runs", "mixed"])
        return {"op": op, "m": m, "n": size(64, 16384), "k": size(64, 5120), "rank": 8 * rng.choice([1, 2, 2, 3, 4, 8, 16]),
                "count": 1 if spread == "one" else rng.randint(2, 16), "p": p if op == "lora_grad" or m > 64 else 0.0,
                "spread": spread, "fast": rng.random() < 0.5}
    c = {"op": op, "tokens": size(1, 16384), "width": size(64, 5120), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
         "p": p or 0.1}
    if op == "dropout":
        c["residual"] = rng.random() < 0.5  # without: the gradient's call
    if op == "norm":
        c["train"] = rng.random() < 0.5
    return c


# -------------------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _laplace(gen, *shape, scale=1e-3, dtype=torch.bfloat16):
    u = torch.rand(*shape, generator=gen, device="cuda") - 0.5
    return (-scale * torch.sign(u) * torch.log1p(-2 * u.abs().clamp(max=0.4999999))).to(dtype)


def _held(x, two_d=False):
    """x quantized, as a program holds it between calls: codes and scales as bytes, the
    scales' rows rounded up to 16."""
    codes, scales = _quantize(x.float(), two_d)
    e = (torch.log2(scales) + 127).to(torch.uint8)
    if not two_d:
        e = torch.nn.functional.pad(e, (0, -x.shape[0] % 16), value=127)
    return codes.view(torch.uint8), e.contiguous(), x.shape[0], x.shape[1], two_d


def _held_transpose(q):
    """The transpose of a tensor with tile scales: the same values."""
    codes, e, rows, cols, two_d = q
    t = torch.zeros(cols, -(-rows // BLOCK) * BLOCK, dtype=torch.uint8, device=codes.device)
    t[:, :rows] = codes[:, :cols].t()
    return t, e.t().contiguous(), cols, rows, two_d


def _index(gen, case):
    """The adapter of each token: all the first, runs of sequences, or a request to a token;
    one in ten of the last two without one."""
    m, n = case["m"], case["count"]
    if case["spread"] == "one":
        return torch.zeros(m, dtype=torch.int32, device="cuda")
    run = 1 if case["spread"] == "mixed" else max(1, m // (2 * n))
    which = torch.randint(0, n, (-(-m // run),), generator=gen, device="cuda")
    if m == 1:
        return which.int()
    none = torch.rand(which.shape, generator=gen, device="cuda") < 0.1
    return torch.where(none, torch.full_like(which, -1), which).repeat_interleave(run)[:m].int().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    op, s = case["op"], {"case": case}
    s["seed"], s["offset"] = seed * 2654435761 % (1 << 62) + (1 << 40), 5 + seed % 1000
    s["step"] = torch.full((1,), 7 + seed % 100, dtype=torch.int64, device="cuda")  # a training run's counter
    if op in ("lora", "lora_grad"):
        m, n, k, r, count = (case[x] for x in ("m", "n", "k", "rank", "count"))
        s["x"] = _held(_normal(gen, m, k))
        w = _held(_normal(gen, n, k, std=0.02), True)
        # rows padded to 8 elements, as the adapters are stored
        s["a"] = torch.zeros(count, r, -(-k // 8) * 8, dtype=torch.bfloat16, device="cuda")
        s["a"][:, :, :k] = _normal(gen, count, r, k, std=k ** -0.5)
        s["b"] = _normal(gen, count, n, r, std=0.05)
        s["scale"] = torch.rand(count, generator=gen, device="cuda") + 0.5
        s["index"] = _index(gen, case)
        if op == "lora":
            s["w"] = w
        else:
            s["w_t"] = _held_transpose(w)
            s["dy"] = _held(_laplace(gen, m, n))
        return s
    m, c, t = case["tokens"], case["width"], DTYPES[case["dtype"]]
    if op == "dropout":
        s["x"] = _normal(gen, m, c, dtype=t)
        s["residual"] = _normal(gen, m, c, std=2.0, dtype=t) if case["residual"] else None
        return s
    s["weight"] = 1 + _normal(gen, c, std=0.1, dtype=torch.float32)
    if op == "norm":
        s["x"], s["residual"] = _normal(gen, m, c, dtype=t), _normal(gen, m, c, std=2.0, dtype=t)
        return s
    s["h"], s["dh"] = _normal(gen, m, c, std=2.0, dtype=t), _laplace(gen, m, c, dtype=t)
    s["dy"] = _laplace(gen, m, c, dtype=t)
    s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
    return s


# ---------------------------------------------------------------------- plain forms

def _scale_of(amax):
    """The smallest power of two with amax <= 448 * 2^e, e in [-126, 127] (1 for a
    block of zeros), from the bits of a non-negative binary32."""
    bits = amax.view(torch.int32)
    e = ((bits + (0x7FFFFF - 0x600000)) >> 23) - 8  # biased
    e = torch.where(bits == 0, torch.full_like(e, 127), e.clamp(1, 254))
    return (e << 23).view(torch.float32)


def _quantize(v, two_d):
    """(codes as E4M3 values, scales as values) of a binary32 tensor, in the layout of
    the module's docstring."""
    rows, cols = v.shape
    kb = -(-cols // BLOCK)
    v = torch.nn.functional.pad(v, (0, kb * BLOCK - cols))
    if two_d:
        rb = -(-rows // BLOCK)
        t = torch.nn.functional.pad(v, (0, 0, 0, rb * BLOCK - rows)).view(rb, BLOCK, kb, BLOCK)
        scale = _scale_of(t.abs().amax((1, 3)))
        codes = (t / scale[:, None, :, None]).view(rb * BLOCK, -1)[:rows]
    else:
        t = v.view(rows, kb, BLOCK)
        scale = _scale_of(t.abs().amax(2))
        codes = (t / scale[:, :, None]).view(rows, -1)
    return codes.contiguous().to(torch.float8_e4m3fn), scale.t().contiguous()


def _values(q):
    """The binary32 values that a held quantized tensor stands for."""
    codes, scales, rows, cols, two_d = q
    v = codes.view(torch.float8_e4m3fn).float()
    s = (scales.to(torch.int32) << 23).view(torch.float32).t()
    s = s.repeat_interleave(BLOCK, 0)[:rows] if two_d else s[:rows]
    return (v.view(rows, -1, BLOCK) * s[:, :, None]).view(rows, -1)[:, :cols]


def _as_outputs(q):
    return {"codes": q[0], "scales": q[1].to(torch.float8_e8m0fnu)}


def _threshold(p):
    return int(round(p * 65536))


def _keep(s, rows, cols):
    """The mask of a [rows][cols] tensor: Philox4x32-10 on 64-bit integers that hold 32."""
    groups = -(-cols // 8)
    low = 0xFFFFFFFF
    g = torch.arange(rows * groups, dtype=torch.int64, device="cuda")
    at = s["offset"] + s["step"]
    c = [g & low, g >> 32, (at & low).expand_as(g), (at >> 32).expand_as(g)]
    key = [s["seed"] & low, s["seed"] >> 32]

    def product(m, v):  # the two halves of a 32 x 32-bit product
        high = (m * (v >> 16) + (m * (v & 0xFFFF) >> 16)) >> 16
        return high, (m * v) & low

    for _ in range(10):
        h0, l0 = product(0xD2511F53, c[0])
        h1, l1 = product(0xCD9E8D57, c[2])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    halves = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 1)
    return halves.view(rows, groups * 8)[:, :cols] >= _threshold(s["case"]["p"])


def _dropped(s, x, keep=None):
    """x dropped out, in binary32, by the mask `keep` where it is at hand."""
    t = _threshold(s["case"]["p"])
    if t == 0:
        return x
    keep = _keep(s, *x.shape) if keep is None else keep
    return torch.where(keep, x * (65536 / (65536 - t)), torch.zeros_like(x))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("lora", "lora_grad"):
        k = c["k"]
        x, index = _values(s["x"]), s["index"]
        keep = _keep(s, *x.shape) if c["p"] else None
        xd = _dropped(s, x, keep)
        # the adapters side by side: [count * rank][k] and [count * rank][n]
        a = s["a"][:, :, :k].float().reshape(-1, k)
        b = s["b"].float().transpose(1, 2).reshape(-1, c["n"])
        mine = (index[:, None] == torch.arange(c["count"], device="cuda")).repeat_interleave(c["rank"], 1)
        gain = s["scale"].repeat_interleave(c["rank"])
        t = torch.where(mine, xd @ a.t() * gain, torch.zeros((), device="cuda"))
        if op == "lora":
            return {"y": (x @ _values(s["w"]).t() + t @ b).bfloat16()}
        dy = _values(s["dy"])
        dt = torch.where(mine, dy @ b.t() * gain, torch.zeros((), device="cuda"))
        dx = dy @ _values(s["w_t"]).t() + _dropped(s, dt @ a, keep)
        da = (dt.t() @ xd).view(c["count"], c["rank"], k)
        db = (t.t() @ dy).view(c["count"], c["rank"], c["n"]).transpose(1, 2).contiguous()
        return {"dx": dx.bfloat16(), "da": da, "db": db}
    if op == "dropout":
        y = _dropped(s, s["x"].float())
        return {"y": (y if s["residual"] is None else s["residual"].float() + y).to(s["x"].dtype)}
    if op == "norm":
        h = (_dropped(s, s["x"].float()) + s["residual"].float()).to(s["x"].dtype)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(1) + EPS)
        y = hf * rstd[:, None] * s["weight"]
        out = {"h": h, "y": _as_outputs(_quantize(y, False))}
        if c["train"]:
            out |= {"rstd": rstd, "y_t": _as_outputs(_quantize(y.t().contiguous(), False))}
        return out
    hhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    v = dy * s["weight"]
    dres = s["dh"].float() + s["rstd"][:, None] * (v - hhat * (v * hhat).mean(1, keepdim=True))
    return {"dx": _dropped(s, dres).to(s["h"].dtype), "dresidual": dres.to(s["h"].dtype),
            "dweight": (dy * hhat).double().sum(0).float()}


# ------------------------------------------------------------------ the package's calls

def _package():
    import nvfp4_bit_microscaled_amd as fp4
    return fp4


def _kept(s, name, make):
    """A buffer, descriptor or workspace that a program makes once and uses at every call."""
    key = "_" + name
    if key not in s:
        s[key] = make()
    return s[key]


def _handle(s, name):
    return _kept(s, name, lambda: _package().Fp8Tensor.wrap(*s[name]))


def _outputs_of(q):
    scales = q.scales if q.two_d else q.scales[:, :q.rows]
    return {"codes": q.codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _workspace(s, need):
    return _kept(s, "ws", lambda: torch.empty(max(need(), 16), dtype=torch.uint8, device="cuda"))


def _own(s):
    fp4, c = _package(), s["case"]
    op = c["op"]
    drop = _kept(s, "drop", lambda: fp4.Dropout(c["p"], s["seed"], s["offset"], s["step"]) if c["p"] else None)
    if op in ("lora", "lora_grad"):
        m, n, k, r, count = (c[x] for x in ("m", "n", "k", "rank", "count"))
        ad = _kept(s, "ad", lambda: fp4.LoraAdapters.wrap(s["a"], s["b"], s["scale"], k))
        if op == "lora":
            y = _kept(s, "y", lambda: torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))
            ws = _workspace(s, lambda: fp4.fp8_lora_fprop_ws_bytes(m, n, k, r, fast=c["fast"]))
            fp4.fp8_lora_fprop(_handle(s, "x"), _handle(s, "w"), ad, y, index=s["index"], drop=drop, ws=ws,
                               fast=c["fast"])
            return {"y": y}
        dx = _kept(s, "dx", lambda: torch.empty(m, k, dtype=torch.bfloat16, device="cuda"))
        da = _kept(s, "da", lambda: torch.empty(s["a"].shape, dtype=torch.float32, device="cuda"))
        db = _kept(s, "db", lambda: torch.empty(s["b"].shape, dtype=torch.float32, device="cuda"))
        ws = _workspace(s, lambda: fp4.fp8_lora_backward_ws_bytes(m, n, k, r, count, fast=c["fast"]))
        fp4.fp8_lora_backward(_handle(s, "dy"), _handle(s, "w_t"), _handle(s, "x"), ad, dx, da, db, ws,
                              index=s["index"], drop=drop, fast=c["fast"])
        return {"dx": dx, "da": da[:, :, :k], "db": db}
    m, w = c["tokens"], c["width"]
    if op == "dropout":
        y = _kept(s, "y", lambda: torch.empty_like(s["x"]))
        fp4.fp8_dropout(s["x"], drop, y, residual=s["residual"])
        return {"y": y}
    if op == "norm":
        h, yq = _kept(s, "h", lambda: torch.empty_like(s["x"])), _kept(s, "yq", lambda: fp4.Fp8Tensor(m, w))
        if not c["train"]:
            fp4.fp8_dropout_rms_norm(s["x"], drop, s["weight"], EPS, yq, s["residual"], h)
            return {"h": h, "y": _outputs_of(yq)}
        yq_t = _kept(s, "yq_t", lambda: fp4.Fp8Tensor(w, m))
        rstd = _kept(s, "rstd", lambda: torch.empty(m, dtype=torch.float32, device="cuda"))
        fp4.fp8_dropout_rms_norm(s["x"], drop, s["weight"], EPS, yq, s["residual"], h, yq_t=yq_t, rstd=rstd)
        return {"h": h, "y": _outputs_of(yq), "rstd": rstd, "y_t": _outputs_of(yq_t)}
    dx, dres = (_kept(s, x, lambda: torch.empty_like(s["h"])) for x in ("dx", "dres"))
    dw = _kept(s, "dw", lambda: torch.empty(w, dtype=torch.float32, device="cuda"))
    ws = _workspace(s, lambda: fp4.fp8_rms_norm_ws_bytes(m, w))
    fp4.fp8_dropout_rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], drop, dx, dres, dw, ws, dh=s["dh"])
    return {"dx": dx, "dresidual": dres, "dweight": dw}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------- work and truth

def work(case):
    op = case["op"]
    if op in ("lora", "lora_grad"):
        m, n, k, r, count = (case[x] for x in ("m", "n", "k", "rank", "count"))
        weights = 2 * min(count, m) * r * (k + n)
        if op == "lora":
            return {"bytes": m * k + n * k + weights + 2 * m * n, "flops": 2 * m * n * k + 2 * m * r * (k + n)}
        return {"bytes": m * n + m * k + n * k + weights + 2 * m * k + 4 * count * r * (k + n),
                "flops": 2 * m * n * k + m * r * (6 * k + 4 * n)}
    m, c = case["tokens"], case["width"]
    n, t = m * c, 2 if case["dtype"] == "bf16" else 4
    if op == "dropout":
        return {"bytes": n * t * (3 if case["residual"] else 2), "flops": 3 * n}
    if op == "norm":
        return {"bytes": n * (3 * t + 1 + case["train"]) + 4 * (c + m * case["train"]), "flops": 10 * n}
    return {"bytes": n * 5 * t + 4 * (2 * c + m), "flops": 14 * n}


def _exact_gain(s, rows, cols):
    """What a [rows][cols] tensor is multiplied by: 0 or q, in binary64, from Philox on
    numpy's unsigned integers."""
    t = _threshold(s["case"]["p"])
    if t == 0:
        return torch.ones((), dtype=torch.float64, device="cuda")
    groups = (cols + 7) // 8
    at = s["offset"] + int(s["step"].item())
    u, m32 = np.uint64, np.uint64(0xFFFFFFFF)
    counter = np.arange(rows * groups, dtype=np.uint64)
    x0, x1 = counter & m32, counter >> u(32)
    x2, x3 = np.full_like(x0, at & 0xFFFFFFFF), np.full_like(x0, at >> 32)
    for i in range(10):
        k0 = u((s["seed"] + i * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = u(((s["seed"] >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
        p, q = x0 * u(0xD2511F53), x2 * u(0xCD9E8D57)
        x0, x1, x2, x3 = (q >> u(32)) ^ x1 ^ k0, q & m32, (p >> u(32)) ^ x3 ^ k1, p & m32
    words = np.stack([x0, x1, x2, x3], axis=1).astype("<u4")
    kept = words.view("<u2").reshape(rows, groups * 8)[:, :cols] >= t
    return torch.from_numpy(kept).cuda().double() * (65536 / (65536 - t))


def _e4m3(v):
    """Nearest E4M3 value (ties to the even code) of binary64 values within +-448:
    8 steps to an octave, the octaves below 2^-6 sharing its step."""
    step = torch.exp2(torch.frexp(v)[1].clamp(min=-5).double() - 4)
    return torch.round(v / step) * step


def _exact_quantize(v):
    """(grid values, scales) in binary64, 1 x 128 blocks: the scale from the logarithm's
    definition, corrected where the logarithm rounds across a power of two."""
    rows, cols = v.shape
    kb = -(-cols // BLOCK)
    full = torch.zeros(rows, kb * BLOCK, dtype=torch.float64, device=v.device)
    full[:, :cols] = v
    t = full.view(rows, kb, BLOCK)
    amax = t.abs().amax(2)
    e = torch.ceil(torch.log2(amax / 448))
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e))
    scale = torch.where(amax == 0, torch.ones_like(amax), torch.exp2(e.clamp(-126, 127)))
    return {"codes": _e4m3(t / scale[:, :, None]).view(rows, -1), "scales": scale.t()}


def _exact_held(q):
    codes, scales, rows, cols, two_d = q
    v = codes.view(torch.float8_e4m3fn).double()[:, :cols]
    s = torch.exp2(scales.double() - 127)
    i = torch.arange(rows, device=v.device) // (BLOCK if two_d else 1)
    j = torch.arange(cols, device=v.device) // BLOCK
    return v * s[:, i].t()[:, j]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("lora", "lora_grad"):
        m, k = case["m"], case["k"]
        x, gain = _exact_held(s["x"]), _exact_gain(s, m, k)
        groups = [(i, (s["index"] == i).nonzero()[:, 0]) for i in range(case["count"])]
        a, b, scale = s["a"][:, :, :k].double(), s["b"].double(), s["scale"].double()
        xd = x * gain
        if op == "lora":
            y = x.matmul(_exact_held(s["w"]).t().contiguous())
            for i, rows in groups:
                y[rows] += (xd[rows] @ a[i].t().contiguous() * scale[i]) @ b[i].t().contiguous()
            return {"y": y}
        dy = _exact_held(s["dy"])
        dx = dy.matmul(_exact_held(s["w_t"]).t().contiguous())
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for i, rows in groups:
            delta = (b[i] * scale[i]) @ a[i]  # what the adapter adds to the weight
            dx[rows] += dy[rows] @ delta * (gain[rows] if gain.dim() else gain)
            dyt = dy[rows].t().contiguous() * scale[i]
            da[i] = (dyt.t() @ b[i]).t().contiguous() @ xd[rows]
            db[i] = dyt @ (xd[rows] @ a[i].t().contiguous())
        return {"dx": dx, "da": da, "db": db}
    if op == "dropout":
        y = s["x"].double() * _exact_gain(s, *s["x"].shape)
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    if op == "norm":
        total = s["x"].double() * _exact_gain(s, *s["x"].shape) + s["residual"].double()
        h = total.float().to(s["x"].dtype).double()  # the residual stream's own type
        rstd = 1 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
        y = h * rstd[:, None] * s["weight"].double()
        out = {"h": total, "y": _exact_quantize(y)}
        if case["train"]:
            out |= {"rstd": rstd, "y_t": _exact_quantize(y.t())}
        return out
    h, r, w, dy = (s[n].double() for n in ("h", "rstd", "weight", "dy"))
    wdy = w * dy
    dot = (wdy * h).sum(1) * r ** 3 / h.shape[1]
    dres = s["dh"].double() + wdy * r[:, None] - h * dot[:, None]
    return {"dx": dres * _exact_gain(s, *h.shape), "dresidual": dres, "dweight": r @ (dy * h)}
