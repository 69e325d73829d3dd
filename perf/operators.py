"""Cases, plain forms and exact values of the E4M3 operators of a gated feed-forward
block: root-mean-square norm with the residual's addition and an 8-bit output, its
gradient, block-of-128 quantization, the product of two quantized operands, and the
gated block (both projections, activation and product; down projection) with its
gradients.

A quantized tensor of `rows` x `cols` has E4M3 codes [rows][cols rounded up to 128]
(zeros past cols) and one power-of-two scale (E8M0) per 1 x 128 block, or per 128 x 128
tile for weights, K-block-major: [blocks along cols][rows], or [blocks along cols]
[blocks along rows] for tiles.  The scale is the smallest 2^e with amax <= 448 * 2^e.
"""
import math

import torch

own = False  # True: run() calls the package's operators

EPS = 1e-6
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one token entering a 5120-wide block while decoding: launch latency
        {"name": "norm 1x5120", "op": "norm", "tokens": 1, "width": 5120, "dtype": "bf16", "train": False},
        # a training micro-batch: both layouts of the normalised activations
        {"name": "norm train 16384x5120", "op": "norm", "tokens": 16384, "width": 5120, "dtype": "bf16",
         "train": True},
        # the same micro-batch's backward pass
        {"name": "norm grad 16384x5120", "op": "norm_grad", "tokens": 16384, "width": 5120, "dtype": "bf16"},
        # a width that is no multiple of a block or a vector, in fp32 (a debugging run of a small layer)
        {"name": "norm grad 777x2501 fp32", "op": "norm_grad", "tokens": 777, "width": 2501, "dtype": "fp32"},
        # a gradient's two layouts for dgrad and wgrad
        {"name": "quantize 8192x4096", "op": "quantize", "tokens": 8192, "width": 4096, "dtype": "bf16",
         "two_d": False},
        # a weight after its update, with the transpose that dgrad reads
        {"name": "quantize weight 20480x5120", "op": "quantize", "tokens": 20480, "width": 5120, "dtype": "fp32",
         "two_d": True},
        # a linear layer for four decoded tokens: the weights' bytes
        {"name": "gemm 4x20480x5120", "op": "gemm", "m": 4, "n": 20480, "k": 5120, "two_d": True, "dtype": "bf16"},
        # a ragged prompt through an odd layer
        {"name": "gemm 333x4100x4090", "op": "gemm", "m": 333, "n": 4100, "k": 4090, "two_d": True, "dtype": "bf16"},
        # the weight gradient of an up projection over a micro-batch
        {"name": "gemm 20480x5120x16384", "op": "gemm", "m": 20480, "n": 5120, "k": 16384, "two_d": False,
         "dtype": "fp32"},
        # the gated block for eight decoded tokens
        {"name": "ffn 8x5120x20480", "op": "ffn", "tokens": 8, "width": 5120, "inner": 20480, "train": False},
        # its training pass over 4096 tokens, gate and up kept for the backward
        {"name": "ffn train 4096x5120x20480", "op": "ffn", "tokens": 4096, "width": 5120, "inner": 20480,
         "train": True},
        # and the backward pass of those tokens
        {"name": "ffn grad 4096x5120x20480", "op": "ffn_grad", "tokens": 4096, "width": 5120, "inner": 20480},
    ]


def draw(rng):
    def size(lo, hi):
        """Spread over the logarithm; now and then a round number, most often not."""
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, v // 128 * 128) if v >= 256 and rng.random() < 0.5 else v

    op = rng.choice(["norm", "norm_grad", "quantize", "gemm", "ffn", "ffn_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_grad", "quantize"):
        c = {"op": op, "tokens": size(1, 16384), "width": size(64, 5120), "dtype": dtype}
        if op == "norm":
            c["train"] = rng.random() < 0.5
        if op == "quantize":
            c["two_d"] = rng.random() < 0.3
        return c
    if op == "gemm":
        return {"op": op, "m": size(1, 16384), "n": size(64, 16384), "k": size(64, 8192), "two_d": rng.random() < 0.6,
                "dtype": dtype}
    c = {"op": op, "tokens": size(1, 4096), "width": size(64, 5120), "inner": size(128, 16384)}
    if op == "ffn":
        c["train"] = rng.random() < 0.5
    return c


# -------------------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _laplace(gen, *shape, scale=1e-3, dtype=torch.bfloat16):
    u = torch.rand(*shape, generator=gen, device="cuda") - 0.5
    return (-scale * torch.sign(u) * torch.log1p(-2 * u.abs().clamp(max=0.4999999))).to(dtype)


def _transposed(q):
    """The quantized transpose of a tensor with tile scales (the same values)."""
    codes, scales, rows, cols, two_d = q
    t = torch.zeros(cols, -(-rows // BLOCK) * BLOCK, dtype=torch.uint8, device=codes.device)
    t[:, :rows] = codes[:, :cols].t()
    return t.view(torch.float8_e4m3fn), scales.t().contiguous(), cols, rows, two_d


def _held(x, two_d=False):
    """x quantized, as a program holds it between calls: (codes, scales, rows, cols,
    two_d), codes and scales as bytes, the scales' rows rounded up to 16."""
    codes, scales = _quantize(x.float(), two_d)
    e = (torch.log2(scales) + 127).to(torch.uint8)
    if not two_d:
        e = torch.nn.functional.pad(e, (0, -x.shape[0] % 16), value=127)
    return codes.view(torch.uint8), e.contiguous(), x.shape[0], x.shape[1], two_d


def _bytes(q):
    return q[0].view(torch.uint8), q[1], q[2], q[3], q[4]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_grad", "quantize"):
        m, c, t = case["tokens"], case["width"], DTYPES[case["dtype"]]
        if op == "quantize":
            s["x"] = _normal(gen, m, c, std=0.02, dtype=t) if case["two_d"] else _laplace(gen, m, c, dtype=t)
            return s
        s["weight"] = 1 + _normal(gen, c, std=0.1, dtype=torch.float32)
        if op == "norm":
            s["x"], s["residual"] = _normal(gen, m, c, dtype=t), _normal(gen, m, c, std=2.0, dtype=t)
            return s
        s["h"], s["dh"] = _normal(gen, m, c, std=2.0, dtype=t), _laplace(gen, m, c, dtype=t)
        s["dy"] = _laplace(gen, m, c, dtype=t)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        return s
    if op == "gemm":
        a = _normal(gen, case["m"], case["k"]) if case["two_d"] else _laplace(gen, case["m"], case["k"])
        s["a"] = _held(a)
        s["b"] = _held(_normal(gen, case["n"], case["k"], std=0.02 if case["two_d"] else 1.0), case["two_d"])
        return s
    m, k, f = case["tokens"], case["width"], case["inner"]
    wg = _held(_normal(gen, f, k, std=0.02), True)
    wu = _held(_normal(gen, f, k, std=0.02), True)
    wd = _held(_normal(gen, k, f, std=0.02), True)
    x = _normal(gen, m, k)
    if op == "ffn":
        return s | {"wg": wg, "wu": wu, "wd": wd, "x": _held(x)}
    dy = _laplace(gen, m, k)
    return s | {"wg_t": _bytes(_transposed(wg)), "wu_t": _bytes(_transposed(wu)), "wd_t": _bytes(_transposed(wd)),
                "x_t": _held(x.t()), "dy": _held(dy), "dy_t": _held(dy.t()),
                "g": _normal(gen, m, f), "u": _normal(gen, m, f)}


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


def _round_trip(v):
    codes, scales = _quantize(v, False)
    return (codes.float().view(v.shape[0], -1, BLOCK) * scales.t()[:, :, None]).view(v.shape[0], -1)[:, :v.shape[1]]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(1) + EPS)
        y = hf * rstd[:, None] * s["weight"]
        out = {"h": h, "y": _as_outputs(_quantize(y, False))}
        if c["train"]:
            out |= {"rstd": rstd, "y_t": _as_outputs(_quantize(y.t().contiguous(), False))}
        return out
    if op == "norm_grad":
        hhat = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        v = dy * s["weight"]
        dx = s["dh"].float() + s["rstd"][:, None] * (v - hhat * (v * hhat).mean(1, keepdim=True))
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * hhat).double().sum(0).float()}
    if op == "quantize":
        x = s["x"].float()
        return {"q": _as_outputs(_quantize(x, c["two_d"])),
                "q_t": _as_outputs(_quantize(x.t().contiguous(), c["two_d"]))}
    if op == "gemm":
        return {"c": (_values(s["a"]) @ _values(s["b"]).t()).to(DTYPES[c["dtype"]])}
    if op == "ffn":
        x = _values(s["x"])
        g, u = (x @ _values(s["wg"]).t()).bfloat16(), (x @ _values(s["wu"]).t()).bfloat16()
        gf = g.float()
        y = (_round_trip(gf / (1 + torch.exp(-gf)) * u.float()) @ _values(s["wd"]).t()).bfloat16()
        return {"y": y, "g": g, "u": u} if c["train"] else {"y": y}
    dh = _values(s["dy"]) @ _values(s["wd_t"]).t()
    g, u = s["g"].float(), s["u"].float()
    sig = 1 / (1 + torch.exp(-g))
    act = g * sig
    dg, du = dh * u * (sig * (1 + g * (1 - sig))), dh * act
    x_t, h_t = _values(s["x_t"]), _round_trip((act * u).t())
    dx = _round_trip(dg) @ _values(s["wg_t"]).t() + _round_trip(du) @ _values(s["wu_t"]).t()
    return {"dx": dx.bfloat16(), "dwg": (_round_trip(dg.t()) @ x_t.t()).bfloat16(),
            "dwu": (_round_trip(du.t()) @ x_t.t()).bfloat16(), "dwd": (_values(s["dy_t"]) @ h_t.t()).bfloat16()}


def _as_outputs(q):
    return {"codes": q[0], "scales": q[1].to(torch.float8_e8m0fnu)}


# ------------------------------------------------------------------ the package's calls

def _package():
    import nvfp4_bit_microscaled_amd as fp4
    return fp4


def _handle(s, name):
    """The package's descriptor of a held quantized tensor, made once per state."""
    key = "_" + name
    if key not in s:
        codes, scales, rows, cols, two_d = s[name]
        s[key] = _package().Fp8Tensor.wrap(codes, scales, rows, cols, two_d)
    return s[key]


def _kept(s, name, make):
    """A buffer or workspace that a program allocates once and uses at every call."""
    key = "_" + name
    if key not in s:
        s[key] = make()
    return s[key]


def _outputs_of(q):
    scales = q.scales if q.two_d else q.scales[:, :q.rows]
    return {"codes": q.codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _workspace(s, need):
    return _kept(s, "ws", lambda: torch.empty(max(need(), 16), dtype=torch.uint8, device="cuda"))


def _own(s):
    fp4, c = _package(), s["case"]
    op = c["op"]
    if op == "norm":
        m, w = s["x"].shape
        h, yq = _kept(s, "h", lambda: torch.empty_like(s["x"])), _kept(s, "yq", lambda: fp4.Fp8Tensor(m, w))
        if not c["train"]:
            fp4.fp8_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], h=h, yq=yq)
            return {"h": h, "y": _outputs_of(yq)}
        yq_t = _kept(s, "yq_t", lambda: fp4.Fp8Tensor(w, m))
        rstd = _kept(s, "rstd", lambda: torch.empty(m, dtype=torch.float32, device="cuda"))
        fp4.fp8_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], h=h, yq=yq, yq_t=yq_t, rstd=rstd)
        return {"h": h, "y": _outputs_of(yq), "rstd": rstd, "y_t": _outputs_of(yq_t)}
    if op == "norm_grad":
        m, w = s["h"].shape
        dx = _kept(s, "dx", lambda: torch.empty_like(s["h"]))
        dw = _kept(s, "dw", lambda: torch.empty(w, dtype=torch.float32, device="cuda"))
        ws = _workspace(s, lambda: fp4.fp8_rms_norm_ws_bytes(m, w))
        fp4.fp8_rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dx, dw, ws, dh=s["dh"])
        return {"dx": dx, "dweight": dw}
    if op == "quantize":
        m, w = s["x"].shape
        q = _kept(s, "q", lambda: fp4.Fp8Tensor(m, w, c["two_d"]))
        q_t = _kept(s, "q_t", lambda: fp4.Fp8Tensor(w, m, c["two_d"]))
        fp4.fp8_quantize(s["x"], q, q_t)
        return {"q": _outputs_of(q), "q_t": _outputs_of(q_t)}
    if op == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        out = _kept(s, "c", lambda: torch.empty(m, n, dtype=DTYPES[c["dtype"]], device="cuda"))
        ws = _workspace(s, lambda: fp4.fp8_gemm_ws_bytes(m, n, k))
        # a bf16 product is within its own rounding either way; binary32 gradients are summed in full
        fp4.fp8_gemm(_handle(s, "a"), _handle(s, "b"), out, ws, fast=c["dtype"] == "bf16")
        return {"c": out}
    m, k, f = c["tokens"], c["width"], c["inner"]
    ws = _workspace(s, lambda: fp4.fp8_ffn_ws_bytes(m, k, f))
    if op == "ffn":
        y = _kept(s, "y", lambda: torch.empty(m, k, dtype=torch.bfloat16, device="cuda"))
        hq = _kept(s, "hq", lambda: fp4.Fp8Tensor(m, f))
        g, u = (_kept(s, n, lambda: torch.empty(m, f, dtype=torch.bfloat16, device="cuda")) if c["train"] else None
                for n in ("g", "u"))
        fp4.fp8_ffn_fprop(_handle(s, "x"), _handle(s, "wg"), _handle(s, "wu"), _handle(s, "wd"), hq, y, g=g, u=u, ws=ws)
        return {"y": y, "g": g, "u": u} if c["train"] else {"y": y}
    bufs = _kept(s, "bufs", lambda: fp4.FfnBuffers(m, k, f))
    dx = _kept(s, "dx", lambda: torch.empty(m, k, dtype=torch.bfloat16, device="cuda"))
    dwg, dwu = (_kept(s, n, lambda: torch.empty(f, k, dtype=torch.bfloat16, device="cuda")) for n in ("dwg", "dwu"))
    dwd = _kept(s, "dwd", lambda: torch.empty(k, f, dtype=torch.bfloat16, device="cuda"))
    fp4.fp8_ffn_backward(_handle(s, "dy"), _handle(s, "dy_t"), _handle(s, "x_t"), _handle(s, "wg_t"),
                         _handle(s, "wu_t"), _handle(s, "wd_t"), s["g"], s["u"], bufs, dx, dwg, dwu, dwd, ws=ws)
    return {"dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------- work and truth

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad", "quantize"):
        n, c, m = case["tokens"] * case["width"], case["width"], case["tokens"]
        t = 2 if case["dtype"] == "bf16" else 4
        if op == "quantize":
            return {"bytes": n * (t + 2), "flops": 4 * n}
        if op == "norm":
            return {"bytes": n * (3 * t + 1 + case["train"]) + 4 * (c + m * case["train"]), "flops": 8 * n}
        return {"bytes": n * 4 * t + 4 * (2 * c + m), "flops": 12 * n}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * (2 if case["dtype"] == "bf16" else 4), "flops": 2 * m * n * k}
    m, k, f = case["tokens"], case["width"], case["inner"]
    if op == "ffn":
        return {"bytes": 3 * k * f + m * k * 3 + (4 * m * f if case["train"] else 0), "flops": 6 * m * k * f}
    return {"bytes": 3 * k * f + 3 * m * k + 4 * m * f + 2 * m * k + 6 * k * f, "flops": 12 * m * k * f}


def _e4m3(v):
    """Nearest E4M3 value (ties to the even code) of binary64 values within +-448:
    8 steps to an octave, the octaves below 2^-6 sharing its step."""
    step = torch.exp2(torch.frexp(v)[1].clamp(min=-5).double() - 4)
    return torch.round(v / step) * step


def _exact_quantize(v, two_d):
    """(grid values, scales) in binary64: the scale from the logarithm's definition,
    corrected where the logarithm rounds across a power of two."""
    rows, cols = v.shape
    rb, kb = (-(-rows // BLOCK) if two_d else rows), -(-cols // BLOCK)
    full = torch.zeros(rb * BLOCK if two_d else rows, kb * BLOCK, dtype=torch.float64, device=v.device)
    full[:rows, :cols] = v
    t = full.view(rb, -1, kb, BLOCK)
    amax = t.abs().amax((1, 3))
    e = torch.ceil(torch.log2(amax / 448))
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e))
    scale = torch.where(amax == 0, torch.ones_like(amax), torch.exp2(e.clamp(-126, 127)))
    return _e4m3(t / scale[:, None, :, None]).view(-1, kb * BLOCK)[:rows], scale.t()


def _exact_held(q):
    codes, scales, rows, cols, two_d = q
    v = codes.view(torch.float8_e4m3fn).double()[:, :cols]
    s = torch.exp2(scales.double() - 127)
    i = torch.arange(rows, device=v.device) // (BLOCK if two_d else 1)
    j = torch.arange(cols, device=v.device) // BLOCK
    return v * s[:, i].t()[:, j]


def _exact_through(v):
    """v through its quantization along the last dimension."""
    codes, scale = _exact_quantize(v, False)
    return (codes * scale.t().repeat_interleave(BLOCK, 1))[:, :v.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    named = lambda q: {"codes": q[0], "scales": q[1]}  # noqa: E731
    if op == "norm":
        total = s["x"].double() + s["residual"].double()
        h = total.to(s["x"].dtype).double()  # the residual stream's own type
        rstd = 1 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
        y = torch.einsum("mc,m,c->mc", h, rstd, s["weight"].double())
        out = {"h": total, "y": named(_exact_quantize(y, False))}
        if case["train"]:
            out |= {"rstd": rstd, "y_t": named(_exact_quantize(y.t(), False))}
        return out
    if op == "norm_grad":
        h, r, w, dy = (s[n].double() for n in ("h", "rstd", "weight", "dy"))
        wdy = w * dy
        dot = (wdy * h).sum(1) * r ** 3 / h.shape[1]
        return {"dx": s["dh"].double() + wdy * r[:, None] - h * dot[:, None], "dweight": r @ (dy * h)}
    if op == "quantize":
        x = s["x"].double()
        return {"q": named(_exact_quantize(x, case["two_d"])), "q_t": named(_exact_quantize(x.t(), case["two_d"]))}
    if op == "gemm":
        return {"c": _exact_held(s["a"]).matmul(_exact_held(s["b"]).t().contiguous())}
    if op == "ffn":
        x = _exact_held(s["x"])
        g, u = (x.matmul(_exact_held(s[n]).t().contiguous()) for n in ("wg", "wu"))
        gr, ur = g.bfloat16().double(), u.bfloat16().double()  # the projections are held in bf16
        y = _exact_through(gr * torch.sigmoid(gr) * ur).matmul(_exact_held(s["wd"]).t().contiguous())
        return {"y": y, "g": g, "u": u} if case["train"] else {"y": y}
    dh = _exact_held(s["dy"]).matmul(_exact_held(s["wd_t"]).t().contiguous())
    g, u = s["g"].double(), s["u"].double()
    sig = torch.sigmoid(g)
    du = dh * g * sig
    dg = dh * u * (sig + g * sig * (1 - sig))
    x = _exact_held(s["x_t"]).t().contiguous()
    return {"dx": _exact_through(dg) @ _exact_held(s["wg_t"]).t().contiguous()
            + _exact_through(du) @ _exact_held(s["wu_t"]).t().contiguous(),
            "dwg": _exact_through(dg.t()) @ x, "dwu": _exact_through(du.t()) @ x,
            "dwd": _exact_held(s["dy_t"]) @ _exact_through((g * sig * u).t()).t().contiguous()}
