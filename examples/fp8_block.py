"""A pre-norm gated feed-forward block trained and then decoded with the library's 8-bit
operators: y = h + (silu(n Wg^T) * (n Wu^T)) Wd^T with h = x + r and n the norm of h.

python examples/fp8_block.py [--tokens T --width K --inner F --steps S --lr L]

Each step quantizes the master weights (tile scales, both layouts), runs the forward
pass, takes the gradient of a mean squared error against a fixed target block, runs the
backward pass and updates the weights by plain gradient descent.  Every buffer and
workspace is made once.  Decoding runs the trained block on single tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_bit_microscaled_amd as fp4  # noqa: E402

EPS = 1e-6


class Block:
    """Master weights in binary32, their quantized forms, and the buffers of one
    micro-batch of `tokens`."""

    def __init__(self, tokens, width, inner, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.M, self.K, self.F = tokens, width, inner
        self.norm = torch.ones(width, device="cuda")
        shapes = {"wg": (inner, width), "wu": (inner, width), "wd": (width, inner)}
        self.w = {n: torch.randn(*s, generator=gen, device="cuda") * s[1] ** -0.5 for n, s in shapes.items()}
        self.q = {n: fp4.Fp8Tensor(*s, two_d=True) for n, s in shapes.items()}
        self.q_t = {n: fp4.Fp8Tensor(s[1], s[0], two_d=True) for n, s in shapes.items()}
        self.grad = {n: torch.empty(*s, dtype=torch.bfloat16, device="cuda") for n, s in shapes.items()}
        self.dnorm = torch.empty(width, device="cuda")
        b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.h, self.y, self.dn, self.dx = (b16(tokens, width) for _ in range(4))
        self.g, self.u = b16(tokens, inner), b16(tokens, inner)
        self.rstd = torch.empty(tokens, device="cuda")
        self.n, self.n_t = fp4.Fp8Tensor(tokens, width), fp4.Fp8Tensor(width, tokens)
        self.hq = fp4.Fp8Tensor(tokens, inner)
        self.dy, self.dy_t = fp4.Fp8Tensor(tokens, width), fp4.Fp8Tensor(width, tokens)
        self.bufs = fp4.FfnBuffers(tokens, width, inner)
        self.ws = torch.empty(max(fp4.fp8_ffn_ws_bytes(tokens, width, inner), fp4.fp8_ffn_ws_bytes(1, width, inner),
                                  fp4.fp8_rms_norm_ws_bytes(tokens, width)), dtype=torch.uint8, device="cuda")
        self.quantize_weights()

    def quantize_weights(self):
        for n, w in self.w.items():
            fp4.fp8_quantize(w, self.q[n], self.q_t[n])

    def forward(self, x, residual):
        fp4.fp8_rms_norm(x, self.norm, EPS, self.n, residual=residual, h=self.h, yq_t=self.n_t, rstd=self.rstd)
        fp4.fp8_ffn_fprop(self.n, self.q["wg"], self.q["wu"], self.q["wd"], self.hq, self.y, g=self.g, u=self.u,
                          ws=self.ws)
        return self.h + self.y

    def backward(self, dout):
        """dout: the gradient of forward's result; returns that of x and of the residual."""
        fp4.fp8_quantize(dout, self.dy, self.dy_t)
        fp4.fp8_ffn_backward(self.dy, self.dy_t, self.n_t, self.q_t["wg"], self.q_t["wu"], self.q_t["wd"], self.g, self.u,
                             self.bufs, self.dn, self.grad["wg"], self.grad["wu"], self.grad["wd"], ws=self.ws)
        fp4.fp8_rms_norm_backward(self.dn, self.h, self.norm, self.rstd, self.dx, self.dnorm, self.ws, dh=dout)
        return self.dx

    def update(self, lr):
        for n, w in self.w.items():
            w.sub_(self.grad[n].float(), alpha=lr)
        self.norm.sub_(self.dnorm, alpha=lr)
        self.quantize_weights()

    def decode(self, x, residual):
        """One token, nothing kept for a backward pass."""
        h, y = torch.empty_like(x), torch.empty_like(x)
        n, hq = fp4.Fp8Tensor(1, self.K), fp4.Fp8Tensor(1, self.F)
        fp4.fp8_rms_norm(x, self.norm, EPS, n, residual=residual, h=h)
        fp4.fp8_ffn_fprop(n, self.q["wg"], self.q["wu"], self.q["wd"], hq, y, ws=self.ws)
        return h + y


def train(tokens=512, width=512, inner=1024, steps=30, lr=60.0, seed=1):
    """The losses of `steps` steps, the trained block and the last micro-batch."""
    block, target = Block(tokens, width, inner, seed), Block(tokens, width, inner, seed + 100)
    gen = torch.Generator(device="cuda").manual_seed(seed + 200)
    x, r = (torch.randn(tokens, width, generator=gen, device="cuda").bfloat16() for _ in range(2))
    want = target.forward(x, r).float()
    losses = []
    for _ in range(steps):
        diff = block.forward(x, r).float() - want
        losses.append(float(diff.square().mean()))
        block.backward((diff * (2.0 / diff.numel())).bfloat16())
        block.update(lr)
    return losses, block, (x, r)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, kind, value in (("tokens", int, 512), ("width", int, 512), ("inner", int, 1024), ("steps", int, 30),
                              ("lr", float, 60.0)):
        ap.add_argument(f"--{name}", type=kind, default=value)
    a = ap.parse_args()
    losses, block, (x, r) = train(a.tokens, a.width, a.inner, a.steps, a.lr)
    for i, v in enumerate(losses):
        print(f"step {i} loss {v:.5f}")
    full = block.forward(x, r)
    one = block.decode(x[:1].contiguous(), r[:1].contiguous())
    print(f"decoded token against the batch's: largest difference {float((one - full[:1]).abs().max()):.4f}")


if __name__ == "__main__":
    main()
