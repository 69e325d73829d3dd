"""A frozen 8-bit projection behind a norm, fine-tuned through low-rank adapters and then
served: y = n W^T + s_i (dropout(n) a_i^T) b_i^T with n the norm of h = r + dropout(x).

python examples/lora_block.py [--tokens T --width K --out N --rank R --adapters C --steps S --lr L]

Each micro-batch holds sequences of several tenants, each with an adapter of its own.  A step
quantizes the gradient of a mean squared error against fixed targets, runs the backward pass
and updates the adapters by plain gradient descent; the weight is quantized once.  The masks
of both dropouts come from a counter on the device that each step advances.  Serving runs
single tokens of all tenants in one call, with no dropout.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_bit_microscaled_amd as fp4  # noqa: E402

EPS = 1e-6


class Layer:
    """The frozen weight in both layouts, master adapters in binary32 beside the ones that the
    calls read, and the buffers of one micro-batch of `tokens`."""

    def __init__(self, tokens, width, out, rank=8, adapters=2, p=0.1, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.M, self.K, self.N = tokens, width, out
        w = rnd(out, width) * width ** -0.5
        self.w, self.w_t = fp4.Fp8Tensor(out, width, True), fp4.Fp8Tensor(width, out, True)
        fp4.fp8_quantize(w, self.w, self.w_t)
        self.norm = torch.ones(width, device="cuda")
        self.lora = fp4.LoraAdapters(adapters, rank, out, width)
        self.a, self.b = rnd(*self.lora.a.shape) * width ** -0.5, torch.zeros(self.lora.b.shape, device="cuda")
        self.da, self.db = torch.empty_like(self.a), torch.empty_like(self.b)
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")
        # offsets further apart than the steps of a run: their sum with the step is one number
        self.drop_x, self.drop_n = (fp4.Dropout(p, 1000 + seed, layer << 40, self.step) if p else None for layer in (1, 2))
        b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.h, self.y = b16(tokens, width), b16(tokens, out)
        self.dn, self.dx, self.dr = (b16(tokens, width) for _ in range(3))
        self.rstd, self.dnorm = torch.empty(tokens, device="cuda"), torch.empty(width, device="cuda")
        self.n, self.dy = fp4.Fp8Tensor(tokens, width), fp4.Fp8Tensor(tokens, out)
        need = max(fp4.fp8_lora_fprop_ws_bytes(tokens, out, width, rank), fp4.fp8_rms_norm_ws_bytes(tokens, width),
                   fp4.fp8_lora_backward_ws_bytes(tokens, out, width, rank, adapters))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.store()

    def store(self):
        self.lora.a.copy_(self.a)
        self.lora.b.copy_(self.b)

    def forward(self, x, residual, index):
        if self.drop_x:
            fp4.fp8_dropout_rms_norm(x, self.drop_x, self.norm, EPS, self.n, residual, self.h, rstd=self.rstd)
        else:
            fp4.fp8_rms_norm(x, self.norm, EPS, self.n, residual=residual, h=self.h, rstd=self.rstd)
        fp4.fp8_lora_fprop(self.n, self.w, self.lora, self.y, index=index, drop=self.drop_n, ws=self.ws)
        return self.y

    def backward(self, dy, index):
        """dy: the gradient of forward's result; returns those of x and of the residual."""
        fp4.fp8_quantize(dy, self.dy)
        fp4.fp8_lora_backward(self.dy, self.w_t, self.n, self.lora, self.dn, self.da, self.db, self.ws, index=index,
                              drop=self.drop_n)
        if not self.drop_x:
            fp4.fp8_rms_norm_backward(self.dn, self.h, self.norm, self.rstd, self.dx, self.dnorm, self.ws)
            return self.dx, self.dx
        fp4.fp8_dropout_rms_norm_backward(self.dn, self.h, self.norm, self.rstd, self.drop_x, self.dx, self.dr,
                                          self.dnorm, self.ws)
        return self.dx, self.dr

    def update(self, lr):
        self.a.sub_(self.da, alpha=lr)
        self.b.sub_(self.db, alpha=lr)
        self.store()
        self.step.add_(1)

    def serve(self, x, residual, index):
        """Tokens of several requests, each with its adapter, nothing kept."""
        h, n = torch.empty_like(x), fp4.Fp8Tensor(*x.shape)
        y = torch.empty(x.shape[0], self.N, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(16, fp4.fp8_lora_fprop_ws_bytes(x.shape[0], self.N, self.K, self.lora.rank, mixed=True)),
                         dtype=torch.uint8, device="cuda")
        fp4.fp8_rms_norm(x, self.norm, EPS, n, residual=residual, h=h)
        fp4.fp8_lora_fprop(n, self.w, self.lora, y, index=index, ws=ws, mixed=True)
        return y


def train(tokens=256, width=512, out=384, rank=8, adapters=2, steps=20, lr=20.0, p=0.1, seed=1):
    """The losses of `steps` steps, the layer and the micro-batch."""
    layer, gen = Layer(tokens, width, out, rank, adapters, p, seed), torch.Generator(device="cuda").manual_seed(seed + 7)
    x, r = (torch.randn(tokens, width, generator=gen, device="cuda").bfloat16() for _ in range(2))
    index = (torch.arange(tokens, device="cuda") * adapters // tokens).int()
    # what a few directions of each tenant's own would add
    base = layer.serve(x, r, index).float()
    u = torch.randn(adapters, tokens, 2, generator=gen, device="cuda")
    v = torch.randn(adapters, 2, out, generator=gen, device="cuda") * 0.3
    want = base + torch.stack([u[int(i), t] @ v[int(i)] for t, i in enumerate(index.tolist())])
    losses = []
    for _ in range(steps):
        diff = layer.forward(x, r, index).float() - want
        losses.append(float(diff.square().mean()))
        layer.backward((diff * (2.0 / diff.numel())).bfloat16(), index)
        layer.update(lr)
    return losses, layer, (x, r, index, want)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, kind, value in (("tokens", int, 256), ("width", int, 512), ("out", int, 384), ("rank", int, 8),
                              ("adapters", int, 2), ("steps", int, 20), ("lr", float, 20.0), ("p", float, 0.1)):
        ap.add_argument(f"--{name}", type=kind, default=value)
    a = ap.parse_args()
    losses, layer, (x, r, index, _) = train(**vars(a))
    for i, v in enumerate(losses):
        print(f"step {i} loss {v:.5f}")
    one = layer.serve(x[:1], r[:1], index[:1])
    print(f"a served token's first results: {[round(float(v), 3) for v in one[0, :4]]}")


if __name__ == "__main__":
    main()
