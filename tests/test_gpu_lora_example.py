"""GPU: the norm behind a dropped-out branch, the projection with adapters and both gradients
together, as examples/lora_block.py runs them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference(layer, a, b, x, r, index, masks):
    """y in binary64 of the layer's own 8-bit n and W and the given adapters."""
    import fp8_ref as ref
    n, w = ref.values(layer.n).cuda(), ref.values(layer.w).cuda()
    y = n @ w.t().contiguous()
    for i in range(a.shape[0]):
        rows = (index == i).nonzero()[:, 0]
        y[rows] += (n[rows] * masks[rows]) @ a[i][:, :layer.K].t().contiguous() @ b[i].t().contiguous()
    return y


@pytest.mark.parametrize("tokens,p", [(256, 0.1), (40, 0.25), (256, 0.0)])
def test_the_chain_and_its_gradients(fp4, tokens, p):
    """A step's da and db are the differences of sum(y dy) along random directions: y is
    linear in a and in b, dy is the gradient as the calls hold it, in 8 bits, and n and W are
    the layer's own.  The sums are within 2.1e-5 of their terms' magnitudes each (the bound
    of lora_ref.py), of which the difference's own binary64 rounding is no part."""
    import drop_ref
    import fp8_ref as ref
    import lora_block
    losses, layer, (x, r, index, want) = lora_block.train(tokens=tokens, width=200, out=136, steps=3, p=p, seed=3)
    assert all(v == v for v in losses)
    k = int(layer.step.item())
    y = layer.forward(x, r, index).clone()
    masks = torch.ones(tokens, 200, dtype=torch.float64, device="cuda")
    if p:
        masks = drop_ref.keep(tokens, 200, p, 1003, 2 << 40, k).cuda().double() * drop_ref.gain(p)
    a, b = layer.lora.a.double(), layer.lora.b.double()
    full = reference(layer, a, b, x, r, index, masks)
    # bf16 y: half a step, and the binary32 sums
    assert ((y.double() - full).abs() <= 2.0 ** -8 * full.abs() + 1e-3).all()
    dx, dr = layer.backward((y.float() - want).bfloat16() * 0.01, index)
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dr.float()).all()
    dy = ref.values(layer.dy).cuda()
    gen = torch.Generator(device="cuda").manual_seed(5)
    for which, grad, at in ((0, layer.da.double(), a), (1, layer.db.double(), b)):
        v = torch.randn(at.shape, generator=gen, device="cuda", dtype=torch.float64)
        hi, lo = [a, b], [a, b]
        hi[which], lo[which] = at + v, at - v
        diff = ((reference(layer, *hi, x, r, index, masks) - reference(layer, *lo, x, r, index, masks)) * dy).sum() / 2
        terms = ((reference(layer, *[t.abs() for t in hi], x, r, index, masks).abs() + full.abs()) * dy.abs()).sum()
        assert abs(float(diff - (grad * v).sum())) <= 2.1e-5 * float(terms), which


def test_residuals_gradient_passes_the_dropout(fp4):
    """dx is dropout of dresidual, by the mask of the forward pass at the same step."""
    import drop_ref
    import lora_block
    _, layer, (x, r, index, want) = lora_block.train(tokens=64, width=200, out=136, steps=2, p=0.3, seed=4)
    y = layer.forward(x, r, index)
    dx, dr = layer.backward((y.float() - want).bfloat16(), index)
    mask = drop_ref.keep(64, 200, 0.3, 1004, 1 << 40, int(layer.step.item())).cuda()
    assert (dx[~mask] == 0).all()
    got, ref = dx[mask].float(), dr[mask].float() * drop_ref.gain(0.3)
    assert ((got - ref).abs() <= 2.02 * 2.0 ** -8 * ref.abs()).all()
    kept = drop_ref.keep(64, 200, 0.3, 1004, 1 << 40, int(layer.step.item()))
    assert torch.equal(layer.h.cpu(), (r.cpu().float() + drop_ref.dropout(x.cpu(), 0.3, kept)).bfloat16())


def test_served_tokens_do_not_depend_on_their_batch(fp4):
    """A token's result alone, among a few and among many is the same within two roundings."""
    import lora_block
    _, layer, (x, r, index, _) = lora_block.train(tokens=256, width=200, out=136, steps=2, p=0.1, seed=5)
    many = layer.serve(x, r, index).float()
    few = layer.serve(x[100:120], r[100:120], index[100:120].contiguous()).float()
    one = layer.serve(x[110:111], r[110:111], index[110:111].contiguous()).float()
    tol = 2.0 ** -7 * many[100:120].abs() + 1e-4
    assert ((few - many[100:120]).abs() <= tol).all() and ((one - many[110:111]).abs() <= tol[10:11]).all()
