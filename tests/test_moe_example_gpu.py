"""examples/moe_layer_mxfp4.py: the routed layer against the same layer written
with torch on the decoded weights, and its gradients against autograd.

Two choices of the layer round beyond the weights: activations to MXFP4 before
each product (their decoded values go into the reference) and bf16 between the
steps.  What is left between the two sides are bf16 roundings of d, h and y
(2^-9 each), and where an element of h falls on the other side of a code's
rounding boundary because d differed in its last bit: a relative error of the
whole output well below 1%."""
import os
import sys

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv
from helpers import host_bits
from oracle import mxfp4_oracle as mo

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def decoded(x):
    """What the product sees of bf16 rows, fp64."""
    return torch.from_numpy(mo.dequantize(*mo.quantize(host_bits(x)))).cuda()


@pytest.mark.parametrize("tokens", [1, 9, 150])
def test_layer_against_torch(tokens):
    from moe_layer_mxfp4 import MoELayer
    K, H, E, k = 256, 256, 16, 4
    layer = MoELayer(K, H, E, k, groups=4, topk_groups=2, seed=tokens)
    gen = torch.Generator("cuda").manual_seed(tokens)
    x = torch.randn(tokens, K, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_(True)
    y, weights = layer(x)
    ids = nv.nvfp4_route_topk((x.float() @ layer.router.t()).detach(), k, **layer.form)["expert_ids"].long()

    def w(packed, rows, cols):
        return nv.nvfp4_mxfp4_dequantize(packed["codes"], packed["sf"]).double().reshape(E, rows, cols)

    up, down = w(layer.up, 2 * H, K), w(layer.down, K, H)
    shared = nv.nvfp4_mxfp4_dequantize(layer.shared["codes"], layer.shared["sf"]).double()
    xd = decoded(x.detach())
    want = torch.zeros(tokens, K, dtype=torch.float64, device="cuda")
    for t in range(tokens):
        for j in range(k):
            e = int(ids[t, j])
            d = (up[e] @ xd[t]).to(torch.bfloat16).float()
            h = (torch.nn.functional.silu(d[:H]) * d[H:]).to(torch.bfloat16)
            want[t] += float(weights[t, j].detach()) * (down[e] @ decoded(h[None])[0])
    want += xd @ shared.t()
    err = (y.double() - want).norm() / want.norm()
    assert float(err) < 1e-2, float(err)

    # gradients: the router's through the weights, x's through the shared linear
    c = torch.randn(tokens, k, generator=gen, device="cuda")
    ((weights * c).sum() + y.float().sum()).backward()
    logits = (x.detach().double() @ layer.router.detach().double().t()).requires_grad_(True)
    s = torch.sigmoid(logits).gather(1, ids)
    (s / s.sum(1, keepdim=True) * 2.5 * c.double()).sum().backward()
    want_router = logits.grad.t() @ x.detach().double()
    assert torch.allclose(layer.router.grad.double(), want_router, rtol=1e-4, atol=1e-4 * float(want_router.abs().max()))
    want_x = torch.ones(tokens, K, dtype=torch.float64, device="cuda") @ shared \
        + logits.grad @ layer.router.detach().double()
    assert float((x.grad.double() - want_x).norm() / want_x.norm()) < 1e-2


def test_example_runs():
    import moe_layer_mxfp4
    moe_layer_mxfp4.main()


@pytest.mark.parametrize("tokens", [1, 9, 150])
def test_training_loss_has_its_whole_gradient(tokens):
    """Everything that the example's loss depends on reaches x and the router: its
    gradients against autograd in 64 bits on the decoded weights, the choice held
    fixed.  The shared linear sees x rounded to MXFP4 with the rounding passed
    straight through; left are bf16 roundings of its output and of its gradient."""
    from moe_layer_mxfp4 import MoELayer, training_loss
    K, E, k = 256, 16, 4
    layer = MoELayer(K, 256, E, k, groups=4, topk_groups=2, seed=tokens + 1)
    gen = torch.Generator("cuda").manual_seed(tokens)
    x = torch.randn(tokens, K, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_(True)
    y, weights = layer(x)
    assert not layer.experts(x, *layer.route(x)).requires_grad
    training_loss(layer, x).backward()
    ids = layer.route(x.detach())[0].long()

    shared = nv.nvfp4_mxfp4_dequantize(layer.shared["codes"], layer.shared["sf"]).double()
    xr = x.detach().double().requires_grad_(True)
    router = layer.router.detach().double().requires_grad_(True)
    s = torch.sigmoid(xr @ router.t()).gather(1, ids)
    w = layer.form["scale"] * s / s.sum(1, keepdim=True)
    seen = xr + (decoded(x.detach()) - xr).detach()
    ((seen @ shared.t()).square().mean() + w.square().sum(1).mean()).backward()
    assert float((x.grad.double() - xr.grad).norm() / xr.grad.norm()) < 1e-2
    assert float((layer.router.grad.double() - router.grad).norm() / router.grad.norm()) < 1e-2
