"""A routed expert layer on MXFP4 experts, with the gradients of its router and of
its shared linear.

    x [T, K] -> router logits -> nvfp4_route_topk -> nvfp4_mxfp4_grouped_gemm
      (gate | up projections of the chosen experts) -> SiLU(gate) * up
      -> nvfp4_mxfp4_moe_down_combine -> y [T, K]

plus a shared MXFP4 linear beside the experts with its input gradient.  The
routed products have no gradient: neither the one of x through the experts nor
the one of the routing weights through the weighted sum, so the routed output
is a constant to autograd and belongs into no loss that should train the router
or what makes x.  Run it on a GB300 after building the library:
python examples/moe_layer_mxfp4.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_block_scaled_06_gb300 as nv  # noqa: E402


class RouteTopk(torch.autograd.Function):
    """nvfp4_route_topk as an autograd function of the logits: (expert_ids, weights)."""

    @staticmethod
    def forward(ctx, logits, top_k, form):
        r = nv.nvfp4_route_topk(logits, top_k, **form)
        ctx.save_for_backward(logits, r["expert_ids"])
        ctx.form = {n: form[n] for n in ("score", "renormalize", "scale") if n in form}
        ctx.mark_non_differentiable(r["expert_ids"])
        return r["expert_ids"], r["weights"]

    @staticmethod
    def backward(ctx, _, grad_weights):
        logits, ids = ctx.saved_tensors
        return nv.nvfp4_route_topk_backward(logits, ids, grad_weights.float().contiguous(), **ctx.form), None, None


class MXLinear(torch.autograd.Function):
    """A frozen MXFP4 linear: the product forward, nvfp4_mxfp4_dgrad backward."""

    @staticmethod
    def forward(ctx, x, codes, sf):
        ctx.save_for_backward(codes, sf)
        ctx.shape = (codes.shape[0], 2 * codes.shape[1])
        return nv.nvfp4_mxfp4_gemm(codes, sf, *ctx.shape, a_bf16=x)

    @staticmethod
    def backward(ctx, dy):
        codes, sf = ctx.saved_tensors
        return nv.nvfp4_mxfp4_dgrad(dy.contiguous(), codes, sf, *ctx.shape), None, None


class MoELayer:
    """E experts of hidden size H on model width K, top_k per token."""

    def __init__(self, K, H, E, top_k, groups=1, topk_groups=1, device="cuda", seed=0):
        gen = torch.Generator(device).manual_seed(seed)

        def weights(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * 0.02).to(torch.bfloat16)

        self.K, self.H, self.E, self.top_k = K, H, E, top_k
        self.router = weights(E, K).float().requires_grad_(True)
        self.bias = torch.zeros(E, device=device)          # the balancing bias, updated outside the gradient
        self.form = dict(bias=self.bias, score="sigmoid", num_groups=groups, topk_groups=topk_groups,
                         renormalize=True, scale=2.5)
        # the experts' matrices stacked over their rows: gate | up [E * 2H, K] and down [E * K, H]
        self.up = nv.nvfp4_mxfp4_quantize(weights(E * 2 * H, K))
        self.down = nv.nvfp4_mxfp4_quantize(weights(E * K, H))
        self.shared = nv.nvfp4_mxfp4_quantize(weights(K, K))

    def route(self, x):
        return RouteTopk.apply(x.float() @ self.router.t(), self.top_k, self.form)

    @torch.no_grad()
    def experts(self, x, ids, weights):
        """The routed experts' output, without a gradient (see above)."""
        d, perm, offsets = nv.nvfp4_mxfp4_grouped_gemm(ids, x, self.up["codes"], self.up["sf"], 2 * self.H, self.K,
                                                       self.E)
        gate, up = d[:, :self.H].float(), d[:, self.H:].float()
        h = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
        return nv.nvfp4_mxfp4_moe_down_combine(h, perm, offsets, weights.contiguous(), self.down["codes"],
                                               self.down["sf"], self.K, self.H, self.E)

    def shared_linear(self, x):
        return MXLinear.apply(x, self.shared["codes"], self.shared["sf"])

    def __call__(self, x):
        """(y, routing weights).  The gradient of y is the shared linear's alone;
        the weights carry the router's."""
        ids, weights = self.route(x)
        return self.experts(x, ids, weights) + self.shared_linear(x), weights


def training_loss(layer, x):
    """A loss of the parts whose gradients are whole: the shared linear's output
    and the routing weights."""
    _, weights = layer.route(x)
    return layer.shared_linear(x).float().square().mean() + weights.square().sum(1).mean()


def main():
    torch.manual_seed(0)
    layer = MoELayer(K=1024, H=512, E=32, top_k=4, groups=4, topk_groups=2)
    for tokens in (1, 8, 500):                   # one decoded token, a small batch, a prompt
        x = torch.randn(tokens, layer.K, device="cuda").to(torch.bfloat16).requires_grad_(True)
        with torch.no_grad():
            y, _ = layer(x)
        layer.router.grad = None
        training_loss(layer, x).backward()
        print(f"{tokens:4d} tokens: y {tuple(y.shape)} rms {y.float().square().mean().sqrt():.4f}, "
              f"|dx| {x.grad.float().norm():.3e}, |d router| {layer.router.grad.norm():.3e}")


if __name__ == "__main__":
    main()
