"""A mixture-of-experts feed-forward layer with MXFP4 experts: served, and its router trained.

    python examples/expert_layer.py            # needs the built library and a GPU

`ExpertLayer.forward` is the serving path: one call quantizes the tokens, runs the experts' gate and
up products with SwiGLU, their down products and the weighted sum. `ExpertLayer.train_router` keeps
the experts frozen and trains the router through the gradient of the weighted sum. `MixtureFunction`
shows the routing around experts of the user's own, with gradients for tokens, weights and the experts' parameters.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_gemm_quantize_amd import binding as b  # noqa: E402


def quantize_experts(weights):
    """[E,N,K] weights -> MXFP4 codes [E,N,K/2] and scales [E,ceil(K/256),N,8]."""
    parts = [b.mxfp4_quantize_rows(w) for w in weights]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


class ExpertLayer:
    def __init__(self, experts, top, hidden, ffn, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=g, device=device).mul_(scale).to(torch.bfloat16)

        self.top, self.experts = top, experts
        self.router = normal(experts, hidden, scale=hidden ** -0.5).float()
        gate = normal(experts, ffn, hidden, scale=hidden ** -0.5)
        up = normal(experts, ffn, hidden, scale=hidden ** -0.5)
        # rows 2f and 2f + 1 of an expert's first weight: gate and up of hidden unit f
        w13 = torch.stack((gate, up), dim=2).reshape(experts, 2 * ffn, hidden)
        self.w13 = quantize_experts(w13)
        self.w2 = quantize_experts(normal(experts, hidden, ffn, scale=ffn ** -0.5))

    def route(self, x):
        """Expert ids [T,top] and their softmax weights (differentiable in the router)."""
        top, ids = (x.float() @ self.router.t()).topk(self.top, dim=1)
        return ids, torch.softmax(top, dim=1)

    @torch.no_grad()
    def forward(self, x):
        ids, weights = self.route(x)
        return b.mxfp4_moe(x, ids, weights, *self.w13, *self.w2)

    def train_router(self, x, target, rate):
        """One step of gradient descent on the squared error per token, the experts frozen; the loss."""
        router = self.router.requires_grad_()
        ids, weights = self.route(x)
        with torch.no_grad():
            offsets, slot_pos, row_token = b.moe_sort(ids, self.experts)
            xq, xs = b.mxfp4_quantize_rows(x)
            hq, hs = b.mxfp4_expert_swiglu(xq, xs, offsets, *self.w13, row_token=row_token)
            rows = b.mxfp4_expert_gemm(hq, hs, offsets, *self.w2, out_dtype=x.dtype)
            error = b.moe_combine(rows, slot_pos, weights.contiguous()).float() - target.float()
            d_out = (error * (2.0 / len(x))).to(x.dtype)
            _, d_weights = b.moe_combine_backward(d_out, rows, slot_pos, weights.contiguous())
        weights.backward(d_weights)
        self.router = (router - rate * router.grad).detach()
        return error.square().sum(dim=1).mean().item()


class Gather(torch.autograd.Function):
    """Tokens [T,H] -> rows [T*top,H] in expert order, zeros for slots without an expert."""

    @staticmethod
    def forward(ctx, x, slot_pos):
        ctx.save_for_backward(slot_pos)
        return b.moe_gather(x, slot_pos)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_rows):
        slot_pos, = ctx.saved_tensors
        return b.moe_gather_backward(d_rows.contiguous(), slot_pos), None


class Combine(torch.autograd.Function):
    """Rows in expert order and the router's weights -> their weighted sums [T,H]."""

    @staticmethod
    def forward(ctx, rows, slot_pos, weights):
        rows, weights = rows.contiguous(), weights.contiguous()
        ctx.save_for_backward(rows, slot_pos, weights)
        return b.moe_combine(rows, slot_pos, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        rows, slot_pos, weights = ctx.saved_tensors
        d_rows, d_weights = b.moe_combine_backward(d_out.contiguous(), rows, slot_pos, weights)
        return d_rows, None, d_weights


class MixtureFunction:
    """tokens [T,H], expert ids and weights -> the weighted sum of experts' outputs, where
    `run_experts` maps rows in expert order and their offsets to rows of the same shape (those past
    the last offset have no expert and count for nothing). Gradients reach the tokens, the weights and,
    through `run_experts`, whatever parameters it uses."""

    @staticmethod
    def apply(x, ids, weights, experts, run_experts):
        offsets, slot_pos, _ = b.moe_sort(ids, experts)
        outputs = run_experts(Gather.apply(x, slot_pos), offsets)
        return Combine.apply(outputs, slot_pos, weights)


def main(tokens=256, experts=8, top=2, hidden=1024, ffn=512, steps=30, rate=0.001):
    """Losses of a router that learns to imitate another one over the same experts."""
    torch.manual_seed(0)
    layer, teacher = (ExpertLayer(experts, top, hidden, ffn, seed=1) for _ in range(2))
    teacher.router += 0.7 * hidden ** -0.5 * torch.randn_like(teacher.router)
    x = torch.randn((tokens, hidden), device="cuda:0").to(torch.bfloat16)
    target = teacher.forward(x)
    losses = [layer.train_router(x, target, rate) for _ in range(steps)]
    print("router's loss: %.5f -> %.5f in %d steps" % (losses[0], losses[-1], steps))
    token = layer.forward(x[:1])
    print("one token:", tuple(token.shape), token.dtype)
    return losses


if __name__ == "__main__":
    main()
