"""Gradients of experts of the user's own inside the mixture of the expert layer's example."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("tokens_too", [False, True])
def test_parameters_of_own_experts_get_gradients(tokens_too):
    """Every parameter that run_experts uses gets autograd's gradient of the same mixture written out in
    64 bits (sums of at most T * H terms of order 1 in fp32, through one tanh), with tokens that take
    part in the gradient or do not, and slots without an expert."""
    import expert_layer
    T, E, top, H = 24, 3, 2, 40
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn((T, H), generator=g, device=DEV)
    ids = torch.rand((T, E), generator=g, device=DEV).topk(top, dim=1).indices
    ids[::5, 1] = -1
    w = torch.rand((T, top), generator=g, device=DEV)
    mats = torch.randn((E, H, H), generator=g, device=DEV) * H ** -0.5
    bias = torch.randn((E, H), generator=g, device=DEV)
    d = torch.randn((T, H), generator=g, device=DEV)
    x1, w1, m1, b1 = x.clone().requires_grad_(tokens_too), *[t.clone().requires_grad_() for t in (w, mats, bias)]

    def run_experts(rows, offsets):
        bounds = offsets.tolist()
        parts = [torch.tanh(rows[bounds[e]:bounds[e + 1]] @ m1[e] + b1[e]) for e in range(E)]
        return torch.cat(parts + [rows[bounds[E]:]])

    expert_layer.MixtureFunction.apply(x1, ids, w1, E, run_experts).backward(d)
    x2, w2, m2, b2 = [t.double().requires_grad_() for t in (x, w, mats, bias)]
    every = torch.tanh(torch.stack([x2 @ m2[e] + b2[e] for e in range(E)], dim=1))         # [T, E, H]
    picked = every.gather(1, ids.clamp_min(0).unsqueeze(2).expand(T, top, H)) * (ids >= 0).unsqueeze(2)
    (picked * w2.unsqueeze(2)).sum(dim=1).backward(d.double())
    pairs = [(w1, w2), (m1, m2), (b1, b2)] + ([(x1, x2)] if tokens_too else [])
    for got, want in pairs:
        assert got.grad is not None
        assert torch.allclose(got.grad.double(), want.grad, rtol=0, atol=T * H * 2.0 ** -20)
    assert tokens_too or x1.grad is None
