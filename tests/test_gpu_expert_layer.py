"""The expert layer's example: serving, the router's training, and gradients around own experts."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_example_runs_and_learns():
    import expert_layer
    losses = expert_layer.main(tokens=128, experts=4, top=2, hidden=256, ffn=128, steps=20)
    assert losses[-1] < losses[0]


def test_gradients_around_own_experts():
    """Tokens' and weights' gradients through MixtureFunction equal autograd's through the same
    mixture written out, up to the roundings of fp32 sums."""
    import expert_layer
    T, E, top, H = 24, 3, 2, 40
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn((T, H), generator=g, device=DEV)
    ids = torch.rand((T, E), generator=g, device=DEV).topk(top, dim=1).indices
    w = torch.rand((T, top), generator=g, device=DEV)
    mats = torch.randn((E, H, H), generator=g, device=DEV) * H ** -0.5
    d = torch.randn((T, H), generator=g, device=DEV)

    def run_experts(rows, offsets):
        bounds = offsets.tolist()
        return torch.cat([torch.tanh(rows[bounds[e]:bounds[e + 1]] @ mats[e]) for e in range(E)])

    x1, w1 = x.clone().requires_grad_(), w.clone().requires_grad_()
    expert_layer.MixtureFunction.apply(x1, ids, w1, E, run_experts).backward(d)
    x2, w2 = x.double().requires_grad_(), w.double().requires_grad_()
    every = torch.tanh(torch.stack([x2 @ mats[e].double() for e in range(E)], dim=1))      # [T, E, H]
    out = (every.gather(1, ids.unsqueeze(2).expand(T, top, H)) * w2.unsqueeze(2)).sum(dim=1)
    out.backward(d.double())
    # sums of at most 2 H terms of order 1 in fp32, through one tanh
    assert torch.allclose(x1.grad.double(), x2.grad, rtol=0, atol=2 * H * 2.0 ** -20)
    assert torch.allclose(w1.grad.double(), w2.grad, rtol=0, atol=2 * H * 2.0 ** -20)
