"""The routed-expert example: its gradients against autograd through the plain
formulas, and its run from training to serving."""
import importlib.util
import pathlib

import pytest
import torch
import torch.nn.functional as F

import mx9_dual_axis_amd as mxq
from helpers import require_gpu, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def example(request):
    require_gpu()
    say(request.node.name)
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "routed_experts.py"
    spec = importlib.util.spec_from_file_location("routed_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_layer(x, params, k, valid):
    """The layer in fp32 by dense products, weighted by the picks."""
    router, W1, W2 = params
    p = torch.softmax(x @ router.t(), 1)
    E = p.shape[1]
    top, idx = p.topk(k, dim=1)
    w = torch.zeros_like(p).scatter(1, idx, top / top.sum(1, keepdim=True)) * valid[:, None]
    live = valid.sum()
    counts = (torch.zeros_like(p).scatter(1, idx, 1.0) * valid[:, None]).sum(0)
    balance = E * (counts / (k * live) * (p * valid[:, None]).sum(0) / live).sum()
    y = torch.zeros_like(x)
    for e in range(E):
        gate, up = (x @ W1[e].t()).chunk(2, dim=1)
        y = y + w[:, e:e + 1] * ((F.silu(gate) * up) @ W2[e].t())
    return y, balance


def test_gradients_of_the_layer(example):
    """The picks are equal (routing is in fp32 on both sides).  An MXFP8 product
    moves its result by at most 2^-4 of its norm (an element's half step is
    2^-4 of it, and the errors of a contraction are not aligned); four of them
    follow one another at most, from the input to a gradient."""
    T, E, K, H, k = 300, 8, 256, 128, 2
    params = example.init(E, K, H, DEV, 5)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    x = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    dy = torch.randn((T, K), generator=g, device=DEV)
    valid = torch.rand(T, generator=g, device=DEV) < 0.9
    xa, xb = x.clone().requires_grad_(), x.float().requires_grad_()
    plan = mxq.mx_routing(T, E, k, align=128, device=DEV)
    y, balance = example.train_layer(xa, params, plan, valid)
    ((y.float() * dy).sum() + 3 * balance.sum()).backward()
    twin = [p.detach().clone().requires_grad_() for p in params]
    yy, bb = plain_layer(xb, twin, k, valid.float())
    ((yy * dy).sum() + 3 * bb).backward()
    rel = lambda a, b: float((a.detach().float() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    assert rel(y, yy) < 2 * 2.0 ** -4
    assert rel(balance, bb) < 1e-4
    for name, a, b in zip(("x", "router", "W1", "W2"), (xa, *params), (xb, *twin)):
        assert rel(a.grad, b.grad) < 4 * 2.0 ** -4, name
    assert not y[~valid].any()


def test_example_trains_and_serves(example):
    """Training halves the loss; int8 serving stays within its own and the
    MXFP8 products' distance (two products of 2^-4 each) of the layer."""
    losses, dist = example.main(steps=60)
    assert losses[-1] < 0.5 * losses[0]
    assert max(dist.values()) < 2 * 2.0 ** -4
