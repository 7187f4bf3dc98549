"""GPU tests of what a routing holds between a forward and its backward."""
import importlib.util
import pathlib

import pytest
import torch

import mx9_dual_axis_amd as mxq
from helpers import require_gpu, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu(request):
    require_gpu()
    say(request.node.name)


def load_example():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "routed_experts.py"
    spec = importlib.util.spec_from_file_location("routed_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def batches(n, T, K):
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    return [torch.randn((T, K), generator=g, device=DEV).bfloat16() for _ in range(n)]


def test_two_forwards_on_one_routing_before_a_backward():
    """The second forward writes the first one's picks over: the first one's
    backward is refused, the second one's is right."""
    ex = load_example()
    T, E, K, H, k = 200, 8, 256, 128, 2
    params = ex.init(E, K, H, DEV, 5)
    xa, xb = batches(2, T, K)
    plan = mxq.mx_routing(T, E, k, align=128, device=DEV)
    ya, ba = ex.train_layer(xa, params, plan)
    yb, bb = ex.train_layer(xb, params, plan)
    with pytest.raises(ValueError, match="written"):
        (ya.float().sum() + ba.sum()).backward()
    for p in params:
        p.grad = None
    (yb.float().sum() + bb.sum()).backward()
    got = [p.grad.clone() for p in params]
    for p in params:
        p.grad = None
    y, b = ex.train_layer(xb, params, mxq.mx_routing(T, E, k, align=128, device=DEV))
    (y.float().sum() + b.sum()).backward()
    for p, d in zip(params, got):
        assert torch.equal(p.grad, d)


def test_every_step_of_the_layer_refuses_a_routing_written_since():
    """Each autograd function by itself: the router's gradient, the rows', the
    experts' and the weights'."""
    ex = load_example()
    T, E, K, k = 130, 4, 128, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    logits = torch.randn((T, E), generator=g, device=DEV, requires_grad=True)
    x = torch.randn((T, K), generator=g, device=DEV).bfloat16().requires_grad_()
    W = torch.randn((E, 128, K), generator=g, device=DEV).bfloat16().requires_grad_()
    plan = mxq.mx_routing(T, E, k, align=128, device=DEV)
    weight, loss = ex.Route.apply(logits, plan, None)
    rows = ex.Dispatch.apply(x, plan)
    leaf = rows.detach().requires_grad_()
    h = ex.Experts.apply(leaf, W, plan)
    back = h.detach().requires_grad_()
    y = ex.Combine.apply(back, weight.detach().requires_grad_(), plan)
    mxq.mx_route(logits.detach() + 1, out=plan)
    for out in (weight, rows, h, y):
        with pytest.raises(ValueError, match="written"):
            out.sum().backward()
    assert logits.grad is None and x.grad is None and W.grad is None and back.grad is None


def test_two_forwards_on_two_routings():
    """Micro-batches whose losses meet in one backward: the sum of their own
    gradients, each formed by itself (fp32 sums of two terms: half an ulp)."""
    ex = load_example()
    T, E, K, H, k = 200, 8, 256, 128, 2
    params = ex.init(E, K, H, DEV, 5)
    parts = batches(2, T, K)
    plans = [mxq.mx_routing(T, E, k, align=128, device=DEV) for _ in parts]
    each = []
    for x, plan in zip(parts, plans):
        y, b = ex.train_layer(x, params, plan)
        (y.float().sum() + b.sum()).backward()
        each.append([p.grad.clone() for p in params])
        for p in params:
            p.grad = None
    sums = [ex.train_layer(x, params, plan) for x, plan in zip(parts, plans)]
    sum(y.float().sum() + b.sum() for y, b in sums).backward()
    for p, a, b in zip(params, *each):
        assert ((p.grad - (a + b)).abs() <= 2.0 ** -23 * (a.abs() + b.abs())).all()


def test_gradient_names_the_generation_it_is_of():
    T, E, k = 70, 16, 3
    z = torch.randn((T, E), device=DEV)
    plan = mxq.mx_routing(T, E, k, align=1, device=DEV)
    assert plan.generation == 0
    first = mxq.mx_route(z, out=plan).generation
    dw = torch.ones((T, k), device=DEV)
    want = mxq.mx_route_grad(z, plan, dw)
    assert first == 1 and torch.equal(mxq.mx_route_grad(z, plan, dw, generation=first), want)
    mxq.mx_route(z + 1, out=plan)
    with pytest.raises(ValueError, match="written"):
        mxq.mx_route_grad(z, plan, dw, generation=first)
    assert mxq.mx_route_grad(z, plan, dw, generation=plan.generation).shape == (T, E)
    with pytest.raises(ValueError):
        mxq.mx_route(z[:, :5], out=plan)                  # refused: nothing was written
    assert plan.generation == 2


# ---- tokens left out
@pytest.mark.parametrize("filler", [float("nan"), 0.0])
def test_gradient_without_the_mask_of_its_routing(filler):
    """Tokens that the routing left out have no gradient: a call that does not
    say which they are is refused."""
    T, E, k = 90, 16, 3
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    z = torch.randn((T, E), generator=g, device=DEV)
    valid = torch.rand(T, generator=g, device=DEV) < 0.7
    z[~valid] = filler
    dl = torch.ones(1, device=DEV)
    r = mxq.mx_route(z, k, valid=valid)
    d = mxq.mx_route_grad(z, r, dloss=dl, valid=valid)
    assert not d[~valid].any() and d[valid].any()
    with pytest.raises(ValueError, match="valid"):
        mxq.mx_route_grad(z, r, dloss=dl)
    z[~valid] = 0
    mxq.mx_route(z, k, out=r)                             # the next routing takes every token
    assert mxq.mx_route_grad(z, r, dloss=dl).isfinite().all()
    # a gradient of fewer tokens than were routed: that of the others is 0
    d = mxq.mx_route_grad(z, r, dloss=dl, valid=valid)
    assert not d[~valid].any() and torch.equal(d[valid], mxq.mx_route_grad(z, r, dloss=dl)[valid])
