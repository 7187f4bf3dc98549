"""The operators of a layer with scored routing and gated experts, run together:
in the routed-expert example's training and serving, and in a graph with the
bias's step."""
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


def plain_layer(x, params, bias, idx, valid):
    """The layer in fp32 by dense products, for the picks idx."""
    router, W1, W2 = params
    s = torch.sigmoid(x @ router.t())
    E, k = s.shape[1], idx.shape[1]
    picked = s.gather(1, idx)
    w = torch.zeros_like(s).scatter(1, idx, picked / (picked.sum(1, keepdim=True) + 1e-20)) * valid[:, None]
    live = valid.sum()
    counts = (torch.zeros_like(s).scatter(1, idx, 1.0) * valid[:, None]).sum(0)
    p = s / (s.sum(1, keepdim=True) + 1e-20) * valid[:, None]
    balance = E * (counts / (k * live) * p.sum(0) / live).sum()
    y = torch.zeros_like(x)
    for e in range(E):
        gate, up = (x @ W1[e].t()).chunk(2, dim=1)
        y = y + w[:, e:e + 1] * ((F.silu(gate) * up) @ W2[e].t())
    return y, balance


def picks(logits, bias, k, groups, top_groups):
    """The formula's picks in binary64."""
    s = torch.sigmoid(logits.double())
    u = s + bias.double()
    T, E = u.shape
    worth = u.view(T, groups, -1).topk(2, dim=2).values.sum(2)
    keep = torch.zeros_like(worth).scatter(1, worth.topk(top_groups, dim=1).indices, 1.0).bool()
    return u.masked_fill(~keep.repeat_interleave(E // groups, 1), float("-inf")).topk(k, dim=1).indices


def test_gradients_of_the_scored_layer(example):
    """The picks are the formula's for the logits that the layer forms.  An MXFP8
    product moves its result by at most 2^-4 of its norm (an element's half step
    is 2^-4 of it, and the errors of a contraction are not aligned); four of
    them follow one another at most, from the input to a gradient."""
    T, E, K, H, k = 300, 8, 256, 128, 2
    params = example.init(E, K, H, DEV, 5)
    g = torch.Generator(device=DEV)
    g.manual_seed(16)
    x = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    dy = torch.randn((T, K), generator=g, device=DEV)
    valid = torch.rand(T, generator=g, device=DEV) < 0.9
    bias = 0.2 * torch.randn(E, generator=g, device=DEV)
    xa, xb = x.clone().requires_grad_(), x.float().requires_grad_()
    plan = mxq.mx_routing(T, E, k, align=128, device=DEV)
    y, balance = example.train_layer(xa, params, plan, valid, bias)
    idx = plan.idx.long()
    with torch.no_grad():
        want = picks(x.float() @ params[0].t(), bias, k, example.SCORED["groups"], example.SCORED["top_groups"])
    assert torch.equal(idx[valid], want[valid]) and (idx[~valid] == -1).all()
    ((y.float() * dy).sum() + 3 * balance.sum()).backward()
    twin = [p.detach().clone().requires_grad_() for p in params]
    yy, bb = plain_layer(xb, twin, bias, want, valid.float())
    ((yy * dy).sum() + 3 * bb).backward()
    rel = lambda a, b: float((a.detach().float() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    assert rel(y, yy) < 2 * 2.0 ** -4
    assert rel(balance, bb) < 1e-4
    for name, a, b in zip(("x", "router", "W1", "W2"), (xa, *params), (xb, *twin)):
        assert rel(a.grad, b.grad) < 4 * 2.0 ** -4, name
    assert not y[~valid].any()


def test_the_example_by_scores_runs(example):
    losses, dist = example.main(steps=4, scored=True)
    assert len(losses) == 4 and all(torch.isfinite(torch.tensor(v)) for v in (*losses, *dist.values()))


@pytest.mark.parametrize("T", [1, 67])
def test_serving_in_a_graph_is_the_eager_step(example, T):
    """Captured and replayed with work between the replays: the bits of the
    same calls one by one."""
    E, K, H, k = 16, 256, 96, 3
    params = [p.detach() for p in example.init(E, K, H, DEV, 8)]
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    serve = example.Server(params, T, k, DEV, bias)
    for _ in range(4):
        x = torch.randn((T, K), generator=g, device=DEV).bfloat16()
        got = serve(x).clone()
        torch.cuda.synchronize()
        other = mxq.mx_route_scored(x.float() @ params[0].t(), k, bias, align=1, **example.SCORED)
        q, s = mxq.mx_dispatch_i8(x, other.slot, other.src)
        h = mxq.i8_grouped_gemm_rows_act(q, s, serve.W1, serve.s1, other.offs, act="silu", gated=True)
        q, s = mxq.i8_quantize_rows(h)
        y = mxq.mx_combine(mxq.i8_grouped_gemm_rows(q, s, serve.W2, serve.s2, other.offs, torch.bfloat16), other.slot,
                           other.weight)
        assert torch.equal(got, y)
        mxq.mx_route_bias_step(bias, other.counts, 0.05, out=bias)      # read again by the next replay


def test_a_training_step_in_a_graph():
    """Route, dispatch, gated product with what its gradient needs, gradient and
    bias's step in one graph: every replay gives the eager step's bits."""
    require_gpu()
    say("training step in a graph")
    T, E, K, H, k = 200, 8, 256, 128, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(10)
    w, sw, _, _ = mxq.mx_quantize_2d_dual((torch.randn((E * 2 * H, K), generator=g, device=DEV) * K ** -0.5).bfloat16())
    w, sw = w.view(E, 2 * H, K), sw.view(E, 2 * H, K // 32)
    ebias = torch.randn((E, 2 * H), generator=g, device=DEV)
    start = 0.05 * torch.randn(E, generator=g, device=DEV)
    logits, x = torch.randn((T, E), generator=g, device=DEV), torch.randn((T, K), generator=g, device=DEV).bfloat16()
    dweight, dloss = torch.randn((T, k), generator=g, device=DEV), torch.ones(1, device=DEV)

    def step(bias, plan):
        r = mxq.mx_route_scored(logits, bias=bias, out=plan, groups=2, top_groups=1, scale=2.5)
        q, s, _, _ = mxq.mx_quantize_grouped(mxq.mx_dispatch(x, r.slot, r.src), r.offs)
        y, pre = mxq.mx_grouped_gemm_rows_act(q, s, w, sw, r.offs, ebias, "silu", True, pre=True)
        dpre, dbias = mxq.mx_act_grad(y, pre, "silu", True, r.offs)
        dlogits = mxq.mx_route_scored_grad(logits, r, dweight, dloss)
        mxq.mx_route_bias_step(bias, r.counts, 0.01, out=bias)
        return y, pre, dpre, dbias, dlogits, r.weight, r.loss

    plan, bias = mxq.mx_routing(T, E, k, align=128, device=DEV), start.clone()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        step(bias, plan)
    torch.cuda.current_stream(DEV).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(bias, plan)
    bias.copy_(start)
    other, eager = mxq.mx_routing(T, E, k, align=128, device=DEV), start.clone()
    for i in range(4):
        logits.normal_(generator=g)
        x.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, other)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
        assert torch.equal(bias, eager)
