"""A routed-expert layer on the library's operators, trained and served.

    python examples/routed_experts.py

Training: the router's picks order the tokens by expert (groups padded to 128
rows), the experts' two products run in MXFP8 with the dual-axis cast's
outputs, and the results return weighted to their tokens.  Each step is an
autograd function over the library's forward and backward calls:

    Route    mx_route            backward  mx_route_grad
    Dispatch mx_dispatch         backward  mx_combine without weights
    Experts  mx_grouped_gemm_rows          mx_grouped_gemm_rows (rows), mx_grouped_gemm_k (weights)
    Combine  mx_combine          backward  mx_combine_grad

The backward calls read the routing again, which the next mx_route on the same
buffers writes over: each function notes the routing's generation and its
backward refuses another one.  Micro-batches, or layers, that are alive at once
take a routing each.

Serving: the trained weights become int8 codes with a scale per output
channel, tokens are quantized on their way to the experts (groups padded to
one row), and the whole step is captured once in a graph and replayed.
"""
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import mx9_dual_axis_amd as mxq  # noqa: E402


# ------------------------------------------------------------------- training
class Route(torch.autograd.Function):
    """(logits, plan, valid) -> the picks' weights and the balance loss; the
    rest of the routing is left in the plan."""

    @staticmethod
    def forward(ctx, logits, plan, valid):
        ctx.save_for_backward(logits, valid)
        ctx.plan = mxq.mx_route(logits, valid=valid, out=plan)
        ctx.generation = plan.generation
        return plan.weight.clone(), plan.loss.clone()     # the plan's own are written again by the next call

    @staticmethod
    def backward(ctx, dweight, dloss):
        logits, valid = ctx.saved_tensors
        dlogits = mxq.mx_route_grad(logits, ctx.plan, dweight.contiguous(), dloss.contiguous(), valid,
                                    generation=ctx.generation)
        return dlogits, None, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan, ctx.generation = plan, plan.generation
        return mxq.mx_dispatch(x, plan.slot, plan.src)

    @staticmethod
    def backward(ctx, drows):
        ctx.plan.require(ctx.generation)
        return mxq.mx_combine(drows.contiguous(), ctx.plan.slot), None


class Experts(torch.autograd.Function):
    """rows [M, K], W [E, N, K] in bf16 -> rows [M, N]: each group's rows by its
    expert.  One cast of either operand serves both directions: rowwise codes
    for this product, colwise ones (transposed) for the gradients."""

    @staticmethod
    def forward(ctx, rows, W, plan):
        E, N, K = W.shape
        q, s, qt, st = mxq.mx_quantize_grouped(rows, plan.offs)
        w, sw, wt, swt = mxq.mx_quantize_2d_dual(W.reshape(E * N, K))
        ctx.save_for_backward(qt, st, wt, swt)
        ctx.plan, ctx.generation, ctx.shape = plan, plan.generation, (E, N, K)
        return mxq.mx_grouped_gemm_rows(q, s, w.view(E, N, K), sw.view(E, N, K // 32), plan.offs, torch.bfloat16)

    @staticmethod
    def backward(ctx, dy):
        ctx.plan.require(ctx.generation)
        qt, st, wt, swt = ctx.saved_tensors
        E, N, K = ctx.shape
        offs = ctx.plan.offs
        g, sg, gt, sgt = mxq.mx_quantize_grouped(dy.contiguous(), offs)
        drows = mxq.mx_grouped_gemm_rows(g, sg, wt.view(K, E, N).permute(1, 0, 2), swt.view(E, N // 32, K).permute(0, 2, 1),
                                         offs, torch.bfloat16)
        dW = mxq.mx_grouped_gemm_k(gt, sgt.t(), qt, st.t(), offs, torch.bfloat16)
        return drows, dW, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weight, plan):
        ctx.save_for_backward(rows, weight)
        ctx.plan, ctx.generation = plan, plan.generation
        return mxq.mx_combine(rows, plan.slot, weight)

    @staticmethod
    def backward(ctx, dy):
        ctx.plan.require(ctx.generation)
        rows, weight = ctx.saved_tensors
        drows, dweight = mxq.mx_combine_grad(dy.contiguous(), rows, ctx.plan.slot, weight, ctx.plan.src)
        return drows, dweight, None


def gated(a):
    gate, up = a.chunk(2, dim=1)
    return F.silu(gate) * up


def train_layer(x, params, plan, valid=None):
    """x bf16 [T, K] -> (y bf16 [T, K], balance loss).  `plan` is this pass's
    until its backward is done."""
    router, W1, W2 = params
    weight, balance = Route.apply(x.float() @ router.t(), plan, valid)
    rows = Dispatch.apply(x, plan)
    h = gated(Experts.apply(rows, W1.bfloat16(), plan))
    return Combine.apply(Experts.apply(h.contiguous(), W2.bfloat16(), plan), weight, plan), balance


def init(E, K, H, device, seed=0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    params = [rnd(E, K) * K ** -0.5, rnd(E, 2 * H, K) * K ** -0.5, rnd(E, K, H) * H ** -0.5]
    return [p.requires_grad_() for p in params]


# -------------------------------------------------------------------- serving
class Server:
    """The layer with int8 experts for batches of T tokens, as a graph."""

    def __init__(self, params, T, k, device):
        router, W1, W2 = (p.detach() for p in params)
        E, H2, K = W1.shape
        self.router = router
        q, s = mxq.i8_quantize_rows(W1.reshape(E * H2, K))
        self.W1, self.s1 = q.view(E, H2, K), s.view(E, H2)
        q, s = mxq.i8_quantize_rows(W2.reshape(E * K, H2 // 2))
        self.W2, self.s2 = q.view(E, K, H2 // 2), s.view(E, K)
        self.plan = mxq.mx_routing(T, E, k, align=1, device=device)
        self.x = torch.zeros((T, K), dtype=torch.bfloat16, device=device)
        side = torch.cuda.Stream(device)
        side.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(side):
            self.step(self.x)                             # libraries set themselves up outside the capture
        torch.cuda.current_stream(device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = self.step(self.x)

    def step(self, x):
        plan = mxq.mx_route(x.float() @ self.router.t(), out=self.plan)
        q, s = mxq.mx_dispatch_i8(x, plan.slot, plan.src)
        h = gated(mxq.i8_grouped_gemm_rows(q, s, self.W1, self.s1, plan.offs, torch.bfloat16))
        q, s = mxq.i8_quantize_rows(h)
        return mxq.mx_combine(mxq.i8_grouped_gemm_rows(q, s, self.W2, self.s2, plan.offs, torch.bfloat16), plan.slot,
                              plan.weight)

    def __call__(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def main(T=2048, E=16, K=512, H=256, k=2, steps=60, device="cuda:0"):
    """Train a layer back to the one it is a disturbed copy of, then serve it;
    returns the losses and the served outputs' distance from the trained
    layer's."""
    target = init(E, K, H, device, 2)
    params = [(p + 0.25 * d).detach().requires_grad_() for p, d in zip(target, init(E, K, H, device, 1))]
    plan = mxq.mx_routing(T, E, k, align=128, device=device)
    opt = torch.optim.Adam(params, lr=1e-3)
    g = torch.Generator(device=device)
    g.manual_seed(3)
    losses = []
    for _ in range(steps):
        x = torch.randn((T, K), generator=g, device=device).bfloat16()
        with torch.no_grad():
            want = train_layer(x, target, plan)[0].float()
        y, balance = train_layer(x, params, plan)
        loss = F.mse_loss(y.float(), want) / want.square().mean()
        opt.zero_grad()
        (loss + 0.01 * balance.sum()).backward()
        opt.step()
        losses.append(float(loss.detach()))
    print(f"trained {steps} steps: loss {losses[0]:.3f} -> {losses[-1]:.3f}, tokens per expert "
          f"{int(plan.counts.min())} to {int(plan.counts.max())}", flush=True)
    dist = {}
    for n in (1, 16, T):
        x = torch.randn((n, K), generator=g, device=device).bfloat16()
        serve = Server(params, n, k, device)
        with torch.no_grad():
            want = train_layer(x, params, mxq.mx_routing(n, E, k, align=128, device=device))[0].float()
        got = serve(x).float()
        dist[n] = float((got - want).norm() / want.norm())
        torch.cuda.synchronize(device)
        t = time.perf_counter()
        for _ in range(100):
            serve(x)
        torch.cuda.synchronize(device)
        print(f"serving {n} tokens: {(time.perf_counter() - t) * 1e4:.1f} us a step, {dist[n]:.3f} from the layer as trained",
              flush=True)
    return losses, dist


if __name__ == "__main__":
    main()
