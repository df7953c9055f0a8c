"""The operators around a block's linears run together, as examples/block_step.py
has them: its gradients against float64 autograd, the same on another stream and
replayed from a graph, and that it trains without an error.

The reference rounds where the step does, products of operands quantized by the
oracle and bf16 in between, so what is left is where the two round to different
neighbours: a product's 1.2e-5 flips one in 200 of the following bf16 roundings
(2^-8 of a value) and one in 6400 of the E4M3 codes behind them (2^-3 of a value):
over the fourteen roundings and ten products of a gradient under 6e-3 of its norm.
In a row of 32 values one flipped code alone is 2^-3 / sqrt(32) = 2.2 %, so 4 % is
allowed."""

import importlib.util
import os

import pytest
import torch

from oracle import fp8
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def step():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "block_step.py")
    spec = importlib.util.spec_from_file_location("block_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def bf16(t):
    return t.float().to(torch.bfloat16).double()


def quantized(t, tile=False):
    return torch.from_numpy(fp8.dequantize(*fp8.quantize(t.numpy(), tile)))


class Round(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x):
        return bf16(x)

    @staticmethod
    def backward(ctx, d):
        return bf16(d)


class RoundForward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x):
        return bf16(x)

    @staticmethod
    def backward(ctx, d):
        return d


class Product(torch.autograd.Function):
    """x w + b of quantized operands; what comes back is rounded before it is quantized."""

    @staticmethod
    def forward(ctx, x, w, b):
        x, w = bf16(x), quantized(bf16(w), True)
        ctx.save_for_backward(x, w)
        return quantized(x) @ w + b

    @staticmethod
    def backward(ctx, d):
        x, w = ctx.saved_tensors
        r = bf16(d)
        dw = quantized(x.t().contiguous()) @ quantized(r.t().contiguous()).t()
        return bf16(quantized(r) @ w.t()), bf16(dw), d.sum(0)


def gelu(z):
    return torch.nn.functional.gelu(z, approximate="tanh")


def activated(z, f):
    """f(z), its slope taken where z has been rounded (as it is kept)."""
    kept = RoundForward.apply(z)
    return f(z).detach() + f(kept) - f(kept).detach()


def reference(params, x, r, target, ids, eps=1e-6):
    """Loss and gradients in float64 on the CPU, for the step's own choice of experts."""
    p = {k: v.double().cpu().requires_grad_() for k, v in params.items()}
    x = x.double().cpu().requires_grad_()
    h = RoundForward.apply(x + r.double().cpu())
    n = RoundForward.apply(h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * p["gain"])
    n = Round.apply(n)                                      # the sum of its gradients is in bf16
    u = activated(Product.apply(n, p["w1"], p["b1"]), gelu)
    out = RoundForward.apply(Product.apply(u, p["w2"], p["b2"]) + h)
    s = torch.sigmoid(n @ p["router"]).gather(1, ids)
    weights = s / s.sum(1, keepdim=True)
    moe, rows = torch.zeros_like(x), n
    for e in range(p["router"].shape[1]):
        token, slot = (ids == e).nonzero(as_tuple=True)
        if len(token) == 0:
            continue
        v = activated(Product.apply(rows[token], p["e1"][e], p["eb1"][e]), torch.nn.functional.silu)
        y = Round.apply(Product.apply(v, p["e2"][e], p["eb2"][e]))
        moe = moe.index_add(0, token, weights[token, slot].unsqueeze(1) * y)
    out = Round.apply(RoundForward.apply(out + RoundForward.apply(moe)))
    loss = 0.5 * (out - target.double().cpu()).square().sum() / x.shape[0]
    loss.backward()
    return loss.detach(), x.grad, {k: v.grad for k, v in p.items()}


def data(tokens, hidden, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]


SIZES = [(320, 256, 320, 8, 160, 2, 4, 2), (77, 128, 96, 6, 64, 3, 3, 2), (1, 64, 64, 4, 32, 2, 2, 1)]


@pytest.mark.parametrize("tokens,hidden,inter,experts,einter,topk,groups,keep", SIZES)
def test_gradients(step, tokens, hidden, inter, experts, einter, topk, groups, keep):
    p = step.init(hidden, inter, experts, einter)
    x, r, target = data(tokens, hidden)
    balance = 0.05 * torch.randn(experts, device="cuda")
    loss, dx, grads, load = step.gradients(p, x, r, target, balance, topk, groups, keep)
    assert int(load.sum()) == tokens * topk
    _, kept = step.forward(p, x, r, balance, topk, groups, keep)
    rloss, rdx, rgrads = reference(p, x, r, target, kept["ids"].long().cpu())
    assert abs(float(loss) - float(rloss)) < 0.04 * float(rloss)
    for name, got, ref in [("dx", dx, rdx)] + [(k, grads[k], rgrads[k]) for k in step.NAMES]:
        got = got.double().cpu()
        assert got.shape == ref.shape, name
        assert float((got - ref).norm()) <= 0.04 * float(ref.norm()), name


def test_stream_and_graph(step):
    """On another stream, and captured and replayed with eager work and
    synchronizations in between: the eager results bit for bit."""
    p = step.init(256, 320, 16, 160)
    x, r, target = data(1000, 256)
    balance = torch.zeros(16, device="cuda")

    def run():
        out, k = step.forward(p, x, r, balance, 4, 4, 2)
        dx, grads = step.backward(p, k, (out.float() - target.float()).to(torch.bfloat16))
        return [out, dx, k["ids"], k["weights"]] + list(grads.values())
    ref = [v.clone() for v in run()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for _ in range(3):
        for v in out:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
        run()


def test_two_captured_steps_share_nothing(step):
    """Two graphs of the calls that have workspaces, replayed in turn on two streams."""
    x = [torch.randn(3000, 512, device="cuda").to(torch.bfloat16) for _ in range(2)]
    w = torch.ones(512, device="cuda")

    def run(t):
        h, rstd, _, q, _ = av.averis_rmsnorm(t, w)
        dh, dw = av.averis_rmsnorm_grad(t, h, w, rstd)
        _, _, db = av.averis_fp8_act_grad(t, z=t, act="gelu")
        return [dh, dw, db]
    ref = [[v.clone() for v in run(t)] for t in x]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in x:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(t))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, ref):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_trains(step):
    p = step.init(256, 320, 8, 128)
    x, r, target = data(512, 256, 6)
    losses = step.train(p, x, r, target, 2, 4, 2, 3, 1.0, 1.0, log=lambda s: None)
    assert len(losses) == 3 and all(v == v for v in losses)
