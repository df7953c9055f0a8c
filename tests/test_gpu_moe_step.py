"""The mixture-of-experts step of examples/moe_step.py: its gradients against
float64 autograd, and its loss on a fit.

fp8: the reference rounds where the step does, products of operands quantized
by the oracle and bf16 in between, so what is left is where the two round to
different neighbours.  The products differ by 1.2e-5 of their norm, which
flips one in 200 of the following bf16 roundings (2^-8 of a value) and one in
6400 of the E4M3 codes behind them (2^-3 of a value): over the ten roundings
and five products of a gradient 4e-3 of its norm.  In a row of 32 values one
flipped code alone is 2^-3 / sqrt(32) = 2.2 %, so 4 % is allowed.

fp4: the reference is unquantized.  E2M1 with 16-element scales errs by about
9.5 % an operand, with stochastic rounding nearly half as much again: 20 % a
product, four of them: too coarse to say more than the direction, so cosine
> 0.7 is asked for."""

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
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_step.py")
    spec = importlib.util.spec_from_file_location("moe_step", path)
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


class Fp8Product(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        x, w = bf16(x), quantized(bf16(w), True)
        ctx.save_for_backward(x, w)
        return bf16(quantized(x) @ w)

    @staticmethod
    def backward(ctx, d):
        x, w = ctx.saved_tensors
        d = bf16(d)
        dw = quantized(x.t().contiguous()) @ quantized(d.t().contiguous()).t()
        return bf16(quantized(d) @ w.t()), bf16(dw)


def plain_product(x, w):
    return x @ (w + (bf16(w) - w).detach())


def reference(params, x, target, topk, linear):
    """Loss and gradients in float64 on the CPU."""
    fp = linear == "fp8"
    product, rnd = (Fp8Product.apply, Round.apply) if fp else (plain_product, lambda t: t)
    p = [v.double().cpu().requires_grad_() for v in params]
    x = x.double().cpu().requires_grad_()
    logits = x @ p[0]
    top, ids = logits.topk(topk, dim=1)
    r = torch.softmax(top, dim=1)
    y, rows = torch.zeros_like(x), rnd(x)
    for e in range(p[0].shape[1]):
        token, slot = (ids == e).nonzero(as_tuple=True)
        if len(token) == 0:
            continue
        gate, up = product(rows[token], p[1][e]).chunk(2, dim=1)
        out = product(torch.nn.functional.silu(gate) * up, p[2][e])
        y = y.index_add(0, token, r[token, slot].unsqueeze(1) * out)
    loss = 0.5 * (rnd(y) - target.double().cpu()).square().sum() / x.shape[0]
    loss.backward()
    return loss.detach(), x.grad, [v.grad for v in p]


@pytest.mark.parametrize("linear", ["fp8", "fp4"])
@pytest.mark.parametrize("tokens,experts,topk,hidden,inter", [(320, 8, 2, 256, 160), (77, 5, 3, 128, 64),
                                                              (1, 4, 4, 64, 32)])
def test_gradients(step, linear, tokens, experts, topk, hidden, inter):
    params = step.init(experts, hidden, inter)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, target = (torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    loss, dx, grads = step.gradients(params, x, target, topk, linear)
    rloss, rdx, rgrads = reference(params, x, target, topk, linear)
    assert abs(float(loss) - float(rloss)) < (0.04 if linear == "fp8" else 0.7) * float(rloss)
    for got, ref in zip([dx] + grads, [rdx] + rgrads):
        got = got.double().cpu()
        assert got.shape == ref.shape
        if linear == "fp8":
            assert float((got - ref).norm()) < 0.04 * float(ref.norm())
        else:
            assert float((got * ref).sum()) > 0.7 * float(got.norm() * ref.norm())


@pytest.mark.parametrize("linear", ["fp8", "fp4"])
def test_loss_falls(step, linear):
    params = step.init(8, 256, 128)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(512, 256, generator=g, device="cuda").to(torch.bfloat16)
    target = torch.tanh(x.float())
    losses = step.train(params, x, target.to(torch.bfloat16), 2, linear, 12, 1.0, 1.0, log=lambda s: None)
    assert losses[-1] < 0.9 * losses[0]
