"""A mixture-of-experts layer trained on one GPU with the library's operators.

    python examples/moe_step.py [--linear fp8|fp4] [--steps N] [--tokens T] ...

The layer: y_t = sum over the top-k experts e of token t, with router weights
r_te, of r_te W2_e (silu(g) * u), [g, u] = W1_e x_t.  One step is

    logits           torch product (fp32)
    averis_moe_route, averis_moe_sort              experts, weights, row order
    averis_moe_dispatch                            rows sorted by expert
    averis_fp8_quant, averis_fp8_gemm              W1 by expert, then W2
    averis_moe_combine                             back to tokens, weighted
    averis_moe_combine_grad                        and each step backwards:
    averis_fp8_gemm, averis_fp8_gemm_wgrad         dgrad, wgrad
    averis_moe_combine, averis_moe_route_grad      dx, dlogits
    averis_grad_clip                               all gradients, one norm

and a plain gradient step on fp32 master weights.  --linear fp4 computes the
forward and dgrad products from the mean-residual FP4 split
(averis_split_quant_grouped_rank1, averis_gemm_grouped_rank1); the weight
gradient stays in fp8.  The task is synthetic: fit a fixed random map."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mean_residual_quantized_amd import averis as av


class Fp8Linear:
    """y = x W by expert segment; W [experts, k, n] in bf16."""

    def __init__(self, w):
        self.wt, self.wd = av.averis_fp8_quant_weight(w)

    def forward(self, x, offsets):
        q, self.xt = av.averis_fp8_quant(x, transposed=True, offsets=offsets)
        return av.averis_fp8_gemm(q, self.wt, offsets=offsets)

    def backward(self, dy, offsets):
        """(dx, dw)"""
        q, dt = av.averis_fp8_quant(dy, transposed=True, offsets=offsets)
        return (av.averis_fp8_gemm(q, self.wd, offsets=offsets),
                av.averis_fp8_gemm_wgrad(self.xt, dt, offsets=offsets, rows=dy.shape[0]))


class Fp4Linear:
    """The same with the forward and dgrad products of the mean-residual split."""

    def __init__(self, w):
        self.wt = av.averis_quant_batched(w, transpose=True)
        self.wd = av.averis_quant_batched(w)

    @staticmethod
    def product(x, w, offsets, seed):
        q, _, _, rho = av.averis_split_quant_grouped_rank1(x, offsets, w, seed=seed)
        return av.averis_gemm_grouped_rank1(q, rho, w, offsets, out_dtype=torch.bfloat16)

    def forward(self, x, offsets):
        _, self.xt = av.averis_fp8_quant(x, transposed=True, offsets=offsets, plain=False)
        return self.product(x, self.wt, offsets, 0)

    def backward(self, dy, offsets):
        _, dt = av.averis_fp8_quant(dy, transposed=True, offsets=offsets, plain=False)
        return (self.product(dy, self.wd, offsets, 1),
                av.averis_fp8_gemm_wgrad(self.xt, dt, offsets=offsets, rows=dy.shape[0]))


LINEARS = {"fp8": Fp8Linear, "fp4": Fp4Linear}


def init(experts, hidden, inter, seed=0):
    """Master weights: router [hidden, experts], W1 [experts, hidden, 2 inter],
    W2 [experts, inter, hidden]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = [(hidden, experts), (experts, hidden, 2 * inter), (experts, inter, hidden)]
    return [torch.randn(s, generator=g, device="cuda") * s[-2] ** -0.5 for s in shapes]


def gradients(params, x, target, topk, linear="fp8"):
    """(loss, dx, gradients of params) of 0.5 mean over tokens |y - target|^2;
    x, target bf16 [tokens, hidden]."""
    router, w1, w2 = params
    lin1, lin2 = (LINEARS[linear](w.to(torch.bfloat16)) for w in (w1, w2))

    logits = x.float() @ router
    ids, weights = av.averis_moe_route(logits, topk)
    offsets, pos, _ = av.averis_moe_sort(ids, router.shape[1])
    rows = av.averis_moe_dispatch(x, pos)
    gate, up = lin1.forward(rows, offsets).float().chunk(2, dim=1)
    s = torch.sigmoid(gate)
    out = lin2.forward((gate * s * up).to(torch.bfloat16), offsets)
    y = av.averis_moe_combine(out, pos, weights)

    diff = y.float() - target.float()
    loss = 0.5 * diff.square().sum() / x.shape[0]

    dout, dweights = av.averis_moe_combine_grad((diff / x.shape[0]).to(torch.bfloat16), out, pos,
                                                weights)
    dh, dw2 = lin2.backward(dout, offsets)
    dh = dh.float()
    dgu = torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], dim=1)
    drows, dw1 = lin1.backward(dgu.to(torch.bfloat16), offsets)
    dlogits = av.averis_moe_route_grad(logits, ids, dweights)
    dx = av.averis_moe_combine(drows, pos).float() + dlogits @ router.t()
    return loss, dx, [x.float().t() @ dlogits, dw1, dw2]


def train(params, x, target, topk, linear, steps, lr, max_norm, log=print):
    """`steps` clipped gradient steps; the losses."""
    losses = []
    for i in range(steps):
        loss, _, grads = gradients(params, x, target, topk, linear)
        norm = av.averis_grad_clip(grads, max_norm)
        for p, g in zip(params, grads):
            p.add_(g.to(p.dtype), alpha=-lr)
        losses.append(float(loss))
        log("step %3d  loss %9.4f  gradient norm %.4f" % (i, losses[-1], float(norm)))
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--linear", choices=sorted(LINEARS), default="fp8")
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--topk", type=int, default=8)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inter", type=int, default=768)
    p.add_argument("--lr", type=float, default=4.0)
    p.add_argument("--max-norm", type=float, default=1.0)
    a = p.parse_args()
    params = init(a.experts, a.hidden, a.inter)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    m = torch.randn(a.hidden, a.hidden, generator=g, device="cuda") * a.hidden ** -0.5
    target = torch.tanh(x.float() @ m).to(torch.bfloat16)
    train(params, x, target, a.topk, a.linear, a.steps, a.lr, a.max_norm)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(5):
        _, _, grads = gradients(params, x, target, a.topk, a.linear)
        av.averis_grad_clip(grads, a.max_norm)
    end.record()
    torch.cuda.synchronize()
    print("forward, backward and clip: %.3f ms a step" % (start.elapsed_time(end) / 5))


if __name__ == "__main__":
    main()
