"""A transformer block's second half trained on one GPU: norm, a dense MLP and
routed experts beside it, in fp8 with everything around the products fused.

    python examples/block_step.py [--steps N] [--tokens T] [--experts E] ...

    h = x + r;  n = norm(h) g;  out = h + MLP(n) + experts(n)

Forward: averis_rmsnorm (the sum, its norm in bf16 and, quantized, in both
orientations), averis_fp8_gemm_act (the up-projection with bias and gelu, its value
before the activation kept; the down-projection with bias, back onto h),
averis_moe_route_groups (sigmoid scores, a bias that balances the experts' load,
groups of experts), averis_moe_sort, averis_moe_dispatch, averis_fp8_gemm_act by expert
(silu), averis_moe_combine.  Backward: averis_moe_combine_grad, averis_fp8_act_grad
(through bias and activation into fp8, with the bias's gradient), averis_fp8_gemm,
averis_fp8_gemm_wgrad, averis_moe_route_groups_grad, averis_rmsnorm_grad; then
averis_grad_clip and a plain gradient step on fp32 master weights.  After each
step the routing bias moves a step towards the experts that got fewer tokens than
the mean.  The task is synthetic: fit a fixed random map."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mean_residual_quantized_amd import averis as av

NAMES = ("gain", "w1", "b1", "w2", "b2", "router", "e1", "eb1", "e2", "eb2")


def init(hidden, inter, experts, einter, seed=0):
    """Master parameters in the order of NAMES."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    weight = lambda *s: rand(*s) * s[-2] ** -0.5
    return dict(gain=1.0 + 0.1 * rand(hidden), w1=weight(hidden, inter), b1=0.1 * rand(inter),
                w2=weight(inter, hidden), b2=0.1 * rand(hidden), router=weight(hidden, experts),
                e1=weight(experts, hidden, einter), eb1=0.1 * rand(experts, einter),
                e2=weight(experts, einter, hidden), eb2=0.1 * rand(experts, hidden))


def forward(p, x, r, balance, topk, groups, topk_groups):
    """(out, what the way back needs); x, r bf16 [tokens, hidden]."""
    q = {k: av.averis_fp8_quant_weight(p[k].to(torch.bfloat16)) for k in ("w1", "w2", "e1", "e2")}
    route = dict(groups=groups, topk_groups=topk_groups)
    h, rstd, n, nq, nt = av.averis_rmsnorm(x, p["gain"], residual=r, y=True, transposed=True)
    u, z = av.averis_fp8_gemm_act(nq, q["w1"][0], bias=p["b1"], act="gelu", save=True)
    uq, ut = av.averis_fp8_quant(u, transposed=True)
    dense = av.averis_fp8_gemm_act(uq, q["w2"][0], bias=p["b2"], residual=h)

    logits = n.float() @ p["router"]
    ids, weights = av.averis_moe_route_groups(logits, topk, bias=balance, **route)
    offsets, pos, _ = av.averis_moe_sort(ids, logits.shape[1])
    rq, rt = av.averis_fp8_quant(av.averis_moe_dispatch(n, pos), transposed=True, offsets=offsets)
    e, ez = av.averis_fp8_gemm_act(rq, q["e1"][0], bias=p["eb1"], act="silu", save=True, offsets=offsets)
    eq, et = av.averis_fp8_quant(e, transposed=True, offsets=offsets)
    rows = av.averis_fp8_gemm_act(eq, q["e2"][0], bias=p["eb2"], offsets=offsets)
    out = dense + av.averis_moe_combine(rows, pos, weights)
    kept = dict(q=q, h=h, rstd=rstd, n=n, nt=nt, z=z, ut=ut, logits=logits, ids=ids, weights=weights,
                offsets=offsets, pos=pos, rt=rt, ez=ez, et=et, rows=rows)
    return out, kept


def backward(p, k, dout):
    """(dx, gradients of p): dx of x and of r alike."""
    q, offs = k["q"], k["offsets"]
    # the experts
    drows, dweights = av.averis_moe_combine_grad(dout, k["rows"], k["pos"], k["weights"])
    dq, dt, deb2 = av.averis_fp8_act_grad(drows, offsets=offs)
    de2 = av.averis_fp8_gemm_wgrad(k["et"], dt, offsets=offs, rows=drows.shape[0])
    dq, dt, deb1 = av.averis_fp8_act_grad(av.averis_fp8_gemm(dq, q["e2"][1], offsets=offs), z=k["ez"], act="silu",
                                          offsets=offs)
    de1 = av.averis_fp8_gemm_wgrad(k["rt"], dt, offsets=offs, rows=drows.shape[0])
    dn = av.averis_moe_combine(av.averis_fp8_gemm(dq, q["e1"][1], offsets=offs), k["pos"])
    dlogits = av.averis_moe_route_groups_grad(k["logits"], k["ids"], dweights)
    dn = (dn.float() + dlogits @ p["router"].t()).to(torch.bfloat16)
    # the dense MLP, added onto it
    dq, dt, db2 = av.averis_fp8_act_grad(dout)
    dw2 = av.averis_fp8_gemm_wgrad(k["ut"], dt)
    dq, dt, db1 = av.averis_fp8_act_grad(av.averis_fp8_gemm(dq, q["w2"][1]), z=k["z"], act="gelu")
    dw1 = av.averis_fp8_gemm_wgrad(k["nt"], dt)
    dn = av.averis_fp8_gemm_act(dq, q["w1"][1], residual=dn)
    dx, dgain = av.averis_rmsnorm_grad(dn, k["h"], p["gain"], k["rstd"], dres=dout)
    drouter = k["n"].float().t() @ dlogits
    return dx, dict(zip(NAMES, (dgain, dw1, db1, dw2, db2, drouter, de1, deb1, de2, deb2)))


def gradients(p, x, r, target, balance, topk, groups, topk_groups):
    """(loss, dx, gradients, tokens of each expert) of 0.5 mean over tokens |out - target|^2."""
    out, kept = forward(p, x, r, balance, topk, groups, topk_groups)
    diff = out.float() - target.float()
    loss = 0.5 * diff.square().sum() / x.shape[0]
    dx, grads = backward(p, kept, (diff / x.shape[0]).to(torch.bfloat16))
    return loss, dx, grads, kept["offsets"].diff()


def train(p, x, r, target, topk, groups, topk_groups, steps, lr, max_norm, log=print):
    """`steps` clipped gradient steps; the losses."""
    balance = torch.zeros(p["router"].shape[1], device="cuda")
    losses = []
    for i in range(steps):
        loss, _, grads, load = gradients(p, x, r, target, balance, topk, groups, topk_groups)
        norm = av.averis_grad_clip(list(grads.values()), max_norm)
        for name, g in grads.items():
            p[name].add_(g.to(p[name].dtype), alpha=-lr)
        load = load.float()
        balance += 1e-3 * torch.sign(load.mean() - load)
        losses.append(float(loss))
        log("step %3d  loss %9.4f  gradient norm %.4f  largest load %.2f of the mean"
            % (i, losses[-1], float(norm), float(load.max() / load.mean())))
    return losses


def main():
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 20), ("tokens", 4096), ("hidden", 2048), ("inter", 4096), ("experts", 64),
                        ("expert-inter", 768), ("topk", 8), ("groups", 8), ("topk-groups", 4)):
        a.add_argument("--" + name, type=int, default=value)
    a.add_argument("--lr", type=float, default=1.0)
    a.add_argument("--max-norm", type=float, default=1.0)
    a = a.parse_args()
    p = init(a.hidden, a.inter, a.experts, a.expert_inter)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    m = torch.randn(a.hidden, a.hidden, generator=g, device="cuda") * a.hidden ** -0.5
    target = (x.float() + r.float() + torch.tanh(x.float() @ m)).to(torch.bfloat16)
    how = (a.topk, a.groups, a.topk_groups)
    train(p, x, r, target, *how, a.steps, a.lr, a.max_norm)
    balance = torch.zeros(a.experts, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(5):
        grads = gradients(p, x, r, target, balance, *how)[2]
        av.averis_grad_clip(list(grads.values()), a.max_norm)
    end.record()
    torch.cuda.synchronize()
    print("forward, backward and clip: %.3f ms a step" % (start.elapsed_time(end) / 5))


if __name__ == "__main__":
    main()
