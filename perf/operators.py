"""What the operators of a mixture-of-experts training step cost, and what they have to compute.

Four groups of cases:

* ``route``     router weights and experts of each token, the order of the tokens' rows by expert, and the
                router's gradient;
* ``exchange``  tokens to their experts' rows and back with the router's weights, and both gradients;
* ``fp8``       linear layers in 8-bit floating point with a power-of-two scale for each block of 128: whole
                training steps (forward, dgrad, wgrad), one weight or one for each expert, and single tokens
                against a weight that is kept quantized;
* ``clip``      the norm over all gradients of a model, and the clipped gradients.

``run`` computes a case in plain torch operations (``own`` false) or with the package's entry points.
"""

import math
import random

import torch

own = False

BLOCK = 128          # elements that share a scale
E4M3_MAX = 448.0
CLIP_EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one batch of single tokens in serving: latency alone
        dict(name="route 16 tokens", op="route", tokens=16, experts=64, topk=8, dtype="bf16",
             renorm=True, masked=0.0, train=False),
        # the mixture-of-experts workload's router, with its gradient
        dict(name="route 4096 tokens", op="route", tokens=4096, experts=64, topk=8, dtype="bf16",
             renorm=True, masked=0.0, train=True),
        # a long batch, fp32 logits, experts masked per token (some rows wholly), plain softmax weights
        dict(name="route 65521 tokens masked", op="route", tokens=65521, experts=128, topk=6,
             dtype="f32", renorm=False, masked=0.3, train=True),
        # the rows of one batch of single tokens
        dict(name="exchange 16 tokens", op="exchange", tokens=16, experts=64, topk=8, cols=2048,
             dtype="bf16", dropped=0.0, train=False),
        # the mixture-of-experts workload: 32768 rows of 2048, forward and both gradients
        dict(name="exchange 4096 tokens", op="exchange", tokens=4096, experts=64, topk=8, cols=2048,
             dtype="bf16", dropped=0.0, train=True),
        # odd sizes in fp32, a tenth of the slots dropped by a capacity limit
        dict(name="exchange 10007 tokens ragged", op="exchange", tokens=10007, experts=30, topk=3,
             cols=999, dtype="f32", dropped=0.1, train=True),
        # single tokens through a projection whose weight is kept in 8 bits
        dict(name="fp8 16 tokens", op="fp8", rows=16, k=2048, n=1024, experts=1, train=False),
        # the gate projection of the block sweep: forward, dgrad and wgrad
        dict(name="fp8 gate 16384 tokens", op="fp8", rows=16384, k=1024, n=3072, experts=1, train=True),
        # the mixture-of-experts linear: 32768 routed rows over 64 experts, forward, dgrad, wgrad
        dict(name="fp8 64 experts", op="fp8", rows=32768, k=2048, n=768, experts=64, train=True),
        # odd sizes on every axis
        dict(name="fp8 ragged", op="fp8", rows=2999, k=1000, n=1333, experts=1, train=True),
        # the gradients of one block's seven weights
        dict(name="clip one block", op="clip", tensors=7, elements=15_728_640, dtype="bf16", odd=False),
        # a model's gradients in fp32, buckets with tensors of every size at odd places
        dict(name="clip 310 tensors", op="clip", tensors=310, elements=268_435_456, dtype="f32", odd=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "exchange", "fp8", "clip"])
    if op == "route":
        e = _log(rng, 4, 256)
        return dict(op=op, tokens=_log(rng, 1, 65536), experts=e, topk=rng.randint(1, min(8, e)),
                    dtype=rng.choice(["bf16", "f32"]), renorm=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.3]), train=rng.random() < 0.5)
    if op == "exchange":
        h, k = _log(rng, 64, 4096), rng.randint(1, 8)
        dtype = rng.choice(["bf16", "f32"])
        most = (1 << 28) // (h * k * _size(dtype))
        return dict(op=op, tokens=_log(rng, 1, max(2, min(65536, most))), experts=_log(rng, 8, 256),
                    topk=k, cols=h, dtype=dtype, dropped=rng.choice([0.0, 0.2]),
                    train=rng.random() < 0.5)
    if op == "fp8" and rng.random() < 0.4:
        return dict(op=op, rows=_log(rng, 1, 512), k=_log(rng, 64, 4096), n=_log(rng, 64, 8192),
                    experts=1, train=False)
    if op == "fp8":
        k, n = _log(rng, 64, 4096), _log(rng, 64, 3000)
        experts = rng.choice([1, 1, _log(rng, 2, max(2, min(64, 100_000_000 // (k * n))))])
        return dict(op=op, rows=_log(rng, 64, min(32768, 50_000_000_000 // (k * n))), k=k, n=n,
                    experts=experts, train=True)
    n = _log(rng, 1, 400)
    return dict(op=op, tensors=n, elements=max(n, _log(rng, 10_000, 250_000_000)),
                dtype=rng.choice(["bf16", "f32"]), odd=rng.random() < 0.5)


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def work(c):
    if c["op"] == "route":
        t, e, k, s = c["tokens"], c["experts"], c["topk"], _size(c["dtype"])
        # logits in; ids, weights, rows of slots, slots of rows and offsets out
        b, f = t * e * s + 16 * t * k + 8 * (e + 1), 4 * t * e
        if c["train"]:
            b += 4 * t * k + t * e * s   # weights' gradient in, logits' gradient out
            f += 4 * t * e
        return dict(bytes=b, flops=f)
    if c["op"] == "exchange":
        t, k, h, s = c["tokens"], c["topk"], c["cols"], _size(c["dtype"])
        # dispatch: x in, rows out; combine: rows and weights in, y out
        b, f = t * h * s * (1 + k) + t * h * s * (1 + k) + 8 * t * k, 2 * t * k * h
        if c["train"]:
            # combine's gradient: dy in, rows' gradient and weights' out (rows are read
            # already); dispatch's: rows' gradient in, dx out
            b += t * h * s * (1 + k) + 4 * t * k + t * h * s * (1 + k)
            f += 4 * t * k * h
        return dict(bytes=b, flops=f)
    if c["op"] == "fp8":
        m, k, n, e = c["rows"], c["k"], c["n"], c["experts"]
        if not c["train"]:
            return dict(bytes=2 * m * k + n * k + 2 * m * n, flops=2 * m * n * k)
        # x, w and the output's gradient in; y, dx and dw out
        return dict(bytes=4 * m * k + 4 * e * k * n + 4 * m * n,
                    flops=3 * 2 * m * n * k)
    s = _size(c["dtype"])
    return dict(bytes=2 * s * c["elements"], flops=3 * c["elements"])


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _biased(g, rows, cols):
    """Activations with a coherent mean over the rows and a few strong directions."""
    x = _randn(g, rows, cols).mul_(0.5)
    x += 3.0 * _randn(g, cols) + 1.5
    x += _randn(g, rows, 1) * _randn(g, cols) * (4.0 / math.sqrt(cols))
    return x.to(torch.bfloat16)


def _offsets(g, rows, experts):
    """Row counts of experts whose popularity falls off as a power law; some get none."""
    p = torch.arange(1, experts + 1, device="cuda").double().pow(-1.1)
    p = p[torch.randperm(experts, generator=g, device="cuda")]
    cuts = torch.round(torch.cumsum(p / p.sum(), 0) * rows).long()
    cuts[-1] = rows
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), cuts])


def _shares(c):
    """Sizes of a model's tensors: a few hold most of the elements, many are vectors."""
    rng, n, total = random.Random(c["elements"]), c["tensors"], c["elements"]
    w = [math.exp(rng.gauss(0.0, 2.5)) for _ in range(n)]
    sizes = [int(v / sum(w) * (total - n)) + 1 for v in w]
    sizes[0] += total - sum(sizes)
    # of any length, or of whole 128-byte lines
    return sizes if c["odd"] else [-(-v // 64) * 64 for v in sizes]


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        logits = _randn(g, t, e) * 1.5 - 1.1 * torch.log(1.0 + torch.arange(e, device="cuda"))
        if c["masked"]:
            # experts closed to a token, and tokens (padding) closed to all of them
            logits[torch.rand(t, e, generator=g, device="cuda") < c["masked"]] = -math.inf
            logits[torch.rand(t, generator=g, device="cuda") < 0.05] = -math.inf
        return dict(case=c, logits=logits.to(_dtype(c["dtype"])), dweights=_randn(g, t, c["topk"]))
    if c["op"] == "exchange":
        t, e, k, h, dt = c["tokens"], c["experts"], c["topk"], c["cols"], _dtype(c["dtype"])
        ids = (torch.rand(t, k, generator=g, device="cuda").pow(1.5) * e).int()
        if c["dropped"]:
            ids[torch.rand(t, k, generator=g, device="cuda") < c["dropped"]] = -1
        pos = _sorted_by_expert(ids, e)[1]
        w = torch.rand(t, k, generator=g, device="cuda")
        s = dict(case=c, pos=pos, weights=w / w.sum(1, keepdim=True), x=_randn(g, t, h).to(dt),
                 rows=_randn(g, t * k, h).to(dt))
        if c["train"]:
            s.update(dy=_randn(g, t, h).to(dt), drows=_randn(g, t * k, h).to(dt))
        return s
    if c["op"] == "fp8":
        m, k, n, e = c["rows"], c["k"], c["n"], c["experts"]
        x = _biased(g, m, k)
        w = (_randn(g, e, k, n) / math.sqrt(k)).to(torch.bfloat16)
        if not c["train"]:
            # the weight as a serving program keeps it: codes and scales of W^T, one scale to a
            # 128 x 128 tile, rows padded to whole blocks and scale rows to whole words
            codes, scales = _tile_codes(w[0].t().float())
            return dict(case=c, x=x, codes=codes, scales=scales)
        d = (0.05 * _randn(g, n) + math.sqrt(1e-3) * _randn(g, m, n)).to(torch.bfloat16)
        offs = _offsets(g, m, e) if e > 1 else None
        return dict(case=c, x=x, w=w if e > 1 else w[0], d=d, offsets=offs,
                    cuts=offs.tolist() if e > 1 else [0, m])
    sizes = _shares(c)   # one after the other in a bucket
    grads = (_randn(g, sum(sizes)) * 1e-2).to(_dtype(c["dtype"]))
    out = torch.zeros_like(grads)
    return dict(case=c, flat=out, grads=list(grads.split(sizes)), out=list(out.split(sizes)),
                max_norm=1.0)


# --------------------------------------------------------------------------
# the operators in plain form: fp32, rounded once
# --------------------------------------------------------------------------

def _softmax_parts(l):
    top = l.max(1, keepdim=True).values
    return torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))


def _routed(logits, topk, renorm):
    l = logits.float()
    top, at = torch.sort(l, dim=1, descending=True, stable=True)
    top, at = top[:, :topk], at[:, :topk]
    open_ = top != -math.inf
    z = _softmax_parts(l)
    zs = torch.where(open_, torch.gather(z, 1, at), torch.zeros_like(top))
    total = zs.sum(1, keepdim=True) if renorm else z.sum(1, keepdim=True)
    w = zs / torch.where(total == 0, torch.ones_like(total), total)
    return torch.where(open_, at, torch.full_like(at, -1)).int(), w


def _routed_gradient(logits, ids, dweights, renorm):
    open_ = ids >= 0
    at = ids.clamp(min=0).long()
    z = _softmax_parts(logits.float())
    zs = torch.where(open_, torch.gather(z, 1, at), torch.zeros_like(dweights))
    total = zs.sum(1, keepdim=True) if renorm else z.sum(1, keepdim=True)
    total = torch.where(total == 0, torch.ones_like(total), total)
    w = zs / total
    mean = (w * dweights).sum(1, keepdim=True)
    if renorm:
        d = torch.zeros_like(z).scatter_add_(1, at, w * (dweights - mean))
    else:
        d = (-mean * (z / total)).scatter_add_(1, at, w * dweights)
    return d.to(logits.dtype)


def _sorted_by_expert(ids, experts):
    """offsets, each slot's row (~row where the slot has no expert), each row's slot."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    src = torch.sort(key, stable=True).indices
    row = torch.empty_like(src)
    row[src] = torch.arange(src.numel(), device=src.device)
    counts = (key[:, None] == torch.arange(experts, device=key.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    pos = torch.where(key < experts, row, ~row)
    return offsets, pos.reshape(ids.shape).int(), src.int()


def _dispatched(x, pos):
    t, k = pos.shape
    p = pos.long()
    rows = torch.empty(t * k, x.shape[1], dtype=x.dtype, device=x.device)
    rows[torch.where(p < 0, ~p, p)] = torch.where((p < 0)[:, :, None], torch.zeros_like(x[:1, :1]), x[:, None, :])
    return rows


def _picked(rows, pos):
    p = pos.long()
    r = rows[p.clamp(min=0)].float()
    return torch.where((p < 0)[:, :, None], torch.zeros_like(r[:1, :1, :1]), r)


def _combined(rows, pos, weights):
    r = _picked(rows, pos)
    return (r if weights is None else r * weights[:, :, None]).sum(1).to(rows.dtype)


def _combined_gradient(dy, rows, pos, weights):
    p, d = pos.long(), dy.float()[:, None, :]
    kept = torch.where(p < 0, torch.zeros_like(weights), weights)
    drows = torch.empty_like(rows)
    drows[torch.where(p < 0, ~p, p)] = (kept[:, :, None] * d).to(rows.dtype)
    return drows, (_picked(rows, pos) * d).sum(2)


def _powers(amax):
    """The smallest 2^e with amax <= 448 * 2^e, at least 2^-127."""
    m, x = torch.frexp(amax)            # amax = m 2^x, m in [0.5, 1); 448 = 0.875 2^9
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax == 0, torch.full_like(e, -127), e).clamp(min=-127)


def _padded(a, rows, cols):
    return torch.nn.functional.pad(a, (0, -a.shape[1] % cols, 0, -a.shape[0] % rows))


def _rounded(t, e):
    """t in E4M3 steps of 2^e, as the values they stand for (e for each element's block)."""
    e = e.float()
    half = torch.exp2(-torch.floor(e / 2)), torch.exp2(-torch.ceil(e / 2))
    q = (t * half[0] * half[1]).to(torch.float8_e4m3fn)
    return q, q.float() / half[0] / half[1]


def _by_runs(a):
    """Values of `a` with one scale for each run of 128 along its columns."""
    r, k = a.shape
    b = _padded(a.float(), 1, BLOCK).reshape(r, -(-k // BLOCK), BLOCK)
    v = _rounded(b, _powers(b.abs().amax(2, keepdim=True)))[1]
    return v.flatten(1)[:, :k]


def _tiles(w):
    n, k = w.shape
    b = _padded(w.float(), BLOCK, BLOCK)
    b = b.reshape(b.shape[0] // BLOCK, BLOCK, b.shape[1] // BLOCK, BLOCK)
    return b, _powers(b.abs().amax((1, 3), keepdim=True))


def _by_tiles(w):
    """Values of `w` with one scale for each 128 x 128 tile."""
    b, e = _tiles(w)
    v = _rounded(b, e)[1]
    return v.reshape(b.shape[0] * BLOCK, -1)[:w.shape[0], :w.shape[1]]


def _tile_codes(w):
    """Codes (rows padded to whole blocks) and scale bytes (rows padded to whole words) of `w`."""
    n = w.shape[0]
    b, e = _tiles(w)
    codes = _rounded(b, e)[0].view(torch.uint8).reshape(b.shape[0] * BLOCK, -1)[:n]
    scales = (e + 127).to(torch.uint8).expand(-1, BLOCK, -1, -1).reshape(b.shape[0] * BLOCK, -1)[:n]
    return codes.contiguous(), _padded(scales, 1, 4).contiguous()


def _linear(s):
    """y = x w, dx = d w^T, dw = x^T d from the quantized values of each product's operands."""
    x, w, d, cuts = s["x"], s["w"], s["d"], s["cuts"]
    stack = w if w.dim() == 3 else w[None]
    parts = [(x[a:b], _by_tiles(stack[i]), d[a:b]) for i, (a, b) in enumerate(zip(cuts, cuts[1:]))]
    y = torch.cat([_by_runs(xs) @ ws for xs, ws, ds in parts])
    dx = torch.cat([_by_runs(ds) @ ws.t() for xs, ws, ds in parts])
    dw = torch.stack([_by_runs(xs.t()) @ _by_runs(ds.t()).t() for xs, ws, ds in parts])
    y, dx, dw = (v.to(torch.bfloat16) for v in (y, dx, dw))
    return dict(y=y, dx=dx, dw=dw if w.dim() == 3 else dw[0])


def _served(s):
    n, k = s["codes"].shape[0], s["x"].shape[1]
    scale = torch.exp2(s["scales"].float() - 127)[:, :s["codes"].shape[1] // BLOCK]
    w = s["codes"].view(torch.float8_e4m3fn).float().reshape(n, -1, BLOCK) * scale[:, :, None]
    return dict(y=(_by_runs(s["x"]) @ w.reshape(n, -1)[:, :k].t()).to(torch.bfloat16))


def _clipped(s):
    norm = torch.sqrt(torch.stack([g.float().square().sum() for g in s["grads"]]).sum())
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    torch._foreach_copy_(s["out"], [g.float() * coef for g in s["grads"]])
    return dict(norm=norm, grads=s["flat"])


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        ids, w = _routed(s["logits"], c["topk"], c["renorm"])
        offsets, pos, src = _sorted_by_expert(ids, c["experts"])
        r = dict(ids=ids, weights=w, offsets=offsets, pos=pos, src=src)
        if c["train"]:
            r["dlogits"] = _routed_gradient(s["logits"], ids, s["dweights"], c["renorm"])
        return r
    if c["op"] == "exchange":
        r = dict(rows=_dispatched(s["x"], s["pos"]), y=_combined(s["rows"], s["pos"], s["weights"]))
        if c["train"]:
            r["drows"], r["dweights"] = _combined_gradient(s["dy"], s["rows"], s["pos"], s["weights"])
            r["dx"] = _combined(s["drows"], s["pos"], None)
        return r
    if c["op"] == "fp8":
        return _linear(s) if c["train"] else _served(s)
    return _clipped(s)


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------

def _own(s):
    from mean_residual_quantized_amd import averis as av

    c = s["case"]
    if c["op"] == "route":
        ids, w = av.averis_moe_route(s["logits"], c["topk"], renorm=c["renorm"])
        offsets, pos, src = av.averis_moe_sort(ids, c["experts"])
        r = dict(ids=ids, weights=w, offsets=offsets, pos=pos, src=src)
        if c["train"]:
            r["dlogits"] = av.averis_moe_route_grad(s["logits"], ids, s["dweights"], renorm=c["renorm"])
        return r
    if c["op"] == "exchange":
        r = dict(rows=av.averis_moe_dispatch(s["x"], s["pos"]),
                 y=av.averis_moe_combine(s["rows"], s["pos"], s["weights"]))
        if c["train"]:
            r["drows"], r["dweights"] = av.averis_moe_combine_grad(s["dy"], s["rows"], s["pos"], s["weights"])
            r["dx"] = av.averis_moe_combine(s["drows"], s["pos"])
        return r
    if c["op"] == "fp8" and c["train"]:
        offs = s["offsets"]
        xq, xt = av.averis_fp8_quant(s["x"], transposed=True, offsets=offs)
        dq, dt = av.averis_fp8_quant(s["d"], transposed=True, offsets=offs)
        wt, wd = av.averis_fp8_quant_weight(s["w"])
        return dict(y=av.averis_fp8_gemm(xq, wt, torch.bfloat16, offsets=offs),
                    dx=av.averis_fp8_gemm(dq, wd, torch.bfloat16, offsets=offs),
                    dw=av.averis_fp8_gemm_wgrad(xt, dt, torch.bfloat16, offsets=offs))
    if c["op"] == "fp8":
        xq = av.averis_fp8_quant(s["x"])
        wt = av.FP8(s["codes"], s["scales"], c["n"], c["k"])
        return dict(y=av.averis_fp8_gemm(xq, wt, torch.bfloat16))
    norm = av.averis_grad_clip(s["grads"], s["max_norm"], eps=CLIP_EPS, out=s["out"])
    return dict(norm=norm, grads=s["flat"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_quantized(t, block_amax):
    """t (float64) rounded to E4M3 on the grid of its block's scale; block_amax broadcasts to t."""
    a = block_amax.clamp(min=1e-300)
    e = torch.ceil(torch.log2(a / E4M3_MAX))
    e = torch.where(a <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)   # log2 is inexact at powers of two
    e = torch.where(a > E4M3_MAX * torch.exp2(e), e + 1, e).clamp(min=-127)
    v = t / torch.exp2(e)
    # spacing of E4M3 at |v|: 2^(floor(log2 |v|) - 3), at least 2^-9
    step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
    return torch.round(v / step) * step * torch.exp2(e)   # torch.round takes ties to even


def _exact_runs(a):
    a = a.double()
    p = torch.nn.functional.pad(a, (0, -a.shape[1] % BLOCK))
    m = p.abs().reshape(a.shape[0], p.shape[1] // BLOCK, BLOCK).amax(2).repeat_interleave(BLOCK, 1)
    return _exact_quantized(p, m)[:, :a.shape[1]]


def _exact_tiles(w):
    w = w.double()
    p = torch.nn.functional.pad(w, (0, -w.shape[1] % BLOCK, 0, -w.shape[0] % BLOCK))
    m = p.abs().unfold(0, BLOCK, BLOCK).unfold(1, BLOCK, BLOCK).amax((2, 3))
    m = m.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
    return _exact_quantized(p, m)[:w.shape[0], :w.shape[1]]


def _exact_route(c, s):
    l, k = s["logits"].double(), c["topk"]
    ids = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
    chosen = torch.zeros_like(l).scatter_(1, ids, 1.0).bool() & (l != -math.inf)
    if c["renorm"]:
        p = torch.softmax(l.masked_fill(~chosen, -math.inf), 1)
    else:
        p = torch.softmax(l, 1)
    p = torch.nan_to_num(p)          # rows with no open expert
    w = torch.gather(p * chosen, 1, ids)
    r = dict(ids=None, weights=w, offsets=None, pos=None, src=None)
    if c["train"]:
        dw = torch.zeros_like(l).scatter_(1, ids, s["dweights"].double()) * chosen
        r["dlogits"] = p * (dw - (p * dw).sum(1, keepdim=True))
    return r


def _exact_exchange(c, s):
    t, k = s["pos"].shape
    p = s["pos"].reshape(-1).long()
    kept = (p >= 0).double()
    at = torch.where(p < 0, ~p, p)
    token = torch.arange(t, device=p.device).repeat_interleave(k)
    rows = torch.zeros(t * k, c["cols"], dtype=torch.float64, device=p.device)
    rows[at] = s["x"].double()[token] * kept[:, None]
    w = s["weights"].double().reshape(-1) * kept
    zero = torch.zeros(t, c["cols"], dtype=torch.float64, device=p.device)
    r = dict(rows=rows, y=zero.index_add(0, token, s["rows"].double()[at] * w[:, None]))
    if c["train"]:
        dy = s["dy"].double()[token]
        drows = torch.zeros_like(rows)
        drows[at] = w[:, None] * dy
        r["drows"] = drows
        r["dweights"] = ((s["rows"].double()[at] * dy).sum(1) * kept).reshape(t, k)
        r["dx"] = zero.index_add(0, token, s["drows"].double()[at] * kept[:, None])
    return r


def _exact_step(x, w, d):
    wq = _exact_tiles(w)
    return (torch.mm(_exact_runs(x), wq), torch.mm(_exact_runs(d), wq.t()),
            torch.mm(_exact_runs(x.t()), _exact_runs(d.t()).t()))


def _exact_fp8(c, s):
    x = s["x"]
    if not c["train"]:
        e = s["scales"].double().repeat_interleave(BLOCK, 1)[:, :s["codes"].shape[1]] - 127
        w = s["codes"].view(torch.float8_e4m3fn).double() * torch.exp2(e)
        return dict(y=_exact_runs(x) @ w[:, :c["k"]].t())
    w, d = s["w"], s["d"]
    stack = w if w.dim() == 3 else w.unsqueeze(0)
    step = [_exact_step(x[a:b], stack[i], d[a:b])
            for i, (a, b) in enumerate(zip(s["cuts"][:-1], s["cuts"][1:]))]
    y, dx, dw = zip(*step)
    return dict(y=torch.cat(y), dx=torch.cat(dx), dw=torch.stack(dw) if w.dim() == 3 else dw[0])


def _exact_clip(c, s):
    g = torch.cat([t.double() for t in s["grads"]])
    norm = g.norm()
    return dict(norm=norm, grads=g * torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, exchange=_exact_exchange, fp8=_exact_fp8,
                clip=_exact_clip)[case["op"]](case, s)
