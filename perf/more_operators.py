"""What the operators around a block's linears cost, and what they have to compute.

Four groups of cases:

* ``norm``    root-mean-square norm with the residual's addition and an output in 8 bits with a power-of-two
              scale for each 128 (rows, and the transposed copy that the weight gradient takes); its gradient;
* ``linear``  8-bit products with bias, activation and residual: dense, by expert segment, single tokens;
* ``act``     the way back through a linear's activation and bias: the gradient before the activation in 8 bits,
              both copies, and the bias's gradient;
* ``route``   experts of each token by softmax or sigmoid scores, with a bias for balance and groups of experts;
              the logits' gradient.

``run`` computes a case in plain torch operations (``own`` false) or with the package's entry points.
"""

import math

import torch

own = False

BLOCK = 128          # elements that share a scale
E4M3_MAX = 448.0
EPS = 1e-6
SCALE = 2.5          # of the router's weights
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715   # gelu(x) = x sigmoid(A (x + B x^3))


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one batch of single tokens in serving: latency alone; the router reads the norm's output too
        dict(name="norm 16 tokens", op="norm", rows=16, cols=2048, dtype="bf16", residual=True,
             y=True, train=False),
        # a training batch of the mixture-of-experts hidden size: both copies for the linear, and the gradient
        dict(name="norm 32768 tokens", op="norm", rows=32768, cols=2048, dtype="bf16", residual=True,
             y=False, train=True),
        # odd sizes in fp32, no residual: a block's first norm
        dict(name="norm ragged fp32", op="norm", rows=2999, cols=1000, dtype="f32", residual=False,
             y=True, train=True),
        # single tokens through an up-projection whose weight is kept in 8 bits
        dict(name="linear 16 tokens", op="linear", rows=16, k=2048, n=1024, experts=1, act="gelu",
             bias=True, residual=False, save=False),
        # a training batch's up-projection: bias and activation, the value before it kept for the gradient
        dict(name="linear up 16384 tokens", op="linear", rows=16384, k=1024, n=4096, experts=1,
             act="gelu", bias=True, residual=False, save=True),
        # its down-projection, back onto the residual stream
        dict(name="linear down 16384 tokens", op="linear", rows=16384, k=4096, n=1024, experts=1,
             act="none", bias=True, residual=True, save=False),
        # the mixture-of-experts linear with each expert's own bias
        dict(name="linear 64 experts", op="linear", rows=32768, k=2048, n=768, experts=64, act="silu",
             bias=True, residual=False, save=True),
        # back through the up-projection's activation
        dict(name="act 16384 tokens", op="act", rows=16384, n=4096, experts=1, act="gelu", dtype="bf16"),
        # back through the experts' activations, a bias gradient for each
        dict(name="act 64 experts", op="act", rows=32768, n=768, experts=64, act="silu", dtype="bf16"),
        # one batch of single tokens: latency alone
        dict(name="route 16 tokens", op="route", tokens=16, experts=64, topk=8, groups=8, topk_groups=4,
             score="sigmoid", bias=True, renorm=True, dtype="bf16", masked=0.0, train=False),
        # a long batch over many experts, some closed to a token, padding closed to all, with the gradient
        dict(name="route 65521 tokens", op="route", tokens=65521, experts=256, topk=8, groups=8,
             topk_groups=4, score="sigmoid", bias=True, renorm=True, dtype="f32", masked=0.2, train=True),
        # groups of twenty, softmax scores without renormalisation, the best expert of a group its score
        dict(name="route odd groups", op="route", tokens=10007, experts=160, topk=6, groups=8, topk_groups=3,
             score="softmax", bias=False, renorm=False, dtype="bf16", masked=0.0, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "act", "route"])
    if op == "norm":
        cols = _log(rng, 64, 8192)
        return dict(op=op, rows=_log(rng, 1, min(65536, (1 << 25) // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]), residual=rng.random() < 0.7,
                    y=rng.random() < 0.5, train=rng.random() < 0.5)
    if op == "linear" and rng.random() < 0.4:
        return dict(op=op, rows=_log(rng, 1, 512), k=_log(rng, 64, 4096), n=_log(rng, 64, 8192), experts=1,
                    act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.7,
                    residual=rng.random() < 0.5, save=False)
    if op == "linear":
        k, n = _log(rng, 64, 4096), _log(rng, 64, 4096)
        experts = rng.choice([1, 1, _log(rng, 2, max(2, min(64, 100_000_000 // (k * n))))])
        return dict(op=op, rows=_log(rng, 512, min(32768, max(1024, 60_000_000_000 // (k * n)))), k=k, n=n,
                    experts=experts, act=rng.choice(["none", "relu", "silu", "gelu"]),
                    bias=rng.random() < 0.7, residual=rng.random() < 0.5, save=rng.random() < 0.5)
    if op == "act":
        n = _log(rng, 64, 8192)
        return dict(op=op, rows=_log(rng, 1, min(65536, (1 << 26) // n)), n=n,
                    experts=rng.choice([1, 1, _log(rng, 2, 128)]),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), dtype=rng.choice(["bf16", "f32"]))
    groups = rng.choice([1, 2, 4, 8, 16, rng.randint(1, 12)])
    experts = groups * _log(rng, 2, max(2, 384 // groups))
    topk_groups = rng.randint(1, groups)
    return dict(op=op, tokens=_log(rng, 1, 65536), experts=experts,
                topk=rng.randint(1, min(8, topk_groups * (experts // groups))), groups=groups,
                topk_groups=topk_groups, score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6,
                renorm=rng.random() < 0.6, dtype=rng.choice(["bf16", "f32"]),
                masked=rng.choice([0.0, 0.3]), train=rng.random() < 0.5)


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def work(c):
    if c["op"] == "norm":
        e, s = c["rows"] * c["cols"], _size(c["dtype"])
        # x (and the residual in, their sum out), codes and scales, y where it is wanted
        b, f = e * s * (3 if c["residual"] else 1) + e + e // BLOCK + (e * s if c["y"] else 0), 5 * e
        if c["train"]:
            # the transposed copy; the gradients of y and of the sum in, the sum, its gradient out
            b, f = b + e + e // BLOCK + 4 * e * s, f + 9 * e
        return dict(bytes=b + 4 * c["cols"], flops=f)
    if c["op"] == "linear":
        m, k, n = c["rows"], c["k"], c["n"]
        b = m * k + c["experts"] * n * k + 2 * m * n * (1 + c["residual"] + c["save"])
        return dict(bytes=b, flops=2 * m * n * k)
    if c["op"] == "act":
        e, s = c["rows"] * c["n"], _size(c["dtype"])
        return dict(bytes=e * s * (1 if c["act"] == "none" else 2) + 2 * e + e // 64 + 4 * c["experts"] * c["n"],
                    flops=12 * e)
    t, e, k, s = c["tokens"], c["experts"], c["topk"], _size(c["dtype"])
    b, f = t * e * s + 8 * t * k, 10 * t * e
    if c["train"]:
        # the weights' gradient in, the logits' out; of the logits the chosen ones, or all where all count
        b, f = b + 4 * t * k + t * e * s, f + 10 * t * k
    return dict(bytes=b, flops=f)


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
    x += 0.6 * _randn(g, cols)
    x += _randn(g, rows, 1) * _randn(g, cols) * (4.0 / math.sqrt(cols))
    return x


def _cuts(g, rows, experts):
    """Row counts of experts whose popularity falls off as a power law; some get none."""
    p = torch.arange(1, experts + 1, device="cuda").double().pow(-1.1)
    p = p[torch.randperm(experts, generator=g, device="cuda")]
    cuts = torch.round(torch.cumsum(p / p.sum(), 0) * rows).long()
    cuts[-1] = rows
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), cuts])


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "norm":
        r, n, dt = c["rows"], c["cols"], _dtype(c["dtype"])
        s = dict(case=c, x=_biased(g, r, n).to(dt), weight=1.0 + 0.2 * _randn(g, n),
                 res=(2.0 * _randn(g, r, n)).to(dt) if c["residual"] else None)
        if c["train"]:
            s.update(dy=(_randn(g, r, n) * 1e-2 + 3e-3 * _randn(g, n)).to(dt),
                     dres=(_randn(g, r, n) * 1e-2).to(dt) if c["residual"] else None)
        return s
    if c["op"] == "linear":
        m, k, n, e = c["rows"], c["k"], c["n"], c["experts"]
        # the activation as the operator before it left it, the weight (its transpose, one scale to a
        # 128 x 128 tile) as a program keeps it: codes, and scale rows padded to whole words
        x = _run_codes(_biased(g, m, k).to(torch.bfloat16))
        w = [_tile_codes(_randn(g, n, k) / math.sqrt(k)) for _ in range(e)]
        offs = _cuts(g, m, e) if e > 1 else None
        return dict(case=c, xc=x[0], xs=_padded(x[1], 1, 4).contiguous(), wc=torch.cat([v[0] for v in w]),
                    ws=torch.cat([v[1] for v in w]), offsets=offs, cuts=offs.tolist() if e > 1 else [0, m],
                    bias=0.3 * _randn(g, e, n) if c["bias"] else None,
                    res=_biased(g, m, n).to(torch.bfloat16) if c["residual"] else None)
    if c["op"] == "act":
        m, n, e, dt = c["rows"], c["n"], c["experts"], _dtype(c["dtype"])
        offs = _cuts(g, m, e) if e > 1 else None
        return dict(case=c, dy=(1e-2 * _randn(g, m, n) + 5e-3 * _randn(g, n)).to(dt),
                    z=(1.5 * _biased(g, m, n)).to(dt) if c["act"] != "none" else None,
                    offsets=offs, cuts=offs.tolist() if e > 1 else [0, m])
    t, e = c["tokens"], c["experts"]
    logits = _randn(g, t, e) * 1.5 - 1.1 * torch.log(1.0 + torch.arange(e, device="cuda")[torch.randperm(e, generator=g, device="cuda")])
    if c["masked"]:
        # experts closed to a token, and tokens (padding) closed to all of them
        logits[torch.rand(t, e, generator=g, device="cuda") < c["masked"]] = -math.inf
        logits[torch.rand(t, generator=g, device="cuda") < 0.05] = -math.inf
    # a bias as its updates leave it: whole steps of a thousandth
    bias = torch.round(60.0 * _randn(g, e)) * 1e-3 if c["bias"] else None
    return dict(case=c, logits=logits.to(_dtype(c["dtype"])), bias=bias, dweights=_randn(g, t, c["topk"]))


# --------------------------------------------------------------------------
# the operators in plain form: fp32, rounded once
# --------------------------------------------------------------------------

def _powers(amax):
    """The smallest 2^e with amax <= 448 * 2^e, at least 2^-127."""
    m, x = torch.frexp(amax)            # amax = m 2^x, m in [0.5, 1); 448 = 0.875 2^9
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax == 0, torch.full_like(e, -127), e).clamp(min=-127)


def _padded(a, rows, cols):
    return torch.nn.functional.pad(a, (0, -a.shape[1] % cols, 0, -a.shape[0] % rows))


def _coded(t, e):
    e = e.float()
    return (t * torch.exp2(-torch.floor(e / 2)) * torch.exp2(-torch.ceil(e / 2))).to(torch.float8_e4m3fn)


def _run_codes(a):
    """Codes (rows padded to whole blocks) and scale bytes of `a`, a scale for each run of 128 along the columns."""
    r, k = a.shape
    b = _padded(a.float(), 1, BLOCK).reshape(r, -(-k // BLOCK), BLOCK)
    e = _powers(b.abs().amax(2, keepdim=True))
    return _coded(b, e).view(torch.uint8).flatten(1), (e + 127).to(torch.uint8)[:, :, 0]


def _tile_codes(w):
    """The same with one scale for each 128 x 128 tile, scale rows padded to whole words."""
    n, k = w.shape
    b = _padded(w.float(), BLOCK, BLOCK)
    b = b.reshape(b.shape[0] // BLOCK, BLOCK, b.shape[1] // BLOCK, BLOCK)
    e = _powers(b.abs().amax((1, 3), keepdim=True))
    codes = _coded(b, e).view(torch.uint8).reshape(b.shape[0] * BLOCK, -1)[:n]
    scales = (e + 127).to(torch.uint8).expand(-1, BLOCK, -1, -1).reshape(b.shape[0] * BLOCK, -1)[:n]
    return codes.contiguous(), _padded(scales, 1, 4).contiguous()


def _values(codes, scales):
    """What codes and scale bytes stand for."""
    s = torch.exp2(scales.float() - 127)[:, :codes.shape[1] // BLOCK]
    v = codes.view(torch.float8_e4m3fn).float().reshape(codes.shape[0], -1, BLOCK)
    return (v * s[:, :, None]).flatten(1)


def _stands(codes, scales):
    """Codes and scale bytes as numbers of their types."""
    return dict(codes=codes.view(torch.float8_e4m3fn), scales=scales.view(torch.float8_e8m0fnu))


def _runs(cuts):
    """Lengths of the segments' parts of a transposed copy: whole runs of 128."""
    return [-(-(b - a) // BLOCK) * BLOCK for a, b in zip(cuts, cuts[1:])]


def _by_segment(a, cuts):
    """The rows of each segment from a multiple of 128 on, zeros between them."""
    return torch.cat([torch.nn.functional.pad(a[r:s], (0, 0, 0, n - (s - r)))
                      for r, s, n in zip(cuts, cuts[1:], _runs(cuts))])


def _normed(s):
    c, x, w = s["case"], s["x"], s["weight"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(x.dtype)
    # the sum in 64 bits: whether a value is past the middle between two codes must not hang on its order
    var = h.double().square().sum(1, keepdim=True) / c["cols"]
    rstd = (1.0 / torch.sqrt(var + EPS)).float()
    xh = h.float() * rstd
    y = (xh * w).to(x.dtype)
    r = dict(h=h, q=_stands(*_run_codes(y)))
    if c["y"]:
        r["y"] = y
    if c["train"]:
        r["qt"] = _stands(*_run_codes(y.t()))
        dy = s["dy"].float()
        wdy = dy * w
        dh = rstd * (wdy - xh * (wdy * xh).mean(1, keepdim=True))
        r["dh"] = (dh if s["dres"] is None else dh + s["dres"].float()).to(x.dtype)
        r["dweight"] = (dy * xh).sum(0)
    return r


def _sigmoid(u):
    return 1.0 / (1.0 + torch.exp(-u))


def _activated(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    return z * _sigmoid(z if act == "silu" else GELU_A * (z + GELU_B * z * z * z))


def _slope(z, act):
    if act == "relu":
        return torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    s = _sigmoid(z if act == "silu" else GELU_A * (z + GELU_B * z * z * z))
    return s + z * s * (1.0 - s) * (1.0 if act == "silu" else GELU_A * (1.0 + 3.0 * GELU_B * z * z))


def _linear(s):
    c, cuts, n, k = s["case"], s["cuts"], s["case"]["n"], s["case"]["k"]
    x, w = _values(s["xc"], s["xs"])[:, :k], _values(s["wc"], s["ws"])[:, :k]
    z = torch.cat([x[a:b] @ w[i * n:(i + 1) * n].t() + (0.0 if s["bias"] is None else s["bias"][i])
                   for i, (a, b) in enumerate(zip(cuts, cuts[1:]))])
    y = _activated(z, c["act"])
    r = dict(y=(y if s["res"] is None else y + s["res"].float()).to(torch.bfloat16))
    if c["save"]:
        r["z"] = z.to(torch.bfloat16)
    return r


def _act_gradient(s):
    dy, cuts = s["dy"], s["cuts"]
    dz = dy.float() if s["z"] is None else dy.float() * _slope(s["z"].float(), s["case"]["act"])
    t = dz.to(dy.dtype)
    return dict(q=_stands(*_run_codes(t)), qt=_stands(*_run_codes(_by_segment(t, cuts).t())),
                dbias=torch.stack([dz[a:b].sum(0) for a, b in zip(cuts, cuts[1:])]))


def _scored(l, score):
    """Scores in l's precision; 0 where an expert is closed."""
    if score == "sigmoid":
        return _sigmoid(l)
    top = l.max(1, keepdim=True).values
    z = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = z.sum(1, keepdim=True)
    return z / torch.where(total == 0, torch.ones_like(total), total)


def _chosen(s):
    """Experts of each token, -1 where none is left; in 64 bits, for equal and nearly equal scores."""
    c, l = s["case"], s["logits"].double()
    t, e = l.shape
    closed = l == -math.inf
    key = _scored(l, c["score"])
    if s["bias"] is not None:
        key = key + s["bias"].double()
    key = torch.where(closed, torch.full_like(key, -math.inf), key)
    if c["topk_groups"] < c["groups"]:
        g = torch.sort(key.reshape(t, c["groups"], -1), dim=2, descending=True).values[:, :, :_group_top(c)]
        total = torch.where(g == -math.inf, torch.zeros_like(g), g).sum(2)
        total = torch.where(g[:, :, 0] == -math.inf, torch.full_like(total, -math.inf), total)
        best = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        kept = torch.zeros_like(total, dtype=torch.bool).scatter_(1, best, True)
        key = torch.where(kept.repeat_interleave(e // c["groups"], 1), key, torch.full_like(key, -math.inf))
    top, at = torch.sort(key, dim=1, descending=True, stable=True)
    at = torch.where(top == -math.inf, torch.full_like(at, -1), at)
    return at[:, :c["topk"]].int()


def _group_top(c):
    """How many of a group's experts make its score: two where a bias moves them, else the best."""
    return 2 if c["bias"] else 1


def _routed(s):
    c, l, ids = s["case"], s["logits"].float(), _chosen(s)
    open_, at = ids >= 0, ids.clamp(min=0).long()
    p = _scored(l, c["score"])
    v = torch.where(open_, torch.gather(p, 1, at), torch.zeros_like(s["dweights"]))
    total = v.sum(1, keepdim=True)
    total = torch.where(total == 0, torch.ones_like(total), total)
    w = v / total if c["renorm"] else v
    r = dict(ids=ids, weights=SCALE * w)
    if c["train"]:
        d = torch.where(open_, SCALE * s["dweights"], torch.zeros_like(v))
        if c["renorm"]:
            d = (d - (w * d).sum(1, keepdim=True)) / total
        d = torch.where(open_, d, torch.zeros_like(d))
        if c["score"] == "sigmoid":
            dl = torch.zeros_like(p).scatter_add_(1, at, d * v * (1.0 - v))
        else:
            dl = (-(d * v).sum(1, keepdim=True) * p).scatter_add_(1, at, d * v)
        r["dlogits"] = dl.to(s["logits"].dtype)
    return r


def _plain(s):
    return dict(norm=_normed, linear=_linear, act=_act_gradient, route=_routed)[s["case"]["op"]](s)


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------

def _own_codes(q, cols):
    """What a call wrote: without the room behind the last segment and the padding of the scales."""
    blocks = -(-cols // BLOCK)
    return _stands(q.codes[:, :blocks * BLOCK], q.scales[:, :blocks])


def _own(s):
    from mean_residual_quantized_amd import averis as av

    c = s["case"]
    if c["op"] == "norm":
        h, rstd, y, q, qt = av.averis_rmsnorm(s["x"], s["weight"], eps=EPS, residual=s["res"], y=c["y"],
                                              transposed=c["train"])
        r = dict(h=h, q=_own_codes(q, c["cols"]))
        if c["y"]:
            r["y"] = y
        if c["train"]:
            r["qt"] = _own_codes(qt, c["rows"])
            r["dh"], r["dweight"] = av.averis_rmsnorm_grad(s["dy"], h, s["weight"], rstd, dres=s["dres"])
        return r
    if c["op"] == "linear":
        x = av.FP8(s["xc"], s["xs"], c["rows"], c["k"])
        w = av.FP8(s["wc"], s["ws"], c["experts"] * c["n"], c["k"])
        bias = s["bias"] if s["bias"] is None or c["experts"] > 1 else s["bias"][0]
        r = av.averis_fp8_gemm_act(x, w, bias=bias, act=c["act"], residual=s["res"], save=c["save"],
                                   out_dtype=torch.bfloat16, offsets=s["offsets"])
        return dict(y=r[0], z=r[1]) if c["save"] else dict(y=r)
    if c["op"] == "act":
        q, qt, db = av.averis_fp8_act_grad(s["dy"], z=s["z"], act=c["act"], offsets=s["offsets"])
        return dict(q=_own_codes(q, c["n"]), qt=_own_codes(qt, sum(_runs(s["cuts"]))),
                    dbias=db if c["experts"] > 1 else db[None])
    ids, w = av.averis_moe_route_groups(s["logits"], c["topk"], bias=s["bias"], score=c["score"],
                                        groups=c["groups"], topk_groups=c["topk_groups"],
                                        group_top=_group_top(c), renorm=c["renorm"], scale=SCALE)
    r = dict(ids=ids, weights=w)
    if c["train"]:
        r["dlogits"] = av.averis_moe_route_groups_grad(s["logits"], ids, s["dweights"], score=c["score"],
                                                       renorm=c["renorm"], scale=SCALE)
    return r


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_quantized(a):
    """Codes' values and scales of `a` (float64) on the grid of each run's scale."""
    p = torch.nn.functional.pad(a, (0, -a.shape[1] % BLOCK))
    p = p.unflatten(1, (-1, BLOCK))
    m = p.abs().amax(2).clamp(min=1e-300)
    e = torch.ceil(torch.log2(m / E4M3_MAX))
    e = torch.where(m <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)   # log2 is inexact at powers of two
    e = torch.where(m > E4M3_MAX * torch.exp2(e), e + 1, e).clamp(min=-127)
    v = p / torch.exp2(e)[:, :, None]
    # spacing of E4M3 at |v|: 2^(floor(log2 |v|) - 3), at least 2^-9
    step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
    return dict(codes=(torch.round(v / step) * step).flatten(1), scales=torch.exp2(e))


def _exact_norm(c, s):
    x = s["x"].double()
    # (the residual stream is held in its type: the norm is of what is stored)
    h = x if s["res"] is None else (x + s["res"].double()).to(s["x"].dtype).double()
    w = s["weight"].double()
    scale = torch.rsqrt(h.pow(2).mean(1) + EPS)[:, None]
    y = h * scale * w
    held = y.to(s["x"].dtype).double()   # (the codes are of y in its type)
    r = dict(h=h, q=_exact_quantized(held))
    if c["y"]:
        r["y"] = y
    if c["train"]:
        r["qt"] = _exact_quantized(held.t())
        dy = s["dy"].double()
        # y = w h scale(h): d scale / d h_j = -scale^3 h_j / n
        dot = (dy * w * h).sum(1, keepdim=True)
        dh = scale * w * dy - scale ** 3 * dot * h / c["cols"]
        r["dh"] = dh if s["dres"] is None else dh + s["dres"].double()
        r["dweight"] = torch.einsum("rc,rc->c", dy, h * scale)
    return r


def _exact_values(codes, scales, k):
    f = torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)[:, :k]
    return codes.view(torch.float8_e4m3fn)[:, :k].double() * f


def _exact_linear(c, s):
    n, k = c["n"], c["k"]
    x, w = _exact_values(s["xc"], s["xs"], k), _exact_values(s["wc"], s["ws"], k)
    z = torch.zeros(c["rows"], n, dtype=torch.float64, device=x.device)
    for i, (a, b) in enumerate(zip(s["cuts"][:-1], s["cuts"][1:])):
        torch.mm(x[a:b], w[i * n:(i + 1) * n].t(), out=z[a:b])
        if s["bias"] is not None:
            z[a:b] += s["bias"][i].double()
    y = z
    if c["act"] == "relu":
        y = z.clamp(min=0.0)
    elif c["act"] == "silu":
        y = z * torch.sigmoid(z)
    elif c["act"] == "gelu":
        y = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    r = dict(y=y if s["res"] is None else y + s["res"].double())
    if c["save"]:
        r["z"] = z
    return r


def _exact_act(c, s):
    dz = s["dy"].double()
    if c["act"] != "none":
        z = s["z"].double()
        if c["act"] == "relu":
            dz = dz * (z > 0)
        elif c["act"] == "silu":
            p = torch.sigmoid(z)
            dz = dz * (p + z * p * torch.sigmoid(-z))
        else:
            a = math.sqrt(2.0 / math.pi)
            t = torch.tanh(a * (z + 0.044715 * z ** 3))
            dz = dz * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z))
    parts = list(torch.split(dz, [b - a for a, b in zip(s["cuts"][:-1], s["cuts"][1:])]))
    held = [p.to(s["dy"].dtype).double() for p in parts]   # (the codes are of dz in dy's type)
    whole = torch.cat([torch.nn.functional.pad(p, (0, 0, 0, -p.shape[0] % BLOCK)) for p in held])
    return dict(q=_exact_quantized(torch.cat(held)), qt=_exact_quantized(whole.t()),
                dbias=torch.stack([p.sum(0) for p in parts]))


def _exact_route(c, s):
    l, k = s["logits"].double(), c["topk"]
    t, e = l.shape
    shut = torch.isneginf(l)
    p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    rank = (p if s["bias"] is None else p + s["bias"].double()).masked_fill(shut, -math.inf)
    if c["topk_groups"] < c["groups"]:
        per = e // c["groups"]
        v = rank.view(t, c["groups"], per)
        best = v.topk(min(_group_top(c), per), dim=2).values
        g = best.masked_fill(torch.isneginf(best), 0.0).sum(2).masked_fill(torch.isneginf(best[:, :, 0]), -math.inf)
        order = torch.argsort(g, dim=1, descending=True, stable=True)
        place = torch.argsort(order, dim=1)
        rank = v.masked_fill((place >= c["topk_groups"])[:, :, None], -math.inf).reshape(t, e)
    ids = torch.argsort(rank, dim=1, descending=True, stable=True)[:, :k]
    taken = torch.zeros_like(l).scatter_(1, ids, 1.0) * ~torch.isneginf(rank)
    v = p * taken
    norm = v.sum(1, keepdim=True).clamp(min=1e-300) if c["renorm"] else torch.ones_like(v[:, :1])
    r = dict(ids=None, weights=SCALE * torch.gather(v / norm, 1, ids))
    if c["train"]:
        d = SCALE * torch.zeros_like(l).scatter_(1, ids, s["dweights"].double()) * taken / norm
        if c["renorm"]:
            d = taken * (d - (d * v).sum(1, keepdim=True) / norm)
        if c["score"] == "sigmoid":
            r["dlogits"] = d * p * torch.sigmoid(-l).masked_fill(shut, 0.0)
        else:
            r["dlogits"] = p * (d - (d * p).sum(1, keepdim=True))
    return r


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, linear=_exact_linear, act=_exact_act, route=_exact_route)[case["op"]](case, s)
