"""The global gradient norm and clipping on the GPU against float64.

Tolerances: the norm's fp64 sums are exact to n 2^-53, its rounding to fp32 is
2^-24 relative; a clipped value has the factor's rounding and its own (2^-24
each in fp32; at most 2^-8 in bf16 after an fp32 product)."""

import numpy as np
import pytest
import torch

from oracle import moe
from tests.parity import BF16_REL
from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()


def make(sizes, dtypes, scale, lead=0):
    """Tensors one after the other in one buffer a type: odd starts."""
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    out = []
    for dt in dtypes:
        n = sum(s for s, d in zip(sizes, _cycle(dtypes, len(sizes))) if d == dt) + lead
        out.append((dt, (torch.randn(n, generator=gen, device="cuda") * scale).to(dt)))
    at = {dt: lead for dt in dtypes}
    grads = []
    for s, dt in zip(sizes, _cycle(dtypes, len(sizes))):
        flat = dict(out)[dt]
        grads.append(flat[at[dt]:at[dt] + s])
        at[dt] += s
    return grads


def _cycle(v, n):
    return [v[i % len(v)] for i in range(n)]


SIZES = [[1], [7], [8192], [16385, 3], [1, 0, 5, 100000, 17], [0, 0], [250] * 300,
         [1 << 20, 1, 1 << 18, 12345, 999999]]


@pytest.mark.parametrize("dtypes", [[F32], [BF16], [F32, BF16]])
@pytest.mark.parametrize("case", range(len(SIZES)))
@pytest.mark.parametrize("max_norm", [1.0, 1e9])
def test_norm_and_clip(case, dtypes, max_norm):
    sizes = SIZES[case]
    grads = make(sizes, dtypes, 0.5, lead=case % 3)
    before = [g.clone() for g in grads]
    norm, ref = moe.grad_clip([g.double().cpu().numpy() for g in grads], max_norm, 1e-6)
    n1 = av.averis_grad_norm(grads)
    assert abs(float(n1) - norm) <= 2.0 ** -23 * norm
    out = [torch.full_like(g, 9.0) for g in grads]
    n2 = av.averis_grad_clip(grads, max_norm, out=out)
    assert torch.equal(n1, n2)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))   # inputs untouched
    for g, o, r in zip(grads, out, ref):
        half = BF16_REL if g.dtype == BF16 else 2.0 ** -24
        if r.size:
            assert np.all(np.abs(o.double().cpu().numpy() - r) <= (1.01 * half + 2.0 ** -23) * np.abs(r))
    n3 = av.averis_grad_clip(grads, max_norm)                       # in place
    assert torch.equal(n3, n1)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))


def test_neighbours_are_untouched():
    buf = torch.full((5000,), 2.0, device="cuda", dtype=BF16)
    g = buf[3:4500]
    av.averis_grad_clip([g], 1.0)
    assert (buf[:3] == 2).all() and (buf[4500:] == 2).all() and (g != 2).all()


def test_large_and_small_values():
    """Squares outside fp32's range: the sums are fp64."""
    for v in (1e30, 1e-30):
        g = torch.full((10000,), v, device="cuda")
        n = float(av.averis_grad_norm([g]))
        ref = 100.0 * float(g[0].double())
        assert abs(n - ref) <= 2.0 ** -23 * ref
    g = torch.full((4,), 3e38, device="cuda")     # a norm past fp32's range
    out = torch.empty_like(g)
    n = av.averis_grad_clip([g], 1.0, out=[out])
    assert torch.isinf(n)
    np.testing.assert_allclose(out.cpu().numpy(), 0.5, rtol=1e-6)


def test_values_that_are_not_finite():
    g = torch.ones(100, device="cuda")
    g[7] = float("inf")
    n = av.averis_grad_clip([g], 1.0)
    assert torch.isinf(n) and torch.isnan(g[7]) and (g[:7] == 0).all()
    g = torch.ones(100, device="cuda")
    g[3] = float("nan")
    n = av.averis_grad_clip([g], 1.0)
    assert torch.isnan(n) and torch.isnan(g).all()


def test_zero_gradients_and_zero_max_norm():
    g = torch.zeros(1000, device="cuda")
    assert float(av.averis_grad_clip([g], 1.0)) == 0.0 and (g == 0).all()
    g = torch.ones(1000, device="cuda")
    av.averis_grad_clip([g], 0.0)
    assert (g == 0).all()
    assert float(av.averis_grad_norm([])) == 0.0


def test_same_bits_and_graph_replay():
    grads = make([100001] * 40, [F32, BF16], 1.0)
    out = [torch.empty_like(g) for g in grads]
    n0 = av.averis_grad_clip(grads, 1.0, out=out).clone()
    ref = [o.clone() for o in out]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = av.averis_grad_clip(grads, 1.0, out=out)
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, n0) and all(torch.equal(a, b) for a, b in zip(out, ref))
        av.averis_grad_norm(out)


def test_tensor_past_2_31_elements():
    n = (1 << 31) + 12345
    g = torch.zeros(n, device="cuda", dtype=BF16)
    g[-1] = 3.0
    g[0] = 4.0
    assert float(av.averis_grad_clip([g], 1.0, eps=0.0)) == 5.0
    assert abs(float(g[-1]) - 0.6) < 0.002 and abs(float(g[0]) - 0.8) < 0.002
