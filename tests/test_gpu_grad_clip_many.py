"""The gradient norm and clipping over thousands of tensors (many launches),
and at the edges of norm, max_norm and eps."""

import numpy as np
import pytest
import torch

from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [128, 129, 256, 257, 5000])
def test_many_tensors(n):
    """Around the number of tensors of one launch, and thousands; tolerances as
    for few tensors (2^-23 of the norm, 1.01 x 2^-24 + 2^-23 of a value)."""
    rng = np.random.default_rng(n)
    sizes = rng.integers(0, 3000, n).tolist()
    flat = torch.from_numpy(rng.standard_normal(sum(sizes)).astype(np.float32)).cuda()
    ref = flat.double().cpu().numpy()
    norm = np.sqrt(np.sum(ref ** 2))
    out = torch.full_like(flat, 9.0)
    n1 = av.averis_grad_clip(list(flat.split(sizes)), 1.0, out=list(out.split(sizes)))
    assert abs(float(n1) - norm) <= 2.0 ** -23 * norm
    assert torch.equal(n1, av.averis_grad_norm(list(flat.split(sizes))))
    ref = ref / (norm + 1e-6)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= (1.01 * 2.0 ** -24 + 2.0 ** -23) * np.abs(ref))
    av.averis_grad_clip(list(flat.split(sizes)), 1.0)      # in place
    assert torch.equal(flat, out)


def test_clipping_grows_with_the_data_alone():
    """The norm reads the gradients once; the clipped ones read them twice more and
    write them, so that 2.7 times the norm's time is what many tensors take.
    Were the norm formed from all the partial sums by every workgroup, it would
    be 14 times at this size.  Replays of a graph: device time alone."""
    n, size = 12000, 131072
    flat = torch.ones(n * size, device="cuda")
    grads = list(flat.split(size))
    ws = torch.empty(av.workspace_bytes(av.OP_GRAD_NORM, 0, 0, n), dtype=torch.uint8, device="cuda")
    times = []
    for call in (lambda: av.averis_grad_norm(grads, ws=ws), lambda: av.averis_grad_clip(grads, 1.0, ws=ws)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        best = float("inf")
        for _ in range(4):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            graph.replay()
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end))
        times.append(best)
    assert times[1] < 6.0 * times[0], times


@pytest.mark.parametrize("n", [1, 200])
def test_zero_gradients_without_eps(n):
    """0 / 0 is no factor: gradients of zero stay zero."""
    for max_norm in (0.0, 1.0, float("inf")):
        grads = [torch.zeros(1000, device="cuda") for _ in range(n)]
        out = [torch.full_like(g, 9.0) for g in grads]
        assert float(av.averis_grad_clip(grads, max_norm, eps=0.0, out=out)) == 0.0
        assert all(bool((o == 0).all()) for o in out)
        av.averis_grad_clip(grads, max_norm, eps=0.0)
        assert all(bool((g == 0).all()) for g in grads)


@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e6])
@pytest.mark.parametrize("value", [3e38, 1.7e35, 1e20])
def test_factors_below_fp32s_normal_numbers(value, max_norm):
    """Norms up to 2^138: the factor, under 2^-126 for the largest, keeps its 24
    bits (2^-23 with the product's rounding; the norm's own is 2^-53)."""
    n = 1 << 20
    g = torch.full((n,), value, device="cuda")
    g[1::2] *= 2.0 ** -20
    ref = g.double().cpu().numpy()
    ref = ref * (max_norm / (np.sqrt(np.sum(ref ** 2)) + 1e-6))
    out = torch.empty_like(g)
    av.averis_grad_clip([g], max_norm, out=[out])
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= 1.01 * 2.0 ** -23 * np.abs(ref))
    b = g.to(torch.bfloat16)
    ref = b.double().cpu().numpy()
    ref = ref * (max_norm / (np.sqrt(np.sum(ref ** 2)) + 1e-6))
    av.averis_grad_clip([b], max_norm)
    assert np.all(np.abs(b.double().cpu().numpy() - ref) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref))
