"""Token counts whose threads do not fit one launch (a grid has fewer than 2^32
of them), up to the 2^31 - 1 slots that the calls take: what each call gives at
its first and last tokens, and that none is left out."""

import pytest
import torch

from mean_residual_quantized_amd import averis as av

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    av.lib()
    yield
    torch.cuda.empty_cache()


def every(*conditions):
    """(Outside assert statements, whose failure would list the tensors.)"""
    ok = [bool(c.all()) for c in conditions]
    assert all(ok), ok


def same(a, b):
    every(a == b)


def reversed_rows(tokens, topk):
    n = tokens * topk
    return torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda").reshape(tokens, topk)


def test_router():
    """Eight lanes a token: 2^29 tokens and more."""
    t, last = (1 << 29) + 1000, 1500
    l = torch.zeros(t, 2, dtype=BF16, device="cuda")
    l[-last:, 1] = 2.0
    ids, w = av.averis_moe_route(l, 1, renorm=False)
    every(ids[:-last] == 0, ids[-last:] == 1)
    p = torch.softmax(torch.tensor([0.0, 2.0], dtype=torch.float64), 0)
    every(w[:-last] == 0.5)
    every((w[-last:].double() - float(p[1])).abs() < 1e-6)
    w.fill_(1.0)
    d = av.averis_moe_route_grad(l, ids, w, renorm=False, out=l)   # in place
    # p_0 p_1 at the chosen expert, minus it at the other
    for rows, chosen, g in ((d[:-last], 0, 0.25), (d[-last:], 1, float(p[0] * p[1]))):
        every((rows[:, chosen].float() - g).abs() <= 2.0 ** -8 * g)
        every(rows[:, 1 - chosen] == -rows[:, chosen])


def test_combine_gradient():
    """64 lanes a slot: 2^26 slots and more.  Small integers: exact."""
    t, k = (1 << 23) + 5, 8
    pos = reversed_rows(t, k)
    rows = (torch.arange(t * k, device="cuda") % 97).to(BF16).reshape(-1, 1)
    dy = (torch.arange(t, device="cuda") % 31 + 1).to(BF16).reshape(-1, 1)
    w = (torch.arange(t * k, device="cuda") % 4 + 1).float().reshape(t, k)
    drows, dw = av.averis_moe_combine_grad(dy, rows, pos, w)
    same(dw, (dy.float() * rows.flip(0).float().reshape(t, k)))
    same(drows.flip(0).reshape(t, k), (w * dy.float()).to(BF16))


def test_exchange_of_narrow_rows():
    """16 lanes' worth of threads a token along the grid: 2^28 tokens and more."""
    t = (1 << 28) + 7
    pos = reversed_rows(t, 1)
    x = (torch.arange(t, device="cuda") % 251 + 1).to(BF16).reshape(-1, 1)
    rows = av.averis_moe_dispatch(x, pos)
    same(rows, x.flip(0))
    y = av.averis_moe_combine(rows, pos)
    same(y, x)
    y = av.averis_moe_combine(rows, pos, torch.full((t, 1), 2.0, device="cuda"))
    same(y, 2 * x)


def test_exchange_of_wide_rows():
    """A workgroup a token: 2^24 tokens and more."""
    t, h = (1 << 24) + 3, 1032
    pos = reversed_rows(t, 1)
    x = torch.zeros(t, h, dtype=BF16, device="cuda")
    mark = (torch.arange(t, device="cuda") % 251 + 1).to(BF16)
    x[:, 0] = mark
    x[:, -1] = mark
    rows = av.averis_moe_dispatch(x, pos)
    for c in (0, h - 1):
        same(rows[:, c], mark.flip(0))
    x.zero_()
    av.averis_moe_combine(rows, pos, out=x)
    for c in (0, h - 1):
        same(x[:, c], mark)
    every(x[-5:, 1:-1] == 0)


def test_order_of_2_30_slots():
    """Each token takes experts 0 .. 7 in turn: slot (t, j) is row j T + t."""
    t, k = (1 << 27) + 5, 8
    ids = torch.arange(k, dtype=torch.int32, device="cuda").repeat(t, 1)
    offsets, pos, src = av.averis_moe_sort(ids, k)
    assert offsets.tolist() == [j * t for j in range(k + 1)]
    row = torch.arange(t, dtype=torch.int32, device="cuda")
    for j in range(k):
        same(pos[:, j], row + j * t)
        same(src[j * t:(j + 1) * t], row * k + j)
