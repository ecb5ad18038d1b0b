"""8-bit products whose scales are far from 1, on every kind of kernel."""
import pytest
import torch

from gated_ref import U
from selective_state_space_69_amd import binding as B

pytestmark = pytest.mark.gpu

# the few-row kernel, split contractions and their join, every kind of tile, ragged edges
SHAPES = [(8, 2560, 640), (20, 333, 70), (70, 5000, 64), (100, 257, 129), (300, 770, 331),
          (2048, 768, 1536), (4100, 200, 4200), (4096, 160, 5120)]


@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("a,b", [(1e-20, 1e-20), (1e-23, 1e-20), (1e20, 1e-25), (1e-25, 1e20), (1e36, 1e-38),
                                 (1e-41, 1e30), (1e20, 1e20), (2.0, 0.5)])
@pytest.mark.parametrize("residual", [False, True])
def test_scales(m, k, n, a, b, residual):
    """y = sum xs ws wherever that is a number of fp32, whatever xs ws alone would be: three
    roundings, and half a step of the smallest number; a sum of 0 gives 0."""
    g = torch.Generator(device="cuda")
    g.manual_seed(m + 3 * k + 7 * n)
    xq = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    xq[m // 2] = 0
    wq[n // 3] = 0
    xs = a * (0.5 + torch.rand(m, generator=g, device="cuda"))
    ws = b * (0.5 + torch.rand(n, generator=g, device="cuda"))
    xs[::7] = 1.0                            # rows of ordinary scale among them
    r = torch.zeros(m, n, device="cuda") if residual else None
    got = B.q8_linear((xq, xs), (wq, ws), residual=r, out_dtype=torch.float32).double()
    want = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
    most = torch.finfo(torch.float32).max
    big = want.abs() > most * (1 - 4 * U)
    assert bool((got[big].abs() > most * (1 - 8 * U)).all())
    off = (got - want).abs()[~big]
    assert bool((off <= 3 * U * want.abs()[~big] + 2.0 ** -150).all()), float((off / want.abs()[~big]).nan_to_num().max())
    assert not bool(got[m // 2].any()) and not bool(got[:, n // 3].any())


@pytest.mark.parametrize("m", [8, 100, 4100])
def test_scales_that_are_not_numbers(m):
    """A scale that is NaN reaches its whole row or column, beside any other scale."""
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    xq = torch.randint(-127, 128, (m, 96), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (200, 96), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.full((m,), 1e-30, device="cuda"), torch.full((200,), 1e-3, device="cuda")
    ws[:9] = 1e30
    xs[3] = float("nan")
    ws[5] = ws[150] = float("nan")
    bad = torch.zeros(m, 200, dtype=torch.bool, device="cuda")
    bad[3] = True
    bad[:, [5, 150]] = True
    got = B.q8_linear((xq, xs), (wq, ws), out_dtype=torch.float32)
    assert torch.equal(torch.isnan(got), bad)
