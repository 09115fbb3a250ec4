"""A 4-bit layer's gradients, as the device leaves them, against what a change of one
weight, or of one input, makes of the device's outputs."""
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import MX, NV, values_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def exact(rows, cols, seed):
    """A matrix of E2M1 values with a 6 in every block of either orientation: both
    quantised forms stand for it exactly."""
    g = torch.Generator().manual_seed(seed)
    x = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0])[torch.randint(6, (rows, cols), generator=g)]
    x[(torch.arange(rows)[:, None] + torch.arange(cols)) % 16 == 0] = 6.0
    return torch.where(torch.rand(rows, cols, generator=g) < 0.5, -x, x)


def both(x, fmt):
    q = dpg.Fp4(*x.shape, fmt), dpg.Fp4(*x.shape[::-1], fmt)
    dpg.dpg_fp4_quantize(x.cuda(), *q)
    assert torch.equal(torch.from_numpy(values_of(q[0])).float(), x)
    assert torch.equal(torch.from_numpy(values_of(q[1])).float(), x.t())
    return q


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("t,out,inn", [(64, 80, 48), (304, 272, 144)])
def test_gradients_against_differences(t, out, inn, fmt):
    x, dy, w = exact(t, inn, 1), exact(t, out, 2), exact(out, inn, 3)
    (xr, xc), (gr, gc), (wr, wc) = both(x, fmt), both(dy, fmt), both(w, fmt)

    def product(a, b):
        c = torch.empty(a.rows, b.rows, device="cuda")
        dpg.dpg_fp4_product(a, b, c)
        return c.cpu().double()

    y, dx, dw = product(xr, wr), product(gr, wc), product(gc, xc)
    # Every value is a multiple of 1/4 and every sum below 36 * 304: exact in fp32.  The loss,
    # sum of y dy, is linear in a weight and in an input.
    places = torch.Generator().manual_seed(4)
    for _ in range(4):
        o, i, r = (int(torch.randint(n, (1,), generator=places)) for n in (out, inn, t))
        if (o + i) % 16 == 0 or (r + i) % 16 == 0:              # (a block's 6 stays)
            i = (i + 1) % inn
        more = w.clone()
        more[o, i] = 1.0 if w[o, i] != 1.0 else 3.0
        moved = ((product(xr, both(more, fmt)[0]) - y) * dy).sum().item()
        assert moved == dw[o, i].item() * (more[o, i] - w[o, i]).item()
        more = x.clone()
        more[r, i] = -2.0 if x[r, i] != -2.0 else 0.5
        moved = ((product(both(more, fmt)[0], wr) - y) * dy).sum().item()
        assert moved == dx[r, i].item() * (more[r, i] - x[r, i]).item()
