"""Layer norm of rows so wide that one chain of fp32 additions to a thread would drift."""
import pytest
import torch

import zero_optimizer_step_gb300 as dpg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


@pytest.mark.parametrize("cols", [1 << 24, (1 << 24) + 3])
def test_rows_of_many_equal_squares(cols):
    # No thread adds more than 128 terms before they go to a 64-bit sum; then a tree of ten levels
    # over the threads and the quotient: 140 roundings of the mean and of the variance.
    x = torch.full((1, cols), 4 / 3, device="cuda")
    half = cols // 2
    x[0, half:] = 2 / 3
    hi, lo = x[0, 0].double().item(), x[0, -1].double().item()
    m64 = (half * hi + (cols - half) * lo) / cols
    v64 = (half * (hi - m64) ** 2 + (cols - half) * (lo - m64) ** 2) / cols
    y, mean, rstd = torch.empty_like(x), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    dpg.dpg_layer_norm(x, None, None, 0.0, y, mean, rstd)
    assert abs(mean.item() - m64) <= 140 * U * m64
    # of the root half of the variance's, of whose terms each has a difference's rounding twice; and
    # the mean's own difference, whose square is nothing beside the variance
    assert abs(rstd.item() * v64 ** 0.5 - 1) <= (75 + 4 + 4) * U
    n64 = (hi - m64) / v64 ** 0.5, (lo - m64) / v64 ** 0.5
    tol = (140 * m64 / v64 ** 0.5 + 90) * U * 1.05
    assert (y[0, :half].double() - n64[0]).abs().max().item() <= tol
    assert (y[0, half:].double() - n64[1]).abs().max().item() <= tol


@pytest.mark.parametrize("cols", [1 << 24, (1 << 24) + 3])
def test_gradients_of_rows_of_many_equal_terms(cols):
    # A row's two sums: at most 128 terms of a thread, of which each has the roundings of n, a tree of
    # nine levels, the quotient: 150 roundings of the mean of magnitudes.
    x, dy = torch.full((1, cols), 1.0, device="cuda"), torch.full((1, cols), 1 / 3, device="cuda")
    half = cols // 2
    x[0, half:] = -1.0
    dy[0, half:] = 1 / 7
    mean, rstd = torch.zeros(1, device="cuda"), torch.full((1,), 1.1, device="cuda")
    r = rstd.double().item()
    g = dy[0, 0].double().item(), dy[0, -1].double().item()
    share = half / cols, (cols - half) / cols
    c1 = share[0] * g[0] + share[1] * g[1]
    c2 = (share[0] * g[0] - share[1] * g[1]) * r
    dx = torch.empty_like(x)
    dpg.dpg_layer_norm_backward(dy, x, None, mean, rstd, dx)
    magnitudes = c1 + r * (c1 * r)
    for at, g0, n in ((slice(0, half), g[0], r), (slice(half, None), g[1], -r)):
        want = r * (g0 - c1 - n * c2)
        assert (dx[0, at].double() - want).abs().max().item() <= r * 160 * U * magnitudes
