"""Checks of the Newton-Schulz coefficients on the host (no GPU)."""
import ctypes

import pytest
import torch

import zero_optimizer_step_gb300 as dpg

BUF = 1 << 20   # an aligned address that is never read: the calls stop before


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def _refusal(coeffs):
    """The message dpg_orthogonalize refuses with; the update is NULL, so that
    coefficients it takes end in that refusal."""
    plan = dpg.dpg_plan_buckets([24], 1 << 20, 1)
    mats = dpg.dpg_plan_matrices(plan, [4], [6])
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_orthogonalize(mats, None, dpg.MuonHParams(coeffs=coeffs), BUF, update_dtype=dpg.DPG_BF16, stream=0)
    assert e.value.status == dpg.DPG_ERR_INVALID_ARG
    return str(e.value)


@pytest.mark.parametrize("c", [0.0, 1e-20, -1e-20, 1e-12, -1e-12, 1e-6, -1e-6, 1e-300, -1e-300])
def test_a_vanishing_quintic_term_is_a_cubic(c):
    # 100 s - 100 s^3 reaches 38.5 at s = 0.577 and vanishes at the end: the
    # extremum has to be found whatever rounding does to a tiny c
    assert "after step 0" in _refusal([(100.0, -100.0, c)])
    # 60 s - 60 s^3 reaches 23.1
    assert "update is NULL" in _refusal([(60.0, -60.0, c)])


@pytest.mark.parametrize("coeffs", [(1e200, -1e200, 0.0), (1e200, -1e200, 1e-5), (1e308, -1e308, 1.0), (0.0, 1e300, -1e300),
                                    (1e155, -2e155, 1e155), (-1e200, 1e200, 0.0)])
def test_huge_coefficients_that_cancel_at_the_end_are_refused(coeffs):
    assert "after step 0" in _refusal([coeffs])


def test_quintic_extrema_inside():
    # s (1 - s^2)^2 k = k s - 2 k s^3 + k s^5: largest at s = 1 / sqrt(5), 0.286 k
    assert "update is NULL" in _refusal([(110.0, -220.0, 110.0)])
    assert "after step 0" in _refusal([(113.0, -226.0, 113.0)])


def _values(hp):
    c = hp.c()
    return [list(c.coeffs[k]) for k in range(c.n_steps)]


def test_coefficients_are_read_at_every_call():
    # values held in objects that are changed in place: not those of an earlier call
    a, row = torch.tensor(3.0), [torch.tensor(2.0), torch.tensor(-1.5), torch.tensor(0.5)]
    hp = dpg.MuonHParams(coeffs=[(a, -1.0, 0.25), row])
    assert _values(hp) == [[3.0, -1.0, 0.25], [2.0, -1.5, 0.5]]
    a.fill_(1.0)
    row[1].fill_(-2.0)
    assert _values(hp) == [[1.0, -1.0, 0.25], [2.0, -2.0, 0.5]]
    table = torch.tensor([[3.0, -1.0, 0.25]], dtype=torch.float64)
    hp = dpg.MuonHParams(coeffs=table)
    assert _values(hp) == [[3.0, -1.0, 0.25]]
    table[0, 0] = 2.0
    assert _values(hp) == [[2.0, -1.0, 0.25]]
    assert ctypes.sizeof(hp.c()) == 16 * 24 + 32 + 16


def test_coefficients_need_three_values_a_step():
    for bad in ([(1.0, 2.0)], [(1.0, 2.0, 3.0, 4.0)]):
        with pytest.raises(ValueError):
            dpg.MuonHParams(coeffs=bad).c()
