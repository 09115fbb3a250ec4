"""Layer norm's results in one place (no GPU): refused before device work, since either
would be written over the other."""
import pytest

import zero_optimizer_step_gb300 as dpg

BUF = 1 << 20   # an aligned address that is never read: the calls stop before


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def refused(fn, *args):
    before = dpg.dpg_launch_count()
    assert fn(*args) == dpg.DPG_ERR_INVALID_ARG
    assert b"share a buffer" in dpg.lib().dpg_last_error()
    assert dpg.dpg_launch_count() == before


@pytest.mark.parametrize("cols", [64, 50000])
def test_refused(cols):
    refused(dpg.lib().dpg_layer_norm, BUF, 0, 4, cols, None, None, 0, 1e-5, BUF, 2 * BUF, 2 * BUF, None)
    for rows in (0, 4):
        refused(dpg.lib().dpg_layer_norm_backward, BUF, BUF, 0, rows, cols, None, 0, 2 * BUF, 3 * BUF, None, 4 * BUF, 4 * BUF, 1, 0,
                BUF, None)
