"""Layer norm's eps has to be a number that fp32 holds (no GPU): the kernels take it
in fp32, where others would become an infinity or a zero."""
import pytest

import zero_optimizer_step_gb300 as dpg

BUF = 1 << 20   # an aligned address that is never read: the calls stop before


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


@pytest.mark.parametrize("eps", [3.5e38, 1e300, 1e-46, 5e-324])
def test_refused(eps):
    before = dpg.dpg_launch_count()
    assert dpg.lib().dpg_layer_norm(BUF, 0, 4, 64, None, None, 0, eps, BUF, None, None, None) == dpg.DPG_ERR_INVALID_ARG
    assert b"eps" in dpg.lib().dpg_last_error()
    assert dpg.dpg_launch_count() == before


@pytest.mark.parametrize("eps", [0.0, -0.0, 1e-45, 1e-12, 3.4e38])
def test_taken(eps):
    assert dpg.lib().dpg_layer_norm(None, 0, 0, 64, None, None, 0, eps, None, None, None, None) == dpg.DPG_OK
