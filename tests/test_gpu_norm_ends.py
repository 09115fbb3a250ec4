"""Layer norm's gradients of rows whose deviations are so small that the square of
their inverse leaves fp32."""
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from test_gpu_norm import check_backward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


# of a warp, of CTAs (one and two rows to an exchange), odd ones, and rows read again
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [96, 500, 600, 768, 1000, 1003, 1504, 2048, 4000, 4099, 5000, 16384, 16390, 20000])
@pytest.mark.parametrize("with_gain", [False, True])
def test_inverse_deviations_whose_squares_leave_fp32(with_gain, cols, dtype):
    rows = 5
    x, dy = make(rows, cols, torch.float32, cols).mul(2.0 ** -70).to(dtype), make(rows, cols, dtype, cols + 1, 0.0) * 1e-2
    gain = 1 + make(1, cols, dtype, 2)[0] * 0.1 if with_gain else None
    mean = x.double().mean(1).float()
    rstd = (1 / (x.double() - mean.double()[:, None]).square().mean(1).sqrt()).float()
    assert (rstd > 2.0 ** 65).all() and rstd.isfinite().all()
    dx, dgain, dbias = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, dx, dgain, dbias, ws)
    assert dx.isfinite().all()
    check_backward(dy, x, gain, mean, rstd, dx, dgain, dbias)
