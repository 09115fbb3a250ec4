"""Host-side checks of layer norm (no GPU): workspace sizes and every refusal,
which comes before any device work."""
import pytest
import torch

import zero_optimizer_step_gb300 as dpg

BUF = 1 << 20   # an aligned address that is never read: the calls stop before
INVALID, MISALIGNED = dpg.DPG_ERR_INVALID_ARG, dpg.DPG_ERR_MISALIGNED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def refused(status, text, fn, *args):
    before = dpg.dpg_launch_count()
    assert fn(*args) == status, dpg.lib().dpg_last_error()
    assert text.encode() in dpg.lib().dpg_last_error(), dpg.lib().dpg_last_error()
    assert dpg.dpg_launch_count() == before


@pytest.mark.parametrize("kw,status,text", [
    (dict(rows=-1), INVALID, "outside"), (dict(cols=-1), INVALID, "outside"),
    (dict(cols=(1 << 30) + 1), INVALID, "outside"), (dict(rows=(1 << 30) + 1), INVALID, "outside"),
    (dict(dtype=2), INVALID, "dtype 2"), (dict(param_dtype=3), INVALID, "param_dtype 3"),
    (dict(eps=-1e-5), INVALID, "eps"), (dict(eps=NAN), INVALID, "eps"), (dict(eps=INF), INVALID, "eps"),
    (dict(mean=None), INVALID, "kept together"), (dict(rstd=None), INVALID, "kept together"),
    (dict(x=None), INVALID, "x is NULL"), (dict(y=None), INVALID, "y is NULL"),
    (dict(x=BUF + 1), MISALIGNED, "x misaligned"), (dict(y=BUF + 1), MISALIGNED, "y misaligned"),
    (dict(gain=BUF + 1), MISALIGNED, "gain misaligned"), (dict(bias=BUF + 1), MISALIGNED, "bias misaligned"),
    (dict(gain=BUF + 2, param_dtype=dpg.DPG_F32), MISALIGNED, "gain misaligned"),
    (dict(mean=BUF + 2), MISALIGNED, "mean misaligned"), (dict(rstd=BUF + 2), MISALIGNED, "rstd misaligned"),
])
def test_norm_refusals(kw, status, text):
    a = dict(x=BUF, dtype=dpg.DPG_BF16, rows=4, cols=64, gain=BUF, bias=BUF, param_dtype=dpg.DPG_BF16, eps=1e-5,
             y=BUF, mean=BUF, rstd=BUF)
    a.update(kw)
    refused(status, text, dpg.lib().dpg_layer_norm, *a.values(), None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(rows=-1), INVALID, "outside"), (dict(cols=-1), INVALID, "outside"),
    (dict(dtype=2), INVALID, "dtype 2"), (dict(param_dtype=3), INVALID, "param_dtype 3"),
    (dict(grad_dtype=4), INVALID, "grad_dtype 4"),
    (dict(accumulate=1, grad_dtype=dpg.DPG_BF16), INVALID, "only fp32"),
    (dict(dy=None), INVALID, "dy is NULL"), (dict(x=None), INVALID, "x is NULL"),
    (dict(mean=None), INVALID, "mean is NULL"), (dict(rstd=None), INVALID, "rstd is NULL"),
    (dict(dy=BUF + 1), MISALIGNED, "dy misaligned"), (dict(dx=BUF + 1), MISALIGNED, "dx misaligned"),
    (dict(dgain=BUF + 2), MISALIGNED, "dgain misaligned"), (dict(dbias=BUF + 2), MISALIGNED, "dbias misaligned"),
    (dict(workspace=None), INVALID, "workspace is NULL"), (dict(workspace=BUF + 8), MISALIGNED, "workspace"),
    (dict(rows=0, dgain=BUF + 2), MISALIGNED, "dgain misaligned"),
])
def test_backward_refusals(kw, status, text):
    a = dict(dy=BUF, x=BUF, dtype=dpg.DPG_BF16, rows=4, cols=64, gain=BUF, param_dtype=dpg.DPG_BF16, mean=BUF,
             rstd=BUF, dx=BUF, dgain=BUF, dbias=BUF, grad_dtype=dpg.DPG_F32, accumulate=0, workspace=BUF)
    a.update(kw)
    refused(status, text, dpg.lib().dpg_layer_norm_backward, *a.values(), None)


def test_nothing_to_do():
    L = dpg.lib()
    before = dpg.dpg_launch_count()
    for rows, cols in ((0, 64), (64, 0), (0, 0)):
        assert L.dpg_layer_norm(None, 0, rows, cols, None, None, 0, 1e-5, None, None, None, None) == dpg.DPG_OK
    none = [None] * 3
    assert L.dpg_layer_norm_backward(None, None, 0, 0, 64, None, 0, None, None, *none, 0, 0, None, None) == dpg.DPG_OK
    assert L.dpg_layer_norm_backward(BUF, BUF, 0, 4, 64, None, 0, BUF, BUF, *none, 0, 0, None, None) == dpg.DPG_OK
    # no rows to add
    assert L.dpg_layer_norm_backward(None, None, 0, 0, 64, None, 0, None, None, None, BUF, BUF, 1, 1, None,
                                     None) == dpg.DPG_OK
    assert dpg.dpg_launch_count() == before


def test_workspace_bytes():
    for rows, cols in ((0, 64), (1, 1), (7, 768), (9000, 768), (9000, 5000), (10, 100000)):
        n = dpg.dpg_layer_norm_workspace(rows, cols)
        assert n > 0 and n % (8 * cols) == 0 and n <= 608 * 8 * cols
    assert dpg.dpg_layer_norm_workspace(4, 0) == 0
    assert dpg.dpg_layer_norm_workspace(-1, 4) == 0 and dpg.dpg_layer_norm_workspace(4, 1 << 31) == 0


def test_binding_refuses_what_it_can_see():
    x, v = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(TypeError):
        dpg.dpg_layer_norm(x, v, v, 1e-5, x, stream=0)             # not on a GPU
    with pytest.raises(TypeError):
        dpg.dpg_layer_norm(x.double(), v, v, 1e-5, x, stream=0)
    with pytest.raises(ValueError):
        dpg.dpg_layer_norm(x.t(), v, v, 1e-5, x, stream=0)
