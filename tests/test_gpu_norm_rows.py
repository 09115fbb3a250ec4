"""Layer norm's gradient sums over so many rows that one chain of fp32 additions to a
thread would drift, and the room that they take in the workspace."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(60_000_001, 8), (2_000_001, 70), (1_200_001, 1025), (400_001, 2056)])
def test_sums_over_many_rows(rows, cols, dtype):
    # A thread adds at most 1024 rows' terms; then eight warps, at most 256 parts to a thread in one
    # chain and as many chains, the threads' tree, and the terms' own roundings.
    x, dy = torch.full((rows, cols), 0.7, dtype=dtype, device="cuda"), torch.full((rows, cols), 1 / 3, dtype=dtype, device="cuda")
    mean, rstd = torch.full((rows,), 0.1, device="cuda"), torch.full((rows,), 1 / 0.7, device="cuda")
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dgain, dbias = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    dpg.dpg_layer_norm_backward(dy, x, None, mean, rstd, None, dgain, dbias, ws)
    g, n = dy[0, 0].double().item(), (x[0, 0].double().item() - mean[0].double().item()) * rstd[0].double().item()
    parts = ws.numel() // (8 * cols)
    depth = 1024 + 8 + min(256, -(-parts // 16)) + -(-parts // 4096) + 4 + 4
    for got, term in ((dgain, g * n), (dbias, g)):
        assert (got.double() / (rows * term) - 1).abs().max().item() <= depth * U


def test_parts_of_either_type_fit_the_workspace():
    """Both types' sums, in a workspace with a border, where rows are shared out again."""
    for rows, cols in ((311_297, 2056), (311_297, 4096), (155_649, 6000), (160_001, 9000)):
        size = dpg.dpg_layer_norm_workspace(rows, cols)
        beside = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        for dtype in (torch.bfloat16, torch.float32):
            x, dy = torch.ones(rows, cols, dtype=dtype, device="cuda"), torch.ones(rows, cols, dtype=dtype, device="cuda")
            dgain, dbias = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            dpg.dpg_layer_norm_backward(dy, x, None, mean, rstd, None, dgain, dbias, beside[:size])
            np.testing.assert_array_equal(dgain.cpu().numpy(), np.full(cols, rows, np.float32))
            np.testing.assert_array_equal(dbias.cpu().numpy(), np.full(cols, rows, np.float32))
            assert (beside[size:] == 0xA5).all()
            del x, dy
