"""dpg_orthogonalize with ``precise``: the rounding to bf16 is all that is left."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from muon_schedules import SCHEDULES, condition, make_low_rank, to_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda"
# Steps' error: fp32's over a few steps and, in directions that bf16 leaves at
# 2^-9 of the rest, that much more of it (1e-6 and 1e-4).
FULL_RANK, LOW_RANK = 1e-5, 2e-4


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("name", ["5", "minimax5", "8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(256, 512), (700, 300), (151, 333), (100, 300), (40, 16), (200, 9000)])
def test_precise(rows, cols, dtype, name):
    kinds = [("gauss", FULL_RANK), ("spiked", FULL_RANK), ("half", LOW_RANK), ("rank4", LOW_RANK),
             ("repeated", LOW_RANK), ("rows4", LOW_RANK), ("rows16", LOW_RANK)]
    rng = np.random.Generator(np.random.Philox(61))
    n = rows * cols
    plan = dpg.dpg_plan_buckets([n * len(kinds)], 1 << 40, 1)
    mats = dpg.dpg_plan_matrices(plan, [rows], [cols])
    us = [to_dtype(make_low_rank(k, rows, cols, rng), dtype == torch.bfloat16) for k, _ in kinds]
    flat = np.zeros(plan.total_padded, np.float32)
    flat[:n * len(kinds)] = np.concatenate([u.reshape(-1) for u in us])
    hp = dpg.MuonHParams(coeffs=SCHEDULES[name], precise=True, eps=1e-20)
    out = torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV)
    dpg.dpg_orthogonalize(mats, torch.from_numpy(flat).to(dtype).to(DEV), hp, out)
    dpg.dpg_matrices_status(mats)
    got = out.double().cpu().numpy()
    for k, (kind, bound) in enumerate(kinds):
        want, moved = condition(us[k], hp.coeffs, hp.eps, rng)
        y = got[k * n:(k + 1) * n].reshape(rows, cols)
        # what is more than half the spacing of bf16 values (8 bits, the first of them 1)
        e = (bound + 2.0 * moved) * np.linalg.norm(want)
        half = 2.0 ** (np.frexp(want)[1] - 1 - 8)
        over = np.maximum(np.abs(y - want) - half, 0.0)
        assert np.linalg.norm(over) <= e, f"{kind}: {np.linalg.norm(over) / np.linalg.norm(want):.2e}, moved {moved:.1e}"
        if kind in ("gauss", "spiked") and name == "5":
            # an error of 1e-5 of the root mean square crosses a rounding boundary in
            # under 2 % of the elements
            rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
            assert np.mean(y != rounded) <= 0.02, kind


def test_precise_is_off_by_default_and_leaves_the_fast_bits():
    rng = np.random.Generator(np.random.Philox(62))
    plan = dpg.dpg_plan_buckets([300 * 400], 1 << 40, 1)
    mats = dpg.dpg_plan_matrices(plan, [300], [400])
    u = torch.from_numpy(rng.standard_normal(plan.total_padded).astype(np.float32)).to(DEV)
    outs = [torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    for o, p in zip(outs, (False, True, False)):
        dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(precise=p), o)
    dpg.dpg_matrices_status(mats)
    assert torch.equal(outs[0], outs[2]) and not torch.equal(outs[0], outs[1])
    assert not dpg.MuonHParams().precise
