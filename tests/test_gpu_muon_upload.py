"""The first call of an object on a stream that does not wait for the default
one: its tables must have arrived before the kernels read them."""
import pytest
import torch

import zero_optimizer_step_gb300 as dpg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("count", [1, 3000])
def test_first_update_on_a_stream_of_its_own(count):
    plan = dpg.dpg_plan_buckets([64 * 48 * count], 1 << 40, 1)
    n = plan.total_padded
    w0, o = torch.randn(n, device=DEV), torch.randn(n, device=DEV).to(torch.bfloat16)
    hp, stream = dpg.MuonHParams(lr=0.5, weight_decay=0.1), torch.cuda.Stream()
    results = []
    for _ in range(4):                      # a new object, so new tables, each time
        mats = dpg.dpg_plan_matrices(plan, [64], [48])
        w = w0.clone()
        torch.cuda.synchronize()
        dpg.dpg_muon_apply(mats, o, hp, w, [], stream=stream)
        torch.cuda.synchronize()
        results.append(w)
    want = w0 - 0.05 * w0 - 0.5 * (64 / 48) ** 0.5 * o.float()
    assert torch.allclose(results[0], want, rtol=1e-5, atol=1e-6)
    assert all(torch.equal(r, results[0]) for r in results)


def test_first_step_on_a_stream_of_its_own():
    plan = dpg.dpg_plan_buckets([700 * 300, 64 * 32 * 20], 1 << 16, 1)
    n = plan.total_padded
    g, stream = [torch.randn(n, device=DEV).to(torch.bfloat16)], torch.cuda.Stream()
    results = []
    for _ in range(3):
        mats = dpg.dpg_plan_matrices(plan, [700, 64], [300, 32])
        w, m, upd = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
        torch.cuda.synchronize()
        dpg.dpg_muon_step(plan, mats, g, [1], dpg.MuonHParams(), w, m, upd, [], stream=stream)
        dpg.dpg_matrices_status(mats, stream=stream)
        results.append(w)
    assert float(results[0].abs().max()) > 0 and all(torch.equal(r, results[0]) for r in results)
