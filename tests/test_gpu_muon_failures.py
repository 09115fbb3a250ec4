"""Waits of the orthogonalisation that run out, and what a step does then."""
import numpy as np
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


def _object(shapes, R=1):
    plan = dpg.dpg_plan_buckets([r * c * k for r, c, k in shapes], 1 << 40, R)
    return plan, dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])


def _timed_out(mats):
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_matrices_status(mats)
    assert e.value.status == dpg.DPG_ERR_DEVICE_TIMEOUT
    dpg.dpg_matrices_status(mats)      # reported once


STEP_SHAPES = [[(300, 700, 2)], [(60, 90, 1), (20, 20, 3)]]


@pytest.mark.parametrize("shapes", STEP_SHAPES)
@pytest.mark.parametrize("upd_dtype", [torch.bfloat16, torch.float32])
def test_step_whose_wait_ran_out_leaves_the_weights(monkeypatch, shapes, upd_dtype):
    plan, mats = _object(shapes, R=2)
    n = plan.total_padded
    g = torch.Generator().manual_seed(8)
    grads = [(torch.randn(n, generator=g) * 1e-3).to(torch.bfloat16).to(DEV) for _ in range(2)]
    w0 = (torch.randn(n, generator=g) * 0.02).to(DEV)
    hp = dpg.MuonHParams(lr=0.02, weight_decay=0.1, eps=1e-12)

    def state():
        return w0.clone(), torch.zeros(n, device=DEV), torch.zeros(n, dtype=upd_dtype, device=DEV), \
            torch.full((n,), 3.0, dtype=torch.bfloat16, device=DEV)

    w, m, upd, view = state()
    dpg.dpg_muon_step(plan, mats, grads, [5, 6], hp, w, m, upd, [view])
    dpg.dpg_matrices_status(mats)
    want_w, want_m, want_view = w, m, view

    w, m, upd, view = state()
    monkeypatch.setenv("DPG_TEST_HOOKS", "1")
    dpg.dpg_set_staged_fault(skip_unit=3, timeout_ns=20_000_000)
    dpg.dpg_muon_step(plan, mats, grads, [5, 6], hp, w, m, upd, [view])
    torch.cuda.synchronize()
    assert torch.equal(w, w0) and torch.all(view == 3.0)       # neither weights nor views
    assert torch.equal(m, want_m)                              # the momentum has taken the gradient
    # until the record is cleared, later updates are held back too
    dpg.dpg_muon_apply(mats, torch.zeros(n, dtype=torch.bfloat16, device=DEV), hp, w, [view])
    torch.cuda.synchronize()
    assert torch.equal(w, w0) and torch.all(view == 3.0)
    _timed_out(mats)
    # the step can be taken again from its momentum: Nesterov's update of it, then the rest
    om = torch.tensor(1.0 - hp.momentum, device=DEV)
    s = (grads[0].float() + grads[1].float()) * torch.tensor(1.0 / 11, device=DEV)
    upd = (s * om + torch.tensor(hp.momentum, device=DEV) * m).to(upd_dtype)
    o = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    dpg.dpg_orthogonalize(mats, upd, hp, o)
    dpg.dpg_muon_apply(mats, o, hp, w, [view])
    dpg.dpg_matrices_status(mats)
    for p, (r, c, k) in enumerate(shapes):
        at = slice(int(plan.param_offset[p]), int(plan.param_offset[p]) + r * c * k)
        assert torch.equal(w[at], want_w[at]) and torch.equal(view[at], want_view[at])


@pytest.mark.parametrize("shapes", [[(16, 40, 2)], [(30, 50, 1)], [(64, 200, 1)], [(100, 128, 1)],
                                    [(5, 7, 1), (128, 90, 1), (40, 41, 1)]])
def test_short_side_waits_are_bounded(monkeypatch, shapes):
    # one value of an exchange is never sent: the waits for it run out, the
    # error is reported once, and the next call is whole
    rng = np.random.Generator(np.random.Philox(41))
    plan, mats = _object(shapes)
    u = torch.from_numpy(rng.standard_normal(plan.total_padded).astype(np.float32)).to(DEV)
    outs = [torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), outs[0])
    dpg.dpg_matrices_status(mats)
    monkeypatch.setenv("DPG_TEST_HOOKS", "1")
    dpg.dpg_set_staged_fault(skip_unit=0, timeout_ns=20_000_000)
    dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), outs[1])
    _timed_out(mats)
    for o in outs[1:]:                 # (the fault is used up)
        dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), o)
        dpg.dpg_matrices_status(mats)
        assert torch.equal(o, outs[0])


def test_fault_is_used_up_by_matrices_of_any_size(monkeypatch):
    _, small = _object([(20, 30, 1)])
    plan, large = _object([(300, 400, 1)])
    u = torch.randn(plan.total_padded, device=DEV)
    o = torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV)
    monkeypatch.setenv("DPG_TEST_HOOKS", "1")
    dpg.dpg_set_staged_fault(skip_unit=-1, timeout_ns=20_000_000)
    dpg.dpg_orthogonalize(small, u, dpg.MuonHParams(), o)
    dpg.dpg_matrices_status(small)
    dpg.dpg_set_staged_fault(skip_unit=0, timeout_ns=20_000_000)
    dpg.dpg_orthogonalize(small, u, dpg.MuonHParams(), o)
    dpg.dpg_orthogonalize(large, u, dpg.MuonHParams(), o)
    dpg.dpg_matrices_status(large)
    _timed_out(small)


@pytest.mark.parametrize("skip", [0, 3, 40])
def test_waits_of_steps_with_both_halves_are_bounded(monkeypatch, skip):
    rng = np.random.Generator(np.random.Philox(42))
    plan, mats = _object([(300, 700, 2)])
    u = torch.from_numpy(rng.standard_normal(plan.total_padded).astype(np.float32)).to(DEV)
    hp = dpg.MuonHParams(precise=True)
    outs = [torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    dpg.dpg_orthogonalize(mats, u, hp, outs[0])
    dpg.dpg_matrices_status(mats)
    monkeypatch.setenv("DPG_TEST_HOOKS", "1")
    dpg.dpg_set_staged_fault(skip_unit=skip, timeout_ns=20_000_000)
    dpg.dpg_orthogonalize(mats, u, hp, outs[1])
    _timed_out(mats)
    dpg.dpg_orthogonalize(mats, u, hp, outs[1])
    dpg.dpg_matrices_status(mats)
    assert torch.equal(outs[0], outs[1])
