"""Host-side checks of the matrix-orthogonalising operators (no GPU): shapes,
workspace sizes, and every refusal, which comes before any device work."""
import ctypes

import numpy as np
import pytest

import zero_optimizer_step_gb300 as dpg
from muon_util import COEFFS, make_matrix, newton_schulz_64

BUF = 1 << 20   # an aligned address that is never read: the calls stop before


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def _mats(shapes=((4, 6), (3, 5)), counts=(1, 2)):
    plan = dpg.dpg_plan_buckets([r * c * k for (r, c), k in zip(shapes, counts)], 1 << 30, 1)
    return plan, dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])


def test_matrices_of_a_plan():
    plan, mats = _mats()
    assert mats.n_matrices == 3 and mats.workspace_bytes > 0
    # 256 x 512 padded: three X arrays, and two 256 x 256 ones, of fp16 each
    _, mats = _mats(((400, 200),), (3,))
    assert mats.n_matrices == 3
    assert mats.workspace_bytes >= 3 * (3 * 256 * 512 + 2 * 256 * 256) * 2
    empty = dpg.dpg_plan_buckets([0, 12, 0], 1 << 20, 1)
    assert dpg.dpg_plan_matrices(empty, [5, 3, 1], [5, 4, 1]).n_matrices == 1
    none = dpg.dpg_plan_buckets([], 1 << 20, 1)
    assert dpg.dpg_plan_matrices(none, [], []).n_matrices == 0


@pytest.mark.parametrize("rows,cols", [(0, 6), (4, 0), (-4, -6), (5, 6), (1 << 24, 1), (24, 2)])
def test_shapes_refused(rows, cols):
    plan = dpg.dpg_plan_buckets([24], 1 << 20, 1)
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_plan_matrices(plan, [rows], [cols])
    assert e.value.status == dpg.DPG_ERR_INVALID_ARG


def test_shape_counts_and_null_handles_refused():
    plan = dpg.dpg_plan_buckets([24, 8], 1 << 20, 1)
    with pytest.raises(ValueError):
        dpg.dpg_plan_matrices(plan, [4], [6])
    L, out = dpg.lib(), ctypes.c_void_p()
    one = np.array([1, 1], np.int64)
    assert L.dpg_plan_matrices(None, one.ctypes.data, one.ctypes.data, ctypes.byref(out)) == dpg.DPG_ERR_INVALID_ARG
    assert L.dpg_plan_matrices(plan.handle, None, one.ctypes.data, ctypes.byref(out)) == dpg.DPG_ERR_INVALID_ARG
    assert L.dpg_plan_matrices(plan.handle, one.ctypes.data, one.ctypes.data, None) == dpg.DPG_ERR_INVALID_ARG
    assert L.dpg_matrices_info(None, None, None) == dpg.DPG_ERR_INVALID_ARG
    assert L.dpg_matrices_upload(None) == dpg.DPG_ERR_INVALID_ARG
    L.dpg_matrices_destroy(None)


def test_matrices_beyond_one_object_refused():
    # workspace rows past the 32-bit coordinate of a copy
    plan = dpg.dpg_plan_buckets([1 << 20] * 64, 1 << 40, 1)
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_plan_matrices(plan, [1] * 64, [1] * 64)
    assert e.value.status == dpg.DPG_ERR_INVALID_ARG and "large" in str(e.value)


def _refused(status, text, fn, *args, **kw):
    before = dpg.dpg_launch_count()
    with pytest.raises(dpg.DpgError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.status == status and text in str(e.value), str(e.value)
    assert dpg.dpg_launch_count() == before


def _ortho(hp=None, update=BUF, dtype=dpg.DPG_BF16, out=BUF):
    _, mats = _mats()
    return (dpg.dpg_orthogonalize, mats, update, hp or dpg.MuonHParams(), out), dict(update_dtype=dtype)


INVALID = dpg.DPG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status,text", [
    (dict(update=None), INVALID, "update is NULL"),
    (dict(out=None), INVALID, "ortho_bf16 is NULL"),
    (dict(dtype=7), INVALID, "dtype 7"),
    (dict(update=BUF + 2), dpg.DPG_ERR_MISALIGNED, "update misaligned"),
    (dict(update=BUF + 16, dtype=dpg.DPG_F32), dpg.DPG_ERR_MISALIGNED, "update misaligned"),
    (dict(out=BUF + 8), dpg.DPG_ERR_MISALIGNED, "ortho_bf16 misaligned"),
    (dict(hp=dpg.MuonHParams(coeffs=[])), INVALID, "n_steps 0"),
    (dict(hp=dpg.MuonHParams(coeffs=[COEFFS] * 17)), INVALID, "n_steps 17"),
    (dict(hp=dpg.MuonHParams(eps=0.0)), INVALID, "eps"),
    (dict(hp=dpg.MuonHParams(eps=float("nan"))), INVALID, "eps"),
    (dict(hp=dpg.MuonHParams(eps=float("inf"))), INVALID, "eps"),
    (dict(hp=dpg.MuonHParams(coeffs=[(float("nan"), 0, 0)])), INVALID, "coeffs[0]"),
    (dict(hp=dpg.MuonHParams(coeffs=[COEFFS, (1, float("inf"), 0)])), INVALID, "coeffs[1]"),
    (dict(hp=dpg.MuonHParams(coeffs=[(3.0, 0.0, 0.0)] * 5)), INVALID, "after step 3"),
    (dict(hp=dpg.MuonHParams(coeffs=[(40.0, 0.0, 0.0)])), INVALID, "after step 0"),
])
def test_orthogonalize_refusals(kw, status, text):
    args, named = _ortho(**kw)
    _refused(status, text, *args, **named)


def test_orthogonalize_null_handles_refused():
    L = dpg.lib()
    hp = dpg.MuonHParams().c()
    assert L.dpg_orthogonalize(None, BUF, 0, ctypes.byref(hp), BUF, None) == INVALID
    _, mats = _mats()
    assert L.dpg_orthogonalize(mats.handle, BUF, 0, None, BUF, None) == INVALID
    assert b"hparams" in L.dpg_last_error()


@pytest.mark.parametrize("change,status,text", [
    (dict(momentum=None), INVALID, "momentum is NULL"),
    (dict(update=None), INVALID, "update is NULL"),
    (dict(grads=[None]), INVALID, "gradient"),
    (dict(grads=[BUF + 8]), dpg.DPG_ERR_MISALIGNED, "gradient"),
    (dict(momentum=BUF + 16), dpg.DPG_ERR_MISALIGNED, "momentum"),
    (dict(tokens=[0]), dpg.DPG_ERR_ZERO_TOKENS, "0"),
    (dict(tokens=[-1]), INVALID, "valid_tokens"),
    (dict(hp=dpg.MuonHParams(momentum=1.0)), INVALID, "momentum must"),
    (dict(hp=dpg.MuonHParams(momentum=float("nan"))), INVALID, "momentum must"),
    (dict(grads_dtype=3), INVALID, "grads_dtype"),
    (dict(update_dtype=3), INVALID, "dtype 3"),
    (dict(last_micro=[BUF]), INVALID, "last_micro"),
    (dict(b0=1, b1=0), INVALID, "bucket range"),
    (dict(b1=5), INVALID, "bucket range"),
])
def test_momentum_refusals(change, status, text):
    plan, _ = _mats()
    c = dict(grads=[BUF], tokens=[10], hp=dpg.MuonHParams(), momentum=BUF, update=BUF,
             grads_dtype=dpg.DPG_BF16, update_dtype=dpg.DPG_BF16)
    c.update(change)
    _refused(status, text, dpg.dpg_muon_momentum, plan, c.pop("grads"), c.pop("tokens"), c.pop("hp"),
             c.pop("momentum"), c.pop("update"), **c)


@pytest.mark.parametrize("change,status,text", [
    (dict(ortho=None), INVALID, "NULL"),
    (dict(master=None), INVALID, "master is NULL"),
    (dict(master=BUF + 16), dpg.DPG_ERR_MISALIGNED, "master"),
    (dict(ortho=BUF + 2), dpg.DPG_ERR_MISALIGNED, "update misaligned"),
    (dict(views=[None]), INVALID, "view is NULL"),
    (dict(views=[BUF] * 65), INVALID, "n_views 65"),
    (dict(hp=dpg.MuonHParams(lr=float("nan"))), INVALID, "lr"),
    (dict(hp=dpg.MuonHParams(weight_decay=float("inf"))), INVALID, "lr"),
    (dict(hp=dpg.MuonHParams(scale_rule=2)), INVALID, "scale_rule 2"),
])
def test_apply_refusals(change, status, text):
    _, mats = _mats()
    c = dict(ortho=BUF, hp=dpg.MuonHParams(), master=BUF, views=[BUF])
    c.update(change)
    _refused(status, text, dpg.dpg_muon_apply, mats, c["ortho"], c["hp"], c["master"], c["views"])


def test_step_refuses_matrices_of_another_plan():
    plan, mats = _mats()
    other = dpg.dpg_plan_buckets([24, 32], 1 << 30, 1)
    _refused(INVALID, "another plan", dpg.dpg_muon_step, other, mats, [BUF], [1], dpg.MuonHParams(),
             BUF, BUF, BUF, [], grads_dtype=0, update_dtype=0)
    _refused(dpg.DPG_ERR_ZERO_TOKENS, "0", dpg.dpg_muon_step, plan, mats, [BUF], [0], dpg.MuonHParams(),
             BUF, BUF, BUF, [], grads_dtype=0, update_dtype=0)
    _refused(INVALID, "scale_rule", dpg.dpg_muon_step, plan, mats, [BUF], [1],
             dpg.MuonHParams(scale_rule=9), BUF, BUF, BUF, [], grads_dtype=0, update_dtype=0)


def test_steps_against_singular_values():
    # the 64-bit form the GPU tests use, pinned: every step maps each singular
    # value s to a s + b s^3 + c s^5 and leaves the singular vectors
    rng = np.random.Generator(np.random.Philox(1))
    for rows, cols in ((7, 12), (12, 7), (1, 5), (6, 6)):
        u = make_matrix("gauss", rows, cols, rng).astype(np.float64)
        U, s, V = np.linalg.svd(u, full_matrices=False)
        s = s / np.linalg.norm(s)
        for a, b, c in [COEFFS] * 5:
            s = a * s + b * s ** 3 + c * s ** 5
        np.testing.assert_allclose(newton_schulz_64(u, [COEFFS] * 5, 1e-7), (U * s) @ V, rtol=0, atol=1e-11)
