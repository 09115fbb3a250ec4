"""dpg_orthogonalize beyond five default steps, and on matrices whose rows
depend on one another, against the steps in 64 bits."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from muon_schedules import FEW_ROWS_REL, LONG_REL, SCHEDULES, STEPS_REL, allowed, condition, make_low_rank, to_dtype

pytestmark = pytest.mark.gpu
DEV = "cuda"
LONG = [k for k in SCHEDULES if k != "5"]
KINDS = ["rank1", "rank4", "half", "tail", "repeated", "equal", "gauss", "spiked"]


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _takes_tiles(mats, upd, out):
    """Whether all of the object's matrices take the tiles: three launches
    (norms, load, steps), where the Gram path takes three for each of its
    phases and six default steps are two of them."""
    before = dpg.dpg_launch_count()
    dpg.dpg_orthogonalize(mats, upd, dpg.MuonHParams(coeffs=SCHEDULES["6"]), out)
    return dpg.dpg_launch_count() - before == 3


def _check(shapes, kinds, name, dtype, steps_rel, tiles, seed=31, first_rel=None):
    """One object over `shapes`; the matrices take `kinds` in turn.  tiles: the
    path its matrices must have been given; first_rel: bound of the first one."""
    rng = np.random.Generator(np.random.Philox(seed))
    plan = dpg.dpg_plan_buckets([r * c * k for r, c, k in shapes], 1 << 40, 1)
    mats = dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])
    hp = dpg.MuonHParams(coeffs=SCHEDULES[name], eps=1e-20)
    flat = np.zeros(plan.total_padded, np.float64)
    items = []
    for p, (r, c, k) in enumerate(shapes):
        for i in range(k):
            at = slice(int(plan.param_offset[p]) + i * r * c, int(plan.param_offset[p]) + (i + 1) * r * c)
            kind = kinds[len(items) % len(kinds)]
            u = to_dtype(make_low_rank(kind, r, c, rng), dtype == torch.bfloat16)
            flat[at] = u.reshape(-1)
            items.append((kind, r, c, at, u))
    upd = torch.from_numpy(flat.astype(np.float32)).to(dtype).to(DEV)
    out = torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV)
    assert _takes_tiles(mats, upd, out) == tiles
    dpg.dpg_orthogonalize(mats, upd, hp, out)
    dpg.dpg_matrices_status(mats)
    got = out.double().cpu().numpy()
    for n, (kind, r, c, at, u) in enumerate(items):
        bound = steps_rel if n or first_rel is None else first_rel
        want, moved = condition(u, hp.coeffs, hp.eps, rng)
        y = got[at].reshape(r, c)
        assert np.all(np.isfinite(y)), f"{kind} {r}x{c}"
        rel = np.linalg.norm(y - want) / np.linalg.norm(want)
        assert rel <= allowed(bound, moved, u.size), f"{kind} {r}x{c}: {rel:.3e}, moved {moved:.1e}"
        # no direction grows past what the steps can make of a singular value
        assert np.linalg.norm(y, 2) <= 2.2, f"{kind} {r}x{c}"


@pytest.mark.parametrize("name", LONG)
@pytest.mark.parametrize("rows,cols", [(16, 40), (40, 16), (32, 64), (64, 300), (128, 600), (600, 100), (5, 7)])
def test_long_schedules_short_side(rows, cols, name):
    _check([(rows, cols, len(KINDS))], KINDS, name, torch.bfloat16, LONG_REL, tiles=False)
    _check([(rows, cols, len(KINDS))], KINDS, name, torch.float32, LONG_REL, tiles=False)


@pytest.mark.parametrize("name", LONG)
@pytest.mark.parametrize("rows,cols", [(150, 260), (260, 150), (256, 512), (520, 300)])
def test_long_schedules_tiles(rows, cols, name):
    _check([(rows, cols, len(KINDS))], KINDS, name, torch.bfloat16, LONG_REL, tiles=True)
    _check([(rows, cols, len(KINDS))], KINDS, name, torch.float32, LONG_REL, tiles=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shapes,tiles", [([(100, 200, 8)], False), ([(200, 100, 8)], False), ([(31, 90, 8)], False),
                                          ([(256, 512, 8)], True), ([(700, 300, 8)], True)])
def test_five_steps_on_dependent_rows(shapes, tiles, dtype):
    _check(shapes, KINDS, "5", dtype, STEPS_REL, tiles)


@pytest.mark.parametrize("name", ["8", "minimax8"])
def test_long_schedules_long_matrices(name):
    # sums in parts, tiles of several widths, many columns
    _check([(200, 9000, 2)], ["spiked", "repeated"], name, torch.bfloat16, LONG_REL, tiles=True)
    _check([(5000, 300, 1), (700, 900, 2)], ["gauss", "rank4", "half"], name, torch.float32, LONG_REL, tiles=True)
    _check([(128, 6000, 2), (3000, 64, 2)], ["rank4", "repeated", "spiked"], name, torch.bfloat16, LONG_REL,
           tiles=False)


def test_long_schedules_are_deterministic_and_leave_no_trace():
    # the same bits every time, also for a default call before and after
    rng = np.random.Generator(np.random.Philox(32))
    shapes = [(300, 500, 2), (64, 90, 2)]
    plan = dpg.dpg_plan_buckets([r * c * k for r, c, k in shapes], 1 << 40, 1)
    mats = dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])
    u = torch.from_numpy(rng.standard_normal(plan.total_padded).astype(np.float32)).to(DEV)
    outs = [torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV) for _ in range(5)]
    for o, name in zip(outs, ("5", "16", "5", "16", "5")):
        dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(coeffs=SCHEDULES[name]), o)
    dpg.dpg_matrices_status(mats)
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[0], outs[4]) and torch.equal(outs[1], outs[3])


def test_step_with_a_long_schedule_in_a_cuda_graph():
    shapes = [(300, 120, 1), (64, 32, 1)]
    plan = dpg.dpg_plan_buckets([r * c * k for r, c, k in shapes], 1 << 18, 1)
    mats = dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])
    g = torch.Generator().manual_seed(4)
    n = plan.total_padded
    grads = [(torch.randn(n, generator=g) * 1e-3).to(torch.bfloat16).to(DEV)]
    w, m = (torch.randn(n, generator=g) * 0.02).to(DEV), torch.zeros(n, device=DEV)
    upd = torch.zeros(n, device=DEV)
    hp = dpg.MuonHParams(eps=1e-12, coeffs=SCHEDULES["8"])
    w2, m2 = w.clone(), m.clone()
    for _ in range(2):      # (the first call of a schedule allocates what it needs)
        dpg.dpg_muon_step(plan, mats, grads, [7], hp, w2, m2, upd, [])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        dpg.dpg_muon_step(plan, mats, grads, [7], hp, w, m, upd, [])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, w2) and torch.equal(m, m2)


@pytest.mark.parametrize("name", ["5", "minimax5", "8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [2, 3, 4, 7, 16, 33, 64, 100, 128])
def test_short_sides_beside_larger_matrices(m, dtype, name):
    # the tiles from 65 rows on here, where fewer rows average less of the rounding
    for k in range(0, 6, 2):
        kinds = ["gauss"] + ["rank1", "repeated", "rank2", "half", "near1", "equal"][k:k + 2]
        _check([(300, 400, 1), (m, 622, 1), (622 + k, m, 1)], kinds, name, dtype, LONG_REL, tiles=m > 64, seed=33 + k,
               first_rel=STEPS_REL)


@pytest.mark.parametrize("name", ["5", "minimax8", "12"])
@pytest.mark.parametrize("n", [1, 2, 777, 4000])
def test_single_rows_on_both_paths(n, name):
    for dtype in (torch.bfloat16, torch.float32):
        _check([(1, n, 2), (n, 1, 1)], ["gauss"], name, dtype, LONG_REL, tiles=False)
        _check([(300, 400, 1), (1, n, 2), (n, 1, 1)], ["gauss"], name, dtype, LONG_REL, tiles=n < 4000)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_dependent_rows(dtype):
    # what five default steps leave in the largest case known (see dpg.h); long
    # schedules' early steps, and short sides, have both halves
    kinds = ["rows3", "rows4", "rows8", "rows16"]
    _check([(256, 512, 4)], kinds, "5", dtype, FEW_ROWS_REL[dtype == torch.bfloat16], tiles=True)
    _check([(700, 300, 4)], kinds, "8", dtype, LONG_REL, tiles=True)
    _check([(100, 300, 4)], kinds, "5", dtype, LONG_REL, tiles=False)
    _check([(300, 400, 1), (100, 622, 4)], ["gauss"] + kinds, "5", dtype, LONG_REL, tiles=True)
