"""dpg_orthogonalize on both of its paths: extreme magnitudes, the floor of the
norm, many short-sided matrices of every padded side, and the same matrix beside
others.  Each test states the path that it is about."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from muon_util import COEFFS, check_ortho, make_matrix, newton_schulz_64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _object(shapes):
    plan = dpg.dpg_plan_buckets([r * c * k for r, c, k in shapes], 1 << 40, 1)
    return plan, dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])


def _slices(plan, shapes):
    for p, (r, c, k) in enumerate(shapes):
        for i in range(k):
            o = int(plan.param_offset[p]) + i * r * c
            yield r, c, slice(o, o + r * c)


def _launches(mats, u, hp):
    """Launches of a call, and its result.  The tiles take three, the Gram path
    three too, or five and more where it launches its steps by padded side; of
    six default steps, its launches after the first double."""
    out = torch.full((u.numel(),), 7.0, dtype=torch.bfloat16, device=DEV)
    before = dpg.dpg_launch_count()
    dpg.dpg_orthogonalize(mats, u, hp, out)
    dpg.dpg_matrices_status(mats)
    return dpg.dpg_launch_count() - before, out.float().cpu().numpy()


def _takes_tiles_alone(mats, u):
    return _launches(mats, u, dpg.MuonHParams(coeffs=[COEFFS] * 6))[0] == 3


def _run(shapes, values, dtype, eps, tiles):
    plan, mats = _object(shapes)
    flat = np.zeros(plan.total_padded, np.float32)
    for k, (r, c, at) in enumerate(_slices(plan, shapes)):
        flat[at] = values(k, r, c).reshape(-1)
    u = torch.from_numpy(flat).to(dtype)
    hp = dpg.MuonHParams(eps=eps)
    assert _takes_tiles_alone(mats, u.to(DEV)) == tiles
    _, got = _launches(mats, u.to(DEV), hp)
    host = u.double().numpy()
    for r, c, at in _slices(plan, shapes):
        check_ortho(got[at].reshape(r, c), newton_schulz_64(host[at].reshape(r, c), hp.coeffs, eps), f"{r}x{c}")


# the tiles: one norm item, several with 16-byte aligned and with odd slices
TILED = [[(150, 260, 1)], [(260, 150, 1)], [(256, 512, 2)], [(151, 333, 3)]]


@pytest.mark.parametrize("shapes,tiles", [(s, True) for s in TILED] + [([(70, 150, 1)], False), ([(33, 9, 2)], False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-30, 1e-25, 1e-16, 1e-12, 1e8, 1e14, 1e16, 1e20, 1e30, 1e35])
def test_scales(shapes, tiles, dtype, scale):
    # squares within and outside of fp32's range, norms above eps
    rng = np.random.Generator(np.random.Philox(51))
    _run(shapes, lambda k, r, c: make_matrix("gauss", r, c, rng, scale), dtype, 1e-30, tiles)


@pytest.mark.parametrize("shapes", TILED)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_entries_of_very_different_sizes(shapes, dtype):
    # rows of 1e18 beside rows of 1e-18, and a few large values in vectors of small ones
    def values(k, r, c):
        rng = np.random.Generator(np.random.Philox(52 + k))
        u = rng.standard_normal((r, c))
        u[::2] *= 1e18
        u[1::2] *= 1e-18
        u[:, ::37] *= 1e-3
        return u.astype(np.float32)
    _run(shapes, values, dtype, 1e-7, True)


@pytest.mark.parametrize("shapes,tiles", [(s, True) for s in TILED] + [([(70, 150, 1)], False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps,scale", [(1.0, 1e-4), (3.0, 1e-3), (1e-3, 1e-7), (1e-30, 1e-34), (1e10, 1e7)])
def test_eps_floor(shapes, tiles, dtype, eps, scale):
    # norms below eps are divided by eps: the iteration starts small
    rng = np.random.Generator(np.random.Philox(53))
    _run(shapes, lambda k, r, c: make_matrix("gauss", r, c, rng, scale), dtype, eps, tiles)


@pytest.mark.parametrize("coeffs", [
    [COEFFS], [COEFFS] * 2, [(1.5, -0.5, 0.0)] * 12, [(2.0, -1.5, 0.5)] * 8,
    [(4.0, -7.0, 3.4), (3.9, -6.0, 2.8), (2.3, -1.9, 0.4), (1.875, -1.25, 0.375)],
    [(1.0, 0.0, 0.0)] * 3], ids=["one", "two", "cubic", "quintic", "schedule", "identity"])
@pytest.mark.parametrize("rows,cols", [(12, 20), (30, 70), (60, 50), (100, 300)])
def test_coefficients_on_the_gram_path(rows, cols, coeffs):
    rng = np.random.Generator(np.random.Philox(54))
    shapes = [(rows, cols, 3)]
    plan, mats = _object(shapes)
    u = torch.zeros(plan.total_padded, dtype=torch.bfloat16)
    for r, c, at in _slices(plan, shapes):
        u[at] = torch.from_numpy(make_matrix("spiked", r, c, rng).reshape(-1)).to(torch.bfloat16)
    assert not _takes_tiles_alone(mats, u.to(DEV))
    _, got = _launches(mats, u.to(DEV), dpg.MuonHParams(coeffs=coeffs))
    for r, c, at in _slices(plan, shapes):
        check_ortho(got[at].reshape(r, c), newton_schulz_64(u[at].double().numpy().reshape(r, c), coeffs, 1e-7))


@pytest.mark.parametrize("n_steps", [5, 8])
def test_many_short_sides_of_every_padded_side(n_steps):
    # more than the launch of mixed sides takes: one launch for each padded side
    shapes = [(100, 128, 2), (7, 50, 6), (40, 90, 4), (20, 33, 5), (128, 70, 2), (3, 3, 3), (64, 64, 3), (31, 17, 2)]
    rng = np.random.Generator(np.random.Philox(55))
    plan, mats = _object(shapes)
    assert mats.n_matrices > 15
    u = torch.zeros(plan.total_padded)
    for r, c, at in _slices(plan, shapes):
        u[at] = torch.from_numpy(make_matrix("spiked", r, c, rng).reshape(-1))
    hp = dpg.MuonHParams(coeffs=[COEFFS] * n_steps)
    launches, got = _launches(mats, u.to(DEV), hp)
    assert launches == (6 if n_steps == 5 else 18)     # a sum, four of steps, an application; in three phases
    for r, c, at in _slices(plan, shapes):
        check_ortho(got[at].reshape(r, c), newton_schulz_64(u[at].double().numpy().reshape(r, c), hp.coeffs, hp.eps),
                    f"{r}x{c}")


def test_the_path_goes_by_the_list_alone():
    # one matrix alone takes the Gram path, beside a larger one the tiles; both
    # are right, and its values change neither the path nor the bits of others
    rng = np.random.Generator(np.random.Philox(56))
    small = make_matrix("spiked", 100, 200, rng)
    want = newton_schulz_64(small.astype(np.float64), [COEFFS] * 5, 1e-7)
    results = []
    for shapes, tiles in (([(100, 200, 1)], False), ([(100, 200, 1), (300, 400, 1)], True)):
        plan, mats = _object(shapes)
        at = slice(int(plan.param_offset[0]), int(plan.param_offset[0]) + 100 * 200)
        flat = rng.standard_normal(plan.total_padded).astype(np.float32)
        flat[at] = small.reshape(-1)
        u = torch.from_numpy(flat).to(DEV)
        assert _takes_tiles_alone(mats, u) == tiles
        _, got = _launches(mats, u, dpg.MuonHParams())
        check_ortho(got[at].reshape(100, 200), want)
        u[at] = 1.0
        _, other = _launches(mats, u, dpg.MuonHParams())
        rest = np.ones(plan.total_padded, bool)
        rest[at] = False
        assert np.array_equal(got[rest], other[rest], equal_nan=True)
        results.append(got[at])
    assert not np.array_equal(results[0], results[1])      # (fp32 against fp16 products)
