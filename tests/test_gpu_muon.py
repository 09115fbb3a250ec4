"""The matrix-orthogonalising (Muon) operators on the GPU against plain forms:
dpg_muon_momentum and dpg_muon_apply bit for bit against the same binary32
operations in numpy, dpg_orthogonalize against the steps in 64 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from muon_util import (COEFFS, apply_f32, bf16_round, check_ortho, make_matrix, momentum_f32,
                       newton_schulz_64, scale_of)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _plan(shapes, R=1, cap=1 << 40):
    """shapes: (rows, cols, count) per parameter."""
    plan = dpg.dpg_plan_buckets([r * c * k for r, c, k in shapes], cap, R)
    return plan, dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])


def _flat(plan, shapes, make, fill=0.0):
    flat = np.full(plan.total_padded, fill, np.float32)
    for p, (r, c, k) in enumerate(shapes):
        o = plan.param_offset[p]
        for i in range(k):
            flat[o + i * r * c:o + (i + 1) * r * c] = make(p, i, r, c).reshape(-1)
    return flat


def _pieces(plan, shapes):
    for p, (r, c, k) in enumerate(shapes):
        for i in range(k):
            o = int(plan.param_offset[p]) + i * r * c
            yield p, i, r, c, slice(o, o + r * c)


def _ortho_case(shapes, kind, dtype, hp=None, scale=1e-3, seed=5, in_place=False):
    rng = np.random.Generator(np.random.Philox(seed))
    plan, mats = _plan(shapes)
    u = torch.from_numpy(_flat(plan, shapes, lambda p, i, r, c: make_matrix(kind, r, c, rng, scale),
                               fill=float("nan"))).to(dtype)
    hp = hp or dpg.MuonHParams()
    upd = u.to(DEV)
    out = upd if in_place else torch.full((plan.total_padded,), 7.0, dtype=torch.bfloat16, device=DEV)
    dpg.dpg_orthogonalize(mats, upd, hp, out)
    torch.cuda.synchronize()
    got, host = out.float().cpu().numpy(), u.double().numpy()
    covered = np.zeros(plan.total_padded, bool)
    for p, i, r, c, at in _pieces(plan, shapes):
        want = newton_schulz_64(host[at].reshape(r, c), hp.coeffs, hp.eps)
        check_ortho(got[at].reshape(r, c), want, f"{kind} {r}x{c} #{i}")
        covered[at] = True
    if not in_place:
        assert np.all(got[~covered] == 7.0)      # padding slots are not written
        assert np.array_equal(upd.cpu().view(torch.uint8).numpy(), u.view(torch.uint8).numpy())


SHAPES = [(1, 1), (1, 777), (777, 1), (2, 2), (3, 1000), (64, 32), (32, 10), (63, 65), (127, 129),
          (128, 128), (128, 512), (255, 257), (256, 256), (257, 256), (130, 2000), (512, 130),
          (300, 301), (768, 768), (513, 1031)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_orthogonalize_shapes(rows, cols, dtype):
    _ortho_case([(rows, cols, 1)], "gauss", dtype)


@pytest.mark.parametrize("kind", ["spiked", "lowrank", "rank1", "outlier", "equal", "diag"])
@pytest.mark.parametrize("rows,cols", [(96, 200), (200, 96), (256, 256), (320, 700)])
def test_orthogonalize_spectra(kind, rows, cols):
    _ortho_case([(rows, cols, 1)], kind, torch.bfloat16)
    _ortho_case([(rows, cols, 1)], kind, torch.float32)


@pytest.mark.parametrize("rows,cols", [(257, 40000), (39100, 300), (700, 26000)])
def test_orthogonalize_many_tiles(rows, cols):
    # enough tiles for clusters of two pairs; odd numbers of them in a row
    _ortho_case([(rows, cols, 1)], "spiked", torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shapes", [[(200, 9000, 1)], [(9001, 300, 2)], [(150, 1030, 3)], [(700, 4300, 1)],
                                    [(513, 2305, 4), (300, 256, 4)], [(129, 2000, 40), (400, 400, 1)]])
def test_orthogonalize_long_matrices(shapes, dtype):
    # sums over the long side in parts, beside matrices that have none, and the
    # same bits every time
    _ortho_case(shapes, "spiked", dtype)
    rng = np.random.Generator(np.random.Philox(14))
    plan, mats = _plan(shapes)
    u = torch.from_numpy(_flat(plan, shapes, lambda p, i, r, c: make_matrix("gauss", r, c, rng))).to(DEV).to(dtype)
    outs = [torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    for o in outs:
        dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), o)
    dpg.dpg_matrices_status(mats)
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(128, 3000), (3000, 128), (65, 66), (16, 16), (17, 5000), (5000, 33),
                                       (1, 40000), (2, 2), (128, 129)])
def test_orthogonalize_short_side(rows, cols, dtype):
    # the path of up to 128 rows: every padded side, partial blocks of columns
    for kind in ("gauss", "rank1"):
        _ortho_case([(rows, cols, 2)], kind, dtype)


@pytest.mark.parametrize("shapes", [[(100, 100, 30)], [(128, 600, 70), (20, 20, 5)],
                                    [(1, 777, 1), (50, 40, 3), (200, 300, 1)], [(7, 64, 900), (260, 260, 1)]])
def test_orthogonalize_short_sides_among_others(shapes):
    # too many for the small launches at once, or beside larger ones
    _ortho_case(shapes, "spiked", torch.bfloat16)


def test_orthogonalize_list_of_matrices():
    # stacks, tall and wide, odd sizes whose slices start off 16-byte boundaries
    _ortho_case([(333, 129, 2), (1, 77, 3), (64, 32, 1), (129, 333, 1), (5, 5, 5), (640, 512, 2),
                 (1, 1, 9), (90, 1100, 1)], "gauss", torch.bfloat16)
    _ortho_case([(31, 33, 3), (0 + 7, 9, 4), (260, 1000, 1)], "spiked", torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16])
def test_orthogonalize_in_place(dtype):
    _ortho_case([(100, 300, 2), (64, 64, 1)], "gauss", dtype, in_place=True)


@pytest.mark.parametrize("scale", [1e-25, 1e-12, 1e8, 1e20, 1e30])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_orthogonalize_scales(scale, dtype):
    # squares below and above fp32's range; eps below the norm
    _ortho_case([(70, 150, 1)], "gauss", dtype, hp=dpg.MuonHParams(eps=1e-30), scale=scale)


def test_orthogonalize_eps_floor():
    # a norm below eps is divided by eps: the iteration starts small
    _ortho_case([(70, 150, 1)], "gauss", torch.float32, hp=dpg.MuonHParams(eps=1.0), scale=1e-4)


@pytest.mark.parametrize("coeffs", [
    [COEFFS], [COEFFS] * 2, [(1.5, -0.5, 0.0)] * 12, [(2.0, -1.5, 0.5)] * 8,
    [(4.0, -7.0, 3.4), (3.9, -6.0, 2.8), (2.3, -1.9, 0.4), (1.875, -1.25, 0.375)],
    [(1.0, 0.0, 0.0)] * 3], ids=["one", "two", "cubic", "quintic", "schedule", "identity"])
def test_orthogonalize_coefficients(coeffs):
    _ortho_case([(150, 70, 1), (300, 420, 1)], "gauss", torch.bfloat16, hp=dpg.MuonHParams(coeffs=coeffs))


@pytest.mark.parametrize("rows,cols", [(40, 60), (150, 140)])
def test_orthogonalize_zero_and_nonfinite_matrices(rows, cols):
    shapes = [(rows, cols, 6)]
    rng = np.random.Generator(np.random.Philox(9))
    plan, mats = _plan(shapes)
    clean = _flat(plan, shapes, lambda p, i, r, c: make_matrix("gauss", r, c, rng))
    flat = clean.copy()
    n = rows * cols
    flat[n:2 * n] = 0.0
    flat[2 * n + 17] = np.nan
    flat[3 * n + 99] = np.inf
    flat[4 * n + 3] = -np.inf
    hp = dpg.MuonHParams()
    outs = []
    for f in (clean, flat):
        out = torch.empty(plan.total_padded, dtype=torch.bfloat16, device=DEV)
        dpg.dpg_orthogonalize(mats, torch.from_numpy(f).to(DEV), hp, out)
        outs.append(out.cpu())
    a, b = outs
    assert torch.equal(a[:n], b[:n]) and torch.equal(a[5 * n:6 * n], b[5 * n:6 * n])
    assert torch.all(b[n:2 * n] == 0)
    assert torch.all(torch.isnan(b[2 * n:5 * n].float()))
    # nothing of it stays in the workspace
    out = torch.empty(plan.total_padded, dtype=torch.bfloat16, device=DEV)
    dpg.dpg_orthogonalize(mats, torch.from_numpy(clean).to(DEV), hp, out)
    assert torch.equal(out.cpu(), a)


def test_orthogonalize_is_deterministic_and_holds_a_shared_plan():
    shapes = [(300, 500, 3), (1000, 260, 1), (20, 30, 2)]
    rng = np.random.Generator(np.random.Philox(10))
    plan, mats = _plan(shapes)
    u = torch.from_numpy(_flat(plan, shapes, lambda p, i, r, c: make_matrix("spiked", r, c, rng))).to(DEV)
    outs = [torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    plan2_total = plan.total_padded
    plan.destroy()                      # the matrices keep what they need of it
    for o in outs[:2]:
        dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), outs[2])
    torch.cuda.synchronize()
    assert plan2_total == outs[0].numel()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_orthogonalize_waits_are_bounded(monkeypatch):
    # one stage of operands is never fetched: the wait for it runs out, every
    # other one gives up, the error is reported once, and the next call is whole
    shapes = [(300, 700, 2), (64, 64, 1)]
    rng = np.random.Generator(np.random.Philox(12))
    plan, mats = _plan(shapes)
    u = torch.from_numpy(_flat(plan, shapes, lambda p, i, r, c: make_matrix("gauss", r, c, rng))).to(DEV)
    out = [torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), out[0])
    dpg.dpg_matrices_status(mats)
    monkeypatch.setenv("DPG_TEST_HOOKS", "1")
    dpg.dpg_set_staged_fault(skip_unit=3, timeout_ns=20_000_000)
    dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), out[1])
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_matrices_status(mats)
    assert e.value.status == dpg.DPG_ERR_DEVICE_TIMEOUT
    dpg.dpg_matrices_status(mats)
    dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), out[1])
    dpg.dpg_matrices_status(mats)
    assert torch.equal(out[0], out[1])


def test_orthogonalize_on_two_streams_at_once():
    # two objects whose kernels each want the whole GPU
    shapes = [(500, 900, 2)]
    rng = np.random.Generator(np.random.Philox(13))
    objs = [_plan(shapes) for _ in range(2)]
    u = torch.from_numpy(_flat(objs[0][0], shapes,
                               lambda p, i, r, c: make_matrix("spiked", r, c, rng))).to(DEV)
    want = torch.zeros_like(u, dtype=torch.bfloat16)
    dpg.dpg_orthogonalize(objs[0][1], u, dpg.MuonHParams(), want)
    torch.cuda.synchronize()
    outs = [torch.zeros_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for (_, mats), o, s in zip(objs, outs, streams):
            dpg.dpg_orthogonalize(mats, u, dpg.MuonHParams(), o, stream=s)
    torch.cuda.synchronize()
    for (_, mats), o in zip(objs, outs):
        dpg.dpg_matrices_status(mats)
        assert torch.equal(o, want)


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("mode", ["bf16", "f32", "f32_last"])
@pytest.mark.parametrize("nesterov,out", [(True, torch.bfloat16), (False, torch.float32)])
def test_momentum_bits(R, mode, nesterov, out):
    shapes = [(13, 77, 1), (64, 32, 2), (1, 5, 1), (500, 33, 1)]
    plan, _ = _plan(shapes, R=R, cap=20000)
    N = plan.total_padded
    g = torch.Generator().manual_seed(100 + R)
    rnd = lambda s: torch.randn(N, generator=g) * s
    grads = [rnd(1e-3).to(torch.bfloat16 if mode == "bf16" else torch.float32) for _ in range(R)]
    last = [rnd(1e-3).to(torch.bfloat16) for _ in range(R)] if mode == "f32_last" else None
    m0, mu = rnd(1e-6), 0.95
    tokens = [3000 + 7 * r for r in range(R)]
    m = m0.to(DEV)
    upd = torch.zeros(N, dtype=out, device=DEV)
    hp = dpg.MuonHParams(momentum=mu, nesterov=nesterov)
    dl = None if last is None else [x.to(DEV) for x in last]
    half = plan.n_buckets // 2
    assert half >= 1
    for b0, b1 in ((0, half), (half, plan.n_buckets)):
        dpg.dpg_muon_momentum(plan, [x.to(DEV) for x in grads], tokens, hp, m, upd, last_micro=dl,
                              b0=b0, b1=b1)
    wm, wu = momentum_f32([x.float().numpy() for x in grads],
                          None if last is None else [x.float().numpy() for x in last], tokens, mu,
                          nesterov, m0.numpy())
    assert np.array_equal(m.cpu().numpy().view(np.uint32), wm.view(np.uint32))
    want = torch.from_numpy(wu).to(out)
    assert torch.equal(upd.cpu(), want)


def test_momentum_propagates_nonfinite_values():
    plan, _ = _plan([(8, 16, 1)], R=2)
    N = plan.total_padded
    grads = [torch.zeros(N, dtype=torch.bfloat16) for _ in range(2)]
    grads[0][3], grads[1][4], grads[0][5] = float("nan"), float("inf"), float("-inf")
    m, upd = torch.zeros(N, device=DEV), torch.zeros(N, device=DEV)
    dpg.dpg_muon_momentum(plan, [x.to(DEV) for x in grads], [1, 1], dpg.MuonHParams(), m, upd)
    for t in (m.cpu(), upd.cpu()):
        assert torch.isnan(t[3]) and t[4] == float("inf") and t[5] == float("-inf")
        keep = torch.ones(N, dtype=torch.bool)
        keep[3:6] = False
        assert torch.all(t[keep] == 0)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("wd", [0.0, 0.1])
@pytest.mark.parametrize("n_views", [0, 1, 3])
def test_apply_bits(rms, wd, n_views):
    shapes = [(13, 77, 1), (77, 13, 2), (1, 5, 1), (500, 33, 1), (64, 64, 1)]
    plan, mats = _plan(shapes)
    N = plan.total_padded
    g = torch.Generator().manual_seed(3)
    w0, o = torch.randn(N, generator=g) * 0.02, (torch.randn(N, generator=g) * 0.03).to(torch.bfloat16)
    w = w0.to(DEV)
    views = [torch.full((N,), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(n_views)]
    hp = dpg.MuonHParams(lr=0.02, weight_decay=wd,
                         scale_rule=dpg.DPG_SCALE_RMS if rms else dpg.DPG_SCALE_SPECTRAL)
    dpg.dpg_muon_apply(mats, o.to(DEV), hp, w, views)
    want = w0.numpy().copy()
    for p, i, r, c, at in _pieces(plan, shapes):
        want[at] = apply_f32(want[at], o[at].float().numpy(), 0.02, wd, scale_of(rms, r, c))
    assert np.array_equal(w.cpu().numpy().view(np.uint32), want.view(np.uint32))
    for v in views:
        for p, i, r, c, at in _pieces(plan, shapes):
            assert torch.equal(v.cpu()[at], bf16_round(want)[at])


def _step_inputs(shapes, R, seed=21):
    plan, mats = _plan(shapes, R=R, cap=1 << 18)
    N = plan.total_padded
    g = torch.Generator().manual_seed(seed)
    live = np.zeros(N, bool)
    for *_, at in _pieces(plan, shapes):
        live[at] = True
    live = torch.from_numpy(live)
    grads = [(torch.randn(N, generator=g) * 1e-3 * live).to(torch.bfloat16).to(DEV) for _ in range(R)]
    w = (torch.randn(N, generator=g) * 0.02 * live).to(DEV)
    m = (torch.randn(N, generator=g) * 1e-8 * live).to(DEV)
    return plan, mats, grads, w, m, [3000 + r for r in range(R)]


@pytest.mark.parametrize("upd_dtype", [torch.bfloat16, torch.float32])
def test_step_is_its_three_operators(upd_dtype):
    shapes = [(300, 120, 2), (64, 32, 1), (97, 211, 1), (256, 512, 1)]
    plan, mats, grads, w, m, tokens = _step_inputs(shapes, R=4)
    N = plan.total_padded
    hp = dpg.MuonHParams(lr=0.02, weight_decay=0.1, eps=1e-12, scale_rule=dpg.DPG_SCALE_RMS)
    w2, m2 = w.clone(), m.clone()
    upd, p = torch.zeros(N, dtype=upd_dtype, device=DEV), torch.zeros(N, dtype=torch.bfloat16, device=DEV)
    upd2, o2, p2 = upd.clone(), torch.zeros_like(p), torch.zeros_like(p)
    for _ in range(2):
        dpg.dpg_muon_step(plan, mats, grads, tokens, hp, w, m, upd, [p])
        dpg.dpg_muon_momentum(plan, grads, tokens, hp, m2, upd2)
        dpg.dpg_orthogonalize(mats, upd2, hp, o2)
        dpg.dpg_muon_apply(mats, o2, hp, w2, [p2])
    assert torch.equal(w, w2) and torch.equal(m, m2)
    got = upd.view(torch.bfloat16)[:N]
    for *_, at in _pieces(plan, shapes):
        assert torch.equal(p[at], p2[at]) and torch.equal(got[at], o2[at])


def test_step_against_64_bits():
    shapes = [(120, 300, 1), (64, 32, 2), (400, 130, 1)]
    plan, mats, grads, w, m, tokens = _step_inputs(shapes, R=3)
    hp = dpg.MuonHParams(lr=0.02, weight_decay=0.1, eps=1e-12)
    w0, m0 = w.double().cpu().numpy(), m.double().cpu().numpy()
    upd = torch.zeros(plan.total_padded, device=DEV)
    dpg.dpg_muon_step(plan, mats, grads, tokens, hp, w, m, upd, [])
    g = sum(x.double().cpu().numpy() for x in grads) / sum(tokens)
    wm = 0.95 * m0 + 0.05 * g
    u = 0.05 * g + 0.95 * wm
    got = w.double().cpu().numpy()
    for p, i, r, c, at in _pieces(plan, shapes):
        o = newton_schulz_64(u[at].reshape(r, c), hp.coeffs, hp.eps).reshape(-1)
        k = hp.lr * scale_of(False, r, c)
        # the update actually applied, against the exact one
        check_ortho((w0[at] * (1 - hp.lr * 0.1) - got[at]).reshape(r, c) / k, o.reshape(r, c), f"{r}x{c}")


def test_step_in_a_cuda_graph():
    shapes = [(300, 120, 1), (64, 32, 1)]
    plan, mats, grads, w, m, tokens = _step_inputs(shapes, R=2)
    hp = dpg.MuonHParams(eps=1e-12)
    upd = torch.zeros(plan.total_padded, device=DEV)
    dpg.dpg_matrices_upload(mats)
    w2, m2 = w.clone(), m.clone()
    for _ in range(3):
        dpg.dpg_muon_step(plan, mats, grads, tokens, hp, w2, m2, upd, [])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dpg.dpg_muon_step(plan, mats, grads, tokens, hp, w, m, upd, [])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, w2) and torch.equal(m, m2)


def test_step_minimises_a_matrix_least_squares():
    # f(W) = |W A - Y|^2 / 2 split over two replicas: the loss falls steadily
    torch.manual_seed(0)
    r, c, n = 96, 160, 512
    plan, mats = _plan([(r, c, 1)], R=2)
    A, Wt = torch.randn(c, n, device=DEV), torch.randn(r, c, device=DEV) / 12
    w = torch.zeros(plan.total_padded, device=DEV)
    m, upd = torch.zeros_like(w), torch.zeros_like(w)
    p = torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV)
    losses = []
    for t in range(30):
        W = p[:r * c].view(r, c).float()
        E = W @ A - Wt @ A
        losses.append(float(E.square().sum()))
        gs = []
        for k in range(2):
            h = slice(k * n // 2, (k + 1) * n // 2)
            g = torch.zeros(plan.total_padded, dtype=torch.bfloat16, device=DEV)
            g[:r * c] = (E[:, h] @ A[:, h].T).reshape(-1)
            gs.append(g)
        dpg.dpg_muon_step(plan, mats, gs, [n // 2, n // 2], dpg.MuonHParams(lr=0.1, momentum=0.8), w, m,
                          upd, [p])
    assert losses[-1] < 0.05 * losses[0]


def test_example_trains_a_small_network():
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(here, "examples", "muon_adam.py")], cwd=here,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    losses = [float(line.split()[-1]) for line in r.stdout.splitlines() if line.startswith("step")]
    assert len(losses) == 4 and losses[-1] < 0.5 * losses[0], r.stdout
