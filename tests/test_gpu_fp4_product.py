"""Products of 4-bit matrices on the GPU against 64-bit products of their values."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import MX, NV, product_bound, quantized, spread, values_of

pytestmark = pytest.mark.gpu
FORMATS = [NV, MX]


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    dpg.dpg_fp4_status()


def operand(rows, cols, fmt, seed, scale=1.0):
    q = dpg.Fp4(rows, cols, fmt)
    dpg.dpg_fp4_quantize(spread(rows, cols, seed, torch.bfloat16, scale).cuda(), q)
    return q


def check(got, a, b, before=None):
    want = a @ b.T + (0 if before is None else before)
    err = np.abs(got.cpu().double().numpy() - want)
    bound = product_bound(a, b, got.dtype, want)
    if before is not None:
        bound = bound + 2.0 ** -23 * np.abs(before)
    assert np.all(err <= bound), f"{np.max(err / bound):.2f} of the bound"


SIZES = [
    (1, 1, 1), (1, 1, 64), (1, 300, 65), (300, 1, 64), (7, 130, 129), (16, 128, 256), (17, 129, 100), (33, 70, 1000),
    (64, 64, 63), (65, 65, 255), (128, 128, 256), (129, 257, 257), (300, 200, 3000), (5, 700, 5000), (700, 40, 2049),
    (24, 24, 20000), (100, 100, 20000),
    # enough tiles for pairs of CTAs: whole ones, odd ones, sums of one step, one row of tiles
    (2560, 2048, 512), (2305, 2177, 97), (200, 19500, 70), (19500, 130, 64),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_sizes(m, n, k, fmt):
    a, b = operand(m, k, fmt, 1), operand(n, k, fmt, 2, 0.02)
    av, bv = values_of(a), values_of(b)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((m, n), float("nan"), device="cuda", dtype=dtype)
        dpg.dpg_fp4_product(a, b, out)
        check(out, av, bv)
    acc = spread(m, n, 3, torch.float32, 1.0).cuda()
    before = acc.cpu().double().numpy()
    dpg.dpg_fp4_product(a, b, acc, accumulate=True)
    check(acc, av, bv, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(9, 200, 100), (200, 9, 100), (200, 150, 600), (2305, 2177, 64)])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 5), (8, 8)])
def test_strided_results_and_what_is_beside_them(offset, pad, m, n, k, dtype):
    a, b = operand(m, k, NV, 4), operand(n, k, NV, 5)
    flat = torch.full((offset + m * (n + pad) + 64,), 7.0, dtype=dtype, device="cuda")
    out = flat[offset:].as_strided((m, n), (n + pad, 1))
    dpg.dpg_fp4_product(a, b, out)
    check(out, values_of(a), values_of(b))
    out.fill_(7.0)
    assert (flat == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n", [(20, 200), (200, 150), (2400, 2400)])
def test_blocks_that_are_not_finite(m, n, fmt):
    x, w = spread(m, 300, 6, torch.bfloat16), spread(n, 300, 7, torch.bfloat16)
    x[3, 100], w[5, 299] = float("nan"), float("inf")
    a, b = dpg.Fp4(m, 300, fmt), dpg.Fp4(n, 300, fmt)
    dpg.dpg_fp4_quantize(x.cuda(), a)
    dpg.dpg_fp4_quantize(w.cuda(), b)
    out = torch.empty(m, n, device="cuda")
    dpg.dpg_fp4_product(a, b, out)
    nan = out.isnan()
    want = torch.zeros_like(nan)
    want[3, :], want[:, 5] = True, True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("sa,sb", [(1e-30, 1e30), (1e30, 1e-34), (1e-36, 1.0), (1e-20, 1e-17), (1e18, 1e15)])
def test_magnitudes(sa, sb):
    # the matrices' powers of two multiply to anything from subnormal results to large ones
    a, b = operand(40, 256, NV, 8, sa), operand(50, 256, NV, 9, sb)
    out = torch.empty(40, 50, device="cuda")
    dpg.dpg_fp4_product(a, b, out)
    check(out, values_of(a), values_of(b))


def test_matrices_of_zeros():
    for fmt in FORMATS:
        z = dpg.Fp4(300, 100, fmt)
        dpg.dpg_fp4_quantize(torch.zeros(300, 100, device="cuda"), z)
        out = torch.full((300, 300), 5.0, device="cuda")
        dpg.dpg_fp4_product(z, z, out)
        assert not out.any()


def test_sum_over_nothing():
    a, b = dpg.Fp4(5, 0), dpg.Fp4(7, 0)
    for dtype in (torch.bfloat16, torch.float32):
        flat = torch.full((5, 9), 3.0, device="cuda", dtype=dtype)
        dpg.dpg_fp4_product(a, b, flat[:, :7])
        assert not flat[:, :7].any() and (flat[:, 7:] == 3.0).all()
    dpg.dpg_fp4_product(a, b, flat[:, 2:], accumulate=True)
    assert (flat[:, 7:] == 3.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(8, 1000, 3000), (200, 300, 4000), (2400, 2400, 800)])
def test_same_bits_on_every_call(m, n, k, fmt):
    a, b = operand(m, k, fmt, 10), operand(n, k, fmt, 11)
    outs = [torch.empty(m, n, device="cuda") for _ in range(4)]
    for o in outs:
        dpg.dpg_fp4_product(a, b, o)
    assert all(torch.equal(outs[0], o) for o in outs)


def test_two_streams_at_once():
    sizes = [(2400, 2400, 2000), (8, 3000, 5000), (300, 300, 6000)]
    ops = [(operand(m, k, NV, 20), operand(n, k, NV, 21), torch.empty(m, n, device="cuda")) for m, n, k in sizes]
    want = []
    for a, b, o in ops:
        dpg.dpg_fp4_product(a, b, o)
        want.append(o.clone())
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (a, b, o) in zip(streams, ops):
            dpg.dpg_fp4_product(a, b, o, stream=s)
    torch.cuda.synchronize()
    for w, (_, _, o) in zip(want, ops):
        assert torch.equal(w, o)


def test_replayed_graph():
    x = spread(2400, 500, 30, torch.bfloat16).cuda()
    w = operand(2400, 500, MX, 31)
    few = operand(9, 500, MX, 32)
    a, y, z = dpg.Fp4(2400, 500, MX), torch.empty(2400, 2400, device="cuda"), torch.zeros(9, 2400, device="cuda")

    def step():
        dpg.dpg_fp4_quantize(x, a)
        dpg.dpg_fp4_product(a, w, y)
        dpg.dpg_fp4_product(few, a, z, accumulate=True)

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    x.copy_(spread(2400, 500, 33, torch.bfloat16))
    z.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    av = quantized(x.double().cpu().numpy(), MX)[2]
    check(y, av, values_of(w))
    one = torch.empty_like(z)
    dpg.dpg_fp4_product(few, a, one)
    check(one, values_of(few), av)
    assert torch.equal(z, one + one)


def test_layer_forward_and_backward():
    """A layer's three products as they are used, into slices of flat buffers."""
    t, out, inn = 300, 260, 140
    plan = dpg.dpg_plan_buckets([out * inn, inn], 1 << 30, 2)
    mats = dpg.dpg_plan_matrices(dpg.dpg_plan_buckets([out * inn], 1 << 30, 1), [out], [inn])
    master = spread(1, out * inn, 40, torch.float32, 0.05).view(-1).cuda()
    pad = torch.zeros(mats.total_padded, device="cuda")
    pad[:out * inn] = master
    w, wt = dpg.Fp4(out, inn), dpg.Fp4(inn, out)
    dpg.dpg_allgather_params_fp4(mats, pad, [w], [wt])
    x, dy = spread(t, inn, 41, torch.bfloat16, 1.0).cuda(), spread(t, out, 42, torch.bfloat16).cuda()
    xr, xc, gr, gc = dpg.Fp4(t, inn), dpg.Fp4(inn, t), dpg.Fp4(t, out), dpg.Fp4(out, t)
    seed = torch.tensor([7], device="cuda")
    y, dx = torch.empty(t, out, device="cuda", dtype=torch.bfloat16), torch.empty(t, inn, device="cuda",
                                                                                dtype=torch.bfloat16)
    grads = torch.zeros(plan.total_padded, device="cuda", dtype=torch.bfloat16)
    at = int(plan.param_offset[0])
    dw = grads[at:at + out * inn].view(out, inn)
    dpg.dpg_fp4_quantize(x, xr, xc)
    dpg.dpg_fp4_product(xr, w, y)
    dpg.dpg_fp4_quantize(dy, gr, gc, seed=seed)
    dpg.dpg_fp4_product(gr, wt, dx)
    dpg.dpg_fp4_product(gc, xc, dw)
    check(y, values_of(xr), values_of(w))
    check(dx, values_of(gr), values_of(wt))
    check(dw, values_of(gc), values_of(xc))
    acc = torch.ones(out, inn, device="cuda")
    dpg.dpg_fp4_product(gc, xc, acc, accumulate=True)
    check(acc, values_of(gc), values_of(xc), np.ones((out, inn)))
    assert not grads[at + out * inn:].any()
    # the sum of y's products with dy changes by dw along a change of w (one element, exactly)
    dw64 = values_of(gc) @ values_of(xc).T
    w64 = values_of(w)
    more = w64.copy()
    more[5, 7] += 0.5
    loss = lambda v: float((values_of(gc).T * (values_of(xc).T @ v.T)).sum())  # noqa: E731
    assert abs((loss(more) - loss(w64)) / 0.5 - dw64[5, 7]) <= 1e-9 * np.abs(dw64).max()


@pytest.mark.parametrize("m,n,k", [(8, 300, 5000), (200, 150, 900), (2400, 2400, 800)])
def test_waits_are_bounded(m, n, k, monkeypatch):
    """A copy that never comes: the kernel ends, says so, and the next call is whole."""
    a, b = operand(m, k, NV, 50), operand(n, k, NV, 51)
    want, out = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    dpg.dpg_fp4_product(a, b, want)
    torch.cuda.synchronize()
    monkeypatch.setenv("DPG_TEST_HOOKS", "1")
    assert dpg.lib().dpg_set_staged_fault(1, 20_000_000) == dpg.DPG_OK
    dpg.dpg_fp4_product(a, b, out)
    with pytest.raises(dpg.DpgError) as e:
        dpg.dpg_fp4_status()
    assert e.value.status == dpg.DPG_ERR_DEVICE_TIMEOUT
    dpg.dpg_fp4_status()
    dpg.dpg_fp4_product(a, b, out)
    assert torch.equal(want, out)
