"""Layer norm and its gradients on the GPU against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def half_step(t):
    return torch.finfo(t).eps / 2


def sum_depth(cols):
    """Roundings on the way of one term of a row's sum: at most 32 terms to a
    thread (cols / 1024 in long rows), then a tree of at most 10 levels, and the
    quotient."""
    return max(32, -(-cols // 1024)) + 12


def forward64(x, gain, bias, eps):
    mean = x.mean(1, keepdims=True)
    var = np.square(x - mean).mean(1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    n = (x - mean) * rstd
    y = n * (1 if gain is None else gain) + (0 if bias is None else bias)
    return y, mean, rstd, n, var


def check_forward(x, gain, bias, eps, y, mean, rstd):
    x64 = x.cpu().double().numpy()
    g64 = np.ones(x64.shape[1]) if gain is None else gain.cpu().double().numpy()
    b64 = np.zeros(x64.shape[1]) if bias is None else bias.cpu().double().numpy()
    want, m64, r64, n, var = forward64(x64, g64, b64, eps)
    d = sum_depth(x64.shape[1])
    dm = d * U * np.abs(x64).mean(1, keepdims=True)                  # of the mean
    # of the variance: the sum's roundings, the differences' own, and (mean - exact mean)^2
    dv = (d + 4) * U * var + np.square(dm) + 2 * U * np.abs(x64).max(1, keepdims=True) * np.sqrt(var)
    dr = r64 * (dv / (2 * (var + eps)) + 4 * U) + (np.square(dm) > var + eps) * r64
    dy = np.abs(g64) * (r64 * (dm + U * np.abs(x64 - m64)) + np.abs(x64 - m64) * dr + 3 * U * np.abs(n)) + U * np.abs(want)
    dy = dy * 1.05 + half_step(x.dtype) * np.abs(want) + 1e-37
    assert np.all(np.abs(y.cpu().double().numpy().reshape(x64.shape) - want) <= dy)
    if mean is not None:
        assert np.all(np.abs(mean.cpu().double().numpy()[:, None] - m64) <= dm * 1.05 + 1e-45)
        assert np.all(np.abs(rstd.cpu().double().numpy()[:, None] - r64) <= dr * 1.05)


def check_backward(dy, x, gain, mean, rstd, dx, dgain, dbias, before=(None, None)):
    y64, x64 = dy.cpu().double().numpy(), x.cpu().double().numpy()
    rows, cols = x64.shape
    g64 = np.ones(cols) if gain is None else gain.cpu().double().numpy()
    m, r = mean.cpu().double().numpy()[:, None], rstd.cpu().double().numpy()[:, None]
    n = (x64 - m) * r
    g = y64 * g64
    if dx is not None:
        c1, c2 = g.mean(1, keepdims=True), (g * n).mean(1, keepdims=True)
        want = r * (g - c1 - n * c2)
        d = sum_depth(cols)
        tol = r * U * (4 * np.abs(g) + (d + 4) * np.abs(g).mean(1, keepdims=True)
                       + np.abs(n) * ((d + 8) * np.abs(g * n).mean(1, keepdims=True) + 8 * np.abs(c2)))
        tol = tol * 1.05 + half_step(dx.dtype) * np.abs(want) + 1e-37
        assert np.all(np.abs(dx.cpu().double().numpy() - want) <= tol)
    # a column: rows one after the other (at most rows / parts of them, 304 parts or one per
    # row or per eight), eight warps, the parts, and n's own roundings
    depth = -(-rows // 304) + 8 + 10 + 5 + 4
    for got, term, old in ((dgain, y64 * n, before[0]), (dbias, y64, before[1])):
        if got is None:
            continue
        want = term.sum(0) + (0 if old is None else old)
        tol = depth * U * np.abs(term).sum(0) * 1.05 + half_step(got.dtype) * np.abs(want) + 1e-37
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= tol)


def make(rows, cols, dtype, seed=0, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * (0.5 + torch.rand(rows, 1, generator=g)) + offset * torch.randn(rows, 1, generator=g)
    return x.to(dtype).cuda()


COLS = [1, 2, 7, 8, 31, 64, 256, 257, 512, 513, 768, 1000, 1024, 1025, 2048, 2056, 4096, 5000, 8192, 8200, 16384,
        16390, 32768, 32776, 40001]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
def test_widths(cols, dtype):
    rows = 13
    x, dy = make(rows, cols, dtype, cols), make(rows, cols, dtype, cols + 1, 0.0) * 1e-2
    gain, bias = 1 + make(1, cols, dtype, 2)[0] * 0.1, make(1, cols, dtype, 3)[0]
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpg.dpg_layer_norm(x, gain, bias, EPS, y, mean, rstd)
    check_forward(x, gain, bias, EPS, y, mean, rstd)
    dx, dgain, dbias = torch.empty_like(x), torch.empty_like(gain), torch.empty_like(bias)
    ws = torch.full((dpg.dpg_layer_norm_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, dx, dgain, dbias, ws)
    check_backward(dy, x, gain, mean, rstd, dx, dgain, dbias)


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 303, 305, 2431, 2433, 5000])
@pytest.mark.parametrize("cols", [40, 1500])
def test_numbers_of_rows(rows, cols):
    x, dy = make(rows, cols, torch.bfloat16, rows), make(rows, cols, torch.bfloat16, rows + 1)
    gain = 1 + make(1, cols, torch.float32, 2)[0] * 0.1
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpg.dpg_layer_norm(x, gain, None, EPS, y, mean, rstd)
    check_forward(x, gain, None, EPS, y, mean, rstd)
    dgain, dbias = torch.full((cols,), 2.0, device="cuda"), torch.full((cols,), -3.0, device="cuda")
    dx = torch.empty_like(x)
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, dx, dgain, dbias, ws, accumulate=True)
    check_backward(dy, x, gain, mean, rstd, dx, dgain, dbias, (2.0, -3.0))


@pytest.mark.parametrize("cols", [768, 2000, 40000])
def test_parts_that_are_left_out(cols):
    rows = 40
    x, dy = make(rows, cols, torch.float32, 1), make(rows, cols, torch.float32, 2)
    gain = 1 + make(1, cols, torch.bfloat16, 3)[0]
    y, z = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpg.dpg_layer_norm(x, None, None, EPS, y)
    check_forward(x, None, None, EPS, y, None, None)
    dpg.dpg_layer_norm(x, gain, None, EPS, z, mean, rstd)
    check_forward(x, gain, None, EPS, z, mean, rstd)
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, dx, dg, db, ws)
    check_backward(dy, x, gain, mean, rstd, dx, dg, db)
    only = [torch.empty_like(t) for t in (dx, dg, db)]
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, only[0])
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, None, only[1], None, ws)
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, None, None, only[2], ws)
    for a, b in zip((dx, dg, db), only):
        assert torch.equal(a, b)
    dpg.dpg_layer_norm_backward(dy, x, None, mean, rstd, dx, dg, db, ws)
    check_backward(dy, x, None, mean, rstd, dx, dg, db)


@pytest.mark.parametrize("cols", [64, 1536, 40000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_slices_and_what_is_beside_them(cols, dtype):
    rows = 9

    def slice_of(n, fill=5.0):
        flat = torch.full((n + 16,), fill, dtype=dtype, device="cuda")
        return flat, flat[3:3 + n]

    (xf, x), (yf, y), (gf, gain), (bf, bias) = slice_of(rows * cols), slice_of(rows * cols), slice_of(cols), slice_of(cols)
    (df, dg), (ef, db) = slice_of(cols), slice_of(cols)
    src = make(rows, cols, dtype, 4)
    x.copy_(src.view(-1))
    gain.copy_(1 + make(1, cols, dtype, 5)[0] * 0.1)
    x, y = x.view(rows, cols), y.view(rows, cols)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpg.dpg_layer_norm(x, gain, bias, EPS, y, mean, rstd)
    check_forward(x, gain, bias, EPS, y, mean, rstd)
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dy = make(rows, cols, dtype, 6)
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, y, dg, db, ws)
    check_backward(dy, x, gain, mean, rstd, y, dg, db)
    for f, s in ((xf, x), (yf, y), (gf, gain), (bf, bias), (df, dg), (ef, db)):
        s.fill_(5.0)
        assert (f == 5.0).all()


@pytest.mark.parametrize("cols", [64, 1024, 4096, 40000])
def test_in_place(cols):
    rows = 21
    x, dy = make(rows, cols, torch.bfloat16, 7), make(rows, cols, torch.bfloat16, 8)
    gain = 1 + make(1, cols, torch.bfloat16, 9)[0] * 0.1
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpg.dpg_layer_norm(x, gain, None, EPS, y, mean, rstd)
    z = x.clone()
    dpg.dpg_layer_norm(z, gain, None, EPS, z)
    assert torch.equal(y, z)
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")]
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, *out, ws)
    for which in (0, 1):
        a, b = dy.clone(), x.clone()
        got = [a if which == 0 else b, torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")]
        dpg.dpg_layer_norm_backward(a, b, gain, mean, rstd, *got, ws)
        assert all(torch.equal(p, q) for p, q in zip(out, got))


def test_rows_that_are_not_finite_and_constant_rows():
    for cols in (96, 3000, 40000):
        x = make(6, cols, torch.float32, 10)
        x[1, 5], x[2, 0], x[4] = float("nan"), float("inf"), 3.25
        y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
        dpg.dpg_layer_norm(x, None, None, EPS, y, mean, rstd)
        assert y[1].isnan().all() and y[2].isnan().all()
        assert not y[4].any() and abs(float(rstd[4]) * EPS ** 0.5 - 1) < 1e-6
        keep = [0, 3, 5]
        check_forward(x[keep], None, None, EPS, y[keep], mean[keep], rstd[keep])


def test_large_means():
    # fp32 keeps what is left of values of 1000 +- 1e-3
    x = (1000 + 1e-3 * torch.randn(5, 768, generator=torch.Generator().manual_seed(1))).cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    dpg.dpg_layer_norm(x, None, None, 0.0, y, mean, rstd)
    check_forward(x, None, None, 0.0, y, mean, rstd)


def test_rows_of_no_elements_and_no_rows():
    e = torch.empty(0, 64, device="cuda")
    v = torch.ones(64, device="cuda")
    dpg.dpg_layer_norm(e, v, v, EPS, e)
    dg, db = torch.full((64,), 4.0, device="cuda"), torch.full((64,), 4.0, device="cuda")
    ws = torch.empty(dpg.dpg_layer_norm_workspace(0, 64), dtype=torch.uint8, device="cuda")
    none = torch.empty(0, device="cuda")
    dpg.dpg_layer_norm_backward(e, e, v, none, none, e, dg, db, ws, accumulate=True)
    assert (dg == 4.0).all()
    dpg.dpg_layer_norm_backward(e, e, v, none, none, e, dg, db, ws)
    assert not dg.any() and not db.any()


def test_gradients_against_differences():
    """Of a weighted sum of y, by central differences of the 64-bit formula."""
    rows, cols = 5, 24
    x, dy = make(rows, cols, torch.float32, 11), make(rows, cols, torch.float32, 12)
    gain, bias = 1 + make(1, cols, torch.float32, 13)[0] * 0.1, make(1, cols, torch.float32, 14)[0]
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpg.dpg_layer_norm(x, gain, bias, EPS, y, mean, rstd)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gain), torch.empty_like(bias)
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, dx, dg, db, ws)
    arrays = [t.cpu().double().numpy() for t in (x, gain, bias)]
    w = dy.cpu().double().numpy()
    loss = lambda a: float((w * forward64(a[0], a[1], a[2], EPS)[0]).sum())  # noqa: E731
    h = 1e-4
    for k, got in enumerate((dx, dg, db)):
        got = got.cpu().double().numpy()
        for at in np.ndindex(arrays[k].shape):
            ends = []
            for s in (h, -h):
                a = [v.copy() for v in arrays]
                a[k][at] += s
                ends.append(loss(a))
            # third derivatives of order 10 leave h^2, binary64 1e-13 / h, the kernel 1e-5 of its terms
            assert abs((ends[0] - ends[1]) / (2 * h) - got[at]) <= 2e-5 * max(1.0, np.abs(got).max())


def test_same_bits_on_every_call_on_two_streams_and_in_a_graph():
    rows, cols = 3000, 768
    x, dy = make(rows, cols, torch.bfloat16, 15), make(rows, cols, torch.bfloat16, 16)
    gain = 1 + make(1, cols, torch.bfloat16, 17)[0] * 0.1

    def buffers():
        return dict(y=torch.empty_like(x), mean=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"),
                    dx=torch.empty_like(x), dg=torch.empty(cols, device="cuda"), db=torch.empty(cols, device="cuda"),
                    ws=torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda"))

    def step(b, stream=None):
        dpg.dpg_layer_norm(x, gain, None, EPS, b["y"], b["mean"], b["rstd"], stream=stream)
        dpg.dpg_layer_norm_backward(dy, x, gain, b["mean"], b["rstd"], b["dx"], b["dg"], b["db"], b["ws"], stream=stream)

    def same(a, b):
        return all(torch.equal(a[k], b[k]) for k in a if k != "ws")

    want, one, two, cap = buffers(), buffers(), buffers(), buffers()
    step(want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        step(one, streams[0])
        step(two, streams[1])
    torch.cuda.synchronize()
    assert same(want, one) and same(want, two)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        step(cap)
    graph.replay()
    torch.cuda.synchronize()
    assert same(want, cap)


def test_gradients_into_slices_of_a_plan():
    """Gradients of a norm's parameters left where the step reads them."""
    cols, R, rows = 72, 2, 50
    plan = dpg.dpg_plan_buckets([cols, cols], 1 << 20, R)
    n = plan.total_padded
    grads = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(R)]
    gain_at, bias_at = (slice(int(o), int(o) + cols) for o in plan.param_offset)
    master = torch.zeros(n, device="cuda")
    master[gain_at] = 1.0
    view = master.to(torch.bfloat16)
    ws = torch.empty(dpg.dpg_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    want = 0.0
    for r in range(R):
        x, dy = make(rows, cols, torch.bfloat16, r), make(rows, cols, torch.bfloat16, 9 + r)
        y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dpg.dpg_layer_norm(x, view[gain_at], view[bias_at], EPS, y, mean, rstd)
        dpg.dpg_layer_norm_backward(dy, x, view[gain_at], mean, rstd, None, grads[r][gain_at], grads[r][bias_at], ws)
        check_backward(dy, x, view[gain_at], mean, rstd, None, grads[r][gain_at], grads[r][bias_at])
        want = want + grads[r].double()
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    dpg.dpg_step(plan, grads, [rows] * R, dpg.HParams(lr=1e-2, step=1), master, m, v, [view])
    # Adam's first step moves each weight by lr against its gradient's sign
    moved = master[bias_at].double()
    g = want[bias_at]
    assert torch.all((moved.sign() == -g.sign()) | (g.abs() < 1e-4))
