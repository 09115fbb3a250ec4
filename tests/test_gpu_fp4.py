"""4-bit quantisation on the GPU against its 64-bit form: every code, scale and
value has to be equal."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import E4M3, LEVELS, MX, NV, block_of, quantized, spread, unpacked, values_of

pytestmark = pytest.mark.gpu
FORMATS = [NV, MX]
SHAPES = [(1, 1), (1, 7), (7, 1), (1, 16), (3, 33), (32, 64), (129, 65), (128, 128), (257, 130), (100, 300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def check(q, x, seed=None, side=0):
    """The stored bytes of q against the form of the float64 matrix x."""
    codes, scales, values = quantized(x, q.format, seed, side)
    c, s, c_pad, s_pad = unpacked(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.rows, q.cols, q.format)
    np.testing.assert_array_equal(s, scales)
    np.testing.assert_array_equal(np.where(x == 0, c & 7, c), np.where(x == 0, 0, codes))   # of -0: either zero
    assert not c_pad.any() and not s_pad.any()
    np.testing.assert_array_equal(values_of(q), values)


def run(x, fmt, seed=None, sides="both"):
    r, c = x.shape
    row = dpg.Fp4(r, c, fmt) if sides != "col" else None
    col = dpg.Fp4(c, r, fmt) if sides != "row" else None
    for q in (row, col):
        if q is not None:              # what is not written shows
            q.codes.fill_(0xA5)
            q.scales.fill_(0xA5)
    t = None if seed is None else torch.tensor([seed], device="cuda")
    dpg.dpg_fp4_quantize(x, row, col, seed=t)
    torch.cuda.synchronize()
    return row, col


def check_both(x, fmt, seed=None, sides="both"):
    row, col = run(x.cuda(), fmt, seed, sides)
    x64 = x.double().cpu().numpy()
    if row is not None:
        check(row, x64, seed, 0)
    if col is not None:
        check(col, x64.T, seed, 1)
    return row, col


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_nearest(rows, cols, fmt, dtype):
    check_both(spread(rows, cols, rows * 1000 + cols, dtype), fmt)


@pytest.mark.parametrize("sides", ["row", "col"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_one_orientation(fmt, sides):
    check_both(spread(130, 200, 1, torch.bfloat16), fmt, None, sides)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (33, 70), (130, 20)])
def test_stochastic(rows, cols, fmt, dtype):
    check_both(spread(rows, cols, rows * 1000 + cols, dtype), fmt, -(1 << 62) + 987654321)


def test_stochastic_is_unbiased():
    # 4096 copies of values between 2 and 3 and between 4 and 6: the mean of n draws of a
    # gap g is within 5 g / (2 sqrt(n)) of the value but for once in a million
    x = torch.full((4096, 16), 2.25)
    x[:, 0], x[:, 1], x[:, 2] = 6.0, 4.5, 0.1
    q, _ = run(x.cuda(), NV, 3, "row")
    m = values_of(q).mean(0)
    for c, g in ((1, 2.0), (2, 0.5), (5, 1.0)):
        assert abs(m[c] - float(x[0, c])) <= 5 * g / (2 * 64) + 2.0 ** -16


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties_and_values_beside_them(fmt):
    # every borderline of every scale (E4M3: fraction 1, 1.125, .. 1.875), and its fp32 neighbours
    b = block_of(fmt)
    rows = []
    for s in ([1.0, 2.0 ** -20, 2.0 ** 30] if fmt == MX else E4M3[[8 + 8 * 6 + k for k in range(8)]]):
        mid = (LEVELS[1:] + LEVELS[:-1]) / 2 * s
        for step in (-1, 0, 1):
            v = mid.astype(np.float32).view(np.int32) + step
            row = np.zeros(b, np.float32)
            row[0] = 6 * s
            row[1:8] = v.view(np.float32)
            row[8:15] = -v.view(np.float32)
            rows.append(row)
    if fmt == NV:                       # e = 0
        rows.append(np.array([2688.0] + [0.0] * (b - 1), np.float32))
    x = torch.from_numpy(np.stack(rows))
    check_both(x, fmt)
    check_both(x.to(torch.bfloat16), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 3e37, 1e-42])
def test_magnitudes(fmt, scale):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 70, generator=g).clamp(-10, 10)
    check_both((x.double() * scale).float(), fmt)
    check_both((x.double() * scale).to(torch.bfloat16), fmt)


@pytest.mark.parametrize("top", [2688.0, 2688.0 * (1 + 2.0 ** -23), 2688.0 * (1 - 2.0 ** -24), 1.3125 * 2.0 ** 100,
                                 3.4e38, 2.0 ** -126, 2.0 ** -149])
def test_powers_of_two_of_a_matrix(top):
    x = torch.zeros(3, 40)
    x[1, 3] = top
    x[2, 20:30] = top / 3
    x[0, 1] = -top / 1000
    check_both(x, NV)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_that_are_not_finite(fmt, dtype):
    x = spread(70, 100, 3, dtype)
    x[5, 40], x[6, 0], x[69, 99], x[20, 50] = float("nan"), float("inf"), float("-inf"), float("nan")
    x[30, :] = 0.0
    x[31, 3] = -0.0
    for seed in (None, 11):
        row, _ = check_both(x, fmt, seed)
        assert np.isnan(values_of(row)).any(1).sum() == 4          # in their rows only
        out = torch.empty(70, 100, device="cuda")
        dpg.dpg_fp4_dequantize(row, out)
        np.testing.assert_array_equal(out.cpu().double().numpy(), values_of(row))


def test_matrix_of_zeros_and_of_nans():
    check_both(torch.zeros(20, 40), NV)
    check_both(torch.zeros(20, 40), MX)
    check_both(torch.full((20, 40), float("nan")), NV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("offset,stride,cols", [(0, 200, 130), (1, 200, 130), (8, 131, 131), (0, 130, 130), (3, 333, 16)])
def test_strided_and_unaligned_inputs(offset, stride, cols, fmt, dtype):
    rows = 140
    flat = spread(1, offset + rows * stride, 9, dtype).cuda().view(-1)
    x = flat[offset:].as_strided((rows, cols), (stride, 1))
    row, col = run(x, fmt)
    check(row, x.double().cpu().numpy())
    check(col, x.double().cpu().numpy().T)


def test_one_row_of_any_stride():
    flat = spread(1, 64, 2, torch.bfloat16).cuda()
    row, _ = run(flat.as_strided((1, 64), (3, 1)), NV)
    check(row, flat.double().cpu().numpy())


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("offset,stride", [(0, 70), (1, 70), (8, 80), (0, 72)])
def test_dequantize(offset, stride, fmt, out_dtype):
    x = spread(33, 70, 4, torch.float32)
    row, _ = run(x.cuda(), fmt)
    flat = torch.full((offset + 33 * stride + 8,), 7.0, dtype=out_dtype, device="cuda")
    out = flat[offset:].as_strided((33, 70), (stride, 1))
    dpg.dpg_fp4_dequantize(row, out)
    np.testing.assert_array_equal(out.cpu().double().numpy(), values_of(row))
    out.fill_(7.0)
    assert (flat == 7.0).all()                                     # nothing else was written


def test_scales_of_a_large_matrix_beyond_32_bits():
    # 2^31 + elements: the last rows of a matrix whose codes pass 2^30 bytes
    rows, cols = 65600, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = spread(70, cols, 6, torch.bfloat16).cuda()
    x[-70:] = tail
    q = dpg.Fp4(rows, cols, MX)
    dpg.dpg_fp4_quantize(x, q)
    out = torch.empty_like(x)
    dpg.dpg_fp4_dequantize(q, out)
    few = dpg.Fp4(70, cols, MX)
    dpg.dpg_fp4_quantize(tail, few)
    want = torch.empty_like(tail)
    dpg.dpg_fp4_dequantize(few, want)
    assert torch.equal(out[-70:], want) and not out[:-70].any()


def test_masters_of_a_plan():
    shapes, counts = [(40, 70), (33, 20), (5, 1)], [1, 2, 3]
    plan = dpg.dpg_plan_buckets([r * c * k for (r, c), k in zip(shapes, counts)], 1 << 30, 4)
    mats = dpg.dpg_plan_matrices(plan, [s[0] for s in shapes], [s[1] for s in shapes])
    master = spread(1, plan.total_padded, 8, torch.float32).view(-1).cuda()
    each = [(i, k) for i in range(3) for k in range(counts[i])]
    for fmt in FORMATS:
        for seed in (None, 41):
            rows = [dpg.Fp4(*shapes[i], fmt) for i, _ in each]
            cols = [dpg.Fp4(*shapes[i][::-1], fmt) for i, _ in each]
            t = None if seed is None else torch.tensor([seed], device="cuda")
            dpg.dpg_allgather_params_fp4(mats, master, rows, cols, seed=t)
            only = [dpg.Fp4(*shapes[i][::-1], fmt) for i, _ in each]
            dpg.dpg_allgather_params_fp4(mats, master, None, only, seed=t)
            for n, (i, k) in enumerate(each):
                r, c = shapes[i]
                at = int(plan.param_offset[i]) + k * r * c
                x = master[at:at + r * c].view(r, c).double().cpu().numpy()
                s = None if seed is None else seed + n
                check(rows[n], x, s, 0)
                check(cols[n], x.T, s, 1)
                check(only[n], x.T, s, 1)


def test_replayed_graph_reads_the_seed_and_the_input():
    x = spread(70, 100, 12, torch.bfloat16).cuda()
    seed = torch.tensor([1], device="cuda")
    row, col = dpg.Fp4(70, 100), dpg.Fp4(100, 70)
    dpg.dpg_fp4_quantize(x, row, col, seed=seed)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        dpg.dpg_fp4_quantize(x, row, col, seed=seed)
    for n in (5, 6):
        seed.fill_(n)
        x.copy_(spread(70, 100, n, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        check(row, x.double().cpu().numpy(), n, 0)
        check(col, x.double().cpu().numpy().T, n, 1)


def test_two_streams_at_once():
    xs = [spread(1000, 1500, n, torch.bfloat16).cuda() for n in range(2)]
    want = [run(x, NV) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(dpg.Fp4(1000, 1500), dpg.Fp4(1500, 1000)) for _ in xs]
        torch.cuda.synchronize()
        for s, x, q in zip(streams, xs, got):
            dpg.dpg_fp4_quantize(x, *q, stream=s)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for p, q in zip(a, b):
                assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales) and torch.equal(p.amax[0], q.amax[0])
