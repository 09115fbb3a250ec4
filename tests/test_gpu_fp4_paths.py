"""Every path of the 4-bit products and of the quantisation, on each side of the
sizes at which another is taken, against the 64-bit forms."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import MX, NV, product_bound, quantized, spread, unpacked, values_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    dpg.dpg_fp4_status()


def operand(rows, cols, fmt, seed):
    q = dpg.Fp4(rows, cols, fmt)
    dpg.dpg_fp4_quantize(spread(rows, cols, seed, torch.bfloat16).cuda(), q)
    return q


# the sum of a tile of 128 x 16, 32, 64 or 128 in one, two, four and eight parts; 37 and 38,
# 75 and 77 tiles of 256 x 256, of which the second numbers (38: with long sums) take pairs of
# CTAs; one row more than a tile
PATHS = [
    (16, 14000, 2100), (13, 4000, 4100), (16, 9000, 4100), (3, 700, 4300), (17, 4000, 2300), (32, 9000, 4000),
    (64, 9000, 4100), (33, 2300, 4096), (64, 16000, 300), (9000, 40, 4100),
    (700, 640, 1000), (1024, 896, 4200), (640, 640, 4100), (130, 200, 4352), (129, 65, 9000), (65, 129, 8193),
    (256, 9472, 300), (512, 4864, 300), (128, 9800, 300), (4864, 257, 260),
    (256, 9472, 2100), (512, 4864, 2100), (4864, 257, 2111), (256, 19200, 130), (256, 19457, 130),
]


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("m,n,k", PATHS)
@pytest.mark.parametrize("pad", [0, 3])
def test_products(m, n, k, pad, fmt):
    a, b = operand(m, k, fmt, 1), operand(n, k, fmt, 2)
    av, bv = values_of(a), values_of(b)
    want = torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().T
    for dtype, add in ((torch.bfloat16, False), (torch.float32, False), (torch.float32, True)):
        flat = torch.full((m * (n + pad),), 0.25, device="cuda", dtype=dtype)
        out = flat.as_strided((m, n), (n + pad, 1))
        dpg.dpg_fp4_product(a, b, out, accumulate=add)
        full = want + 0.25 if add else want
        # the product's bound, and two roundings to fp32 of the sum with 1/4
        bound = product_bound(av, bv, dtype, want.cpu().numpy()) + (2.0 ** -23 * (0.25 + np.abs(want.cpu().numpy())) if add else 0)
        assert np.all((out.double() - full).abs().cpu().numpy() <= bound)
        out.fill_(0.25)
        assert (flat == 0.25).all()                            # nothing beside the rows


def same(q, x, seed=None, side=0):
    codes, scales, values = quantized(x, q.format, seed, side)
    c, s, c_pad, s_pad = unpacked(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.rows, q.cols, q.format)
    np.testing.assert_array_equal(s, scales)
    np.testing.assert_array_equal(np.where(x == 0, c & 7, c), np.where(x == 0, 0, codes))   # of -0: either zero
    assert not c_pad.any() and not s_pad.any()


# more than eight tiles of 128 x 128: the largest magnitude comes from a kernel before
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,stride", [(0, 400), (1, 400), (0, 408), (8, 408), (3, 417)])
@pytest.mark.parametrize("bad", [False, True])
def test_quantisation_of_many_tiles(bad, offset, stride, dtype):
    rows, cols = 390, 400
    flat = spread(1, offset + rows * stride, 3, dtype).view(-1)
    flat[:offset] = 1e30                                       # beside the matrix: no part of it
    x = flat[offset:].as_strided((rows, cols), (stride, 1))
    if stride > cols:
        flat[offset:].as_strided((rows - 1, stride - cols), (stride, 1), offset + cols).fill_(float("inf"))
    # the largest of all where a row's first, or last, elements are looked at singly
    x[rows - 1, cols - 1] = 7.0
    if bad:
        x[5, 0], x[17, 399], x[300, 200] = float("inf"), float("nan"), float("-inf")
    dev = flat.cuda()
    view = dev[offset:].as_strided((rows, cols), (stride, 1))
    for top in (False, True):
        if top:
            view[0, 0] = -11.0
            x[0, 0] = -11.0
        row, col = dpg.Fp4(rows, cols), dpg.Fp4(cols, rows)
        dpg.dpg_fp4_quantize(view, row, col)
        assert row.amax[0].item() == col.amax[0].item() == (11.0 if top else 7.0)
        same(row, x.double().numpy())
        same(col, x.double().numpy().T)


@pytest.mark.parametrize("fmt", [NV, MX])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-3, 1e-38, 3e36])
def test_stochastic_codes_of_many_tiles(scale, dtype, fmt):
    x = spread(260, 390, 5, torch.float32, 1.0).clamp(-30, 30).mul(scale).to(dtype)
    row, col = dpg.Fp4(260, 390, fmt), dpg.Fp4(390, 260, fmt)
    dpg.dpg_fp4_quantize(x.cuda(), row, col, seed=torch.tensor([(5 << 40) + 3], device="cuda"))
    same(row, x.double().numpy(), (5 << 40) + 3, 0)
    same(col, x.double().numpy().T, (5 << 40) + 3, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_stochastic_codes_at_their_thresholds(dtype):
    """Elements on, and one place beside, the values that go up or not.  The matrix
    is laid out so that each element's place between its neighbours is just its own
    threshold (fp32), or as near as bf16 comes to it."""
    from fp4_util import LEVELS, philox
    rows, cols, seed = 40, 64, 77
    u = philox(seed, 0, rows, cols)
    lo = LEVELS[np.arange(rows * cols).reshape(rows, cols) % 7]
    hi = LEVELS[np.arange(rows * cols).reshape(rows, cols) % 7 + 1]
    at = lo + (2 * u + 1) * 2.0 ** -17 * (hi - lo)
    x = torch.from_numpy(at).to(dtype)
    assert dtype != torch.float32 or np.array_equal(x.double().numpy(), at)     # 16 bits and a value: exact
    x[:, ::16] = 6.0                                           # every block's scale is 1 (of a matrix with 2^e = 1: 448)
    x[0, 0] = 2688.0
    for k, step in enumerate((0, 1, -1)):
        y = x.clone()
        if step:
            up = torch.nextafter(x, torch.full_like(x, float("inf") if step > 0 else 0.0))
            y = torch.where((x < 6.0), up, x)
        row = dpg.Fp4(rows, cols)
        dpg.dpg_fp4_quantize(y.cuda(), row, seed=torch.tensor([seed], device="cuda"))
        same(row, y.double().numpy(), seed, 0)


def test_two_graphs_that_share_buffers():
    """Two captured chains, replayed in turn, of which each leaves the other's
    quantised matrices, sums and workspaces overwritten."""
    t, d, h = 384, 256, 512
    x = [spread(t, d, 10 + k, torch.bfloat16, 1.0).cuda() for k in range(2)]
    w, row, col = dpg.Fp4(h, d), dpg.Fp4(t, d), dpg.Fp4(d, t)
    dpg.dpg_fp4_quantize(spread(h, d, 13, torch.bfloat16).cuda(), w)
    gain, bias = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    n, mean, rstd = torch.empty_like(x[0]), torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dx = torch.empty_like(n)
    ws = torch.empty(dpg.dpg_layer_norm_workspace(t, d), dtype=torch.uint8, device="cuda")
    out = [torch.empty(t, h, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    grad = [torch.zeros(2, d, device="cuda") for _ in range(2)]

    def chain(k):
        dpg.dpg_layer_norm(x[k], gain, bias, 1e-5, n, mean, rstd)
        dpg.dpg_fp4_quantize(n, row, col)
        dpg.dpg_fp4_product(row, w, out[k])
        dpg.dpg_layer_norm_backward(n, x[k], gain, mean, rstd, dx, grad[k][0], grad[k][1], ws)

    want = []
    for k in range(2):
        chain(k)
        want.append((out[k].clone(), grad[k].clone()))
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            chain(k)
        graphs.append(g)
    for k in (0, 1, 1, 0, 1):
        out[k].zero_()
        grad[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[k], want[k][0]) and torch.equal(grad[k], want[k][1])


def test_values_of_many_rows():
    """Dequantised rows that start anywhere, in both types, beside what they leave."""
    q = dpg.Fp4(300, 415)
    dpg.dpg_fp4_quantize(spread(300, 415, 21, torch.float32, 1.0).cuda(), q)
    want = values_of(q)
    for dtype in (torch.bfloat16, torch.float32):
        for offset, stride in ((0, 416), (2, 415), (16, 432), (5, 421)):
            flat = torch.full((offset + 300 * stride + 32,), 9.0, device="cuda", dtype=dtype)
            out = flat[offset:].as_strided((300, 415), (stride, 1))
            dpg.dpg_fp4_dequantize(q, out)
            np.testing.assert_array_equal(out.cpu().double().numpy(), want)
            out.fill_(9.0)
            assert (flat == 9.0).all()


@pytest.mark.parametrize("pad", [0, 1])
def test_results_beyond_32_bits(pad):
    """Offsets in C, and in a quantised and a dequantised matrix, of more than 2^31 elements."""
    m, n, k = 66000, 32768, 64
    a, b = operand(256, k, NV, 31), operand(n, k, NV, 32)
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    dpg.dpg_fp4_dequantize(a, x[-256:])
    many = dpg.Fp4(m, k)
    dpg.dpg_fp4_quantize(x, many)
    c = torch.empty(m * (n + pad), dtype=torch.bfloat16, device="cuda").as_strided((m, n), (n + pad, 1))
    dpg.dpg_fp4_product(many, b, c)
    av, bv = values_of(a), values_of(b)
    assert not c[:-256].any()
    want = torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().T
    bound = product_bound(av, bv, torch.bfloat16, want.cpu().numpy())
    assert np.all((c[-256:].double() - want).abs().cpu().numpy() <= bound)
    back, forth = dpg.Fp4(m, n), torch.empty_like(c)
    dpg.dpg_fp4_quantize(c, back)
    dpg.dpg_fp4_dequantize(back, forth)
    few = dpg.Fp4(256, n)
    dpg.dpg_fp4_quantize(c[-256:], few)
    some = torch.empty(256, n, dtype=torch.bfloat16, device="cuda")
    dpg.dpg_fp4_dequantize(few, some)
    assert torch.equal(forth[-256:], some) and not forth[:-256].any()
