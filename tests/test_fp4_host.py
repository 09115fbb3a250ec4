"""Host-side checks of the 4-bit matrices (no GPU): sizes, the test's own plain
form, and every refusal, which comes before any device work."""
import ctypes

import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import E4M3, MX, NV, philox, quantized, unpacked

BUF = 1 << 20   # an aligned address that is never read: the calls stop before
INVALID, MISALIGNED = dpg.DPG_ERR_INVALID_ARG, dpg.DPG_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def sizes(rows, cols, fmt):
    a, b = ctypes.c_int64(-1), ctypes.c_int64(-1)
    st = dpg.lib().dpg_fp4_sizes(rows, cols, fmt, ctypes.byref(a), ctypes.byref(b))
    return st, a.value, b.value


@pytest.mark.parametrize("rows,cols,fmt,codes,scales", [
    (0, 0, NV, 0, 0), (1, 1, NV, 16, 512), (1, 64, NV, 32, 512), (128, 65, NV, 128 * 48, 1024),
    (129, 64, MX, 129 * 32, 1024), (129, 129, MX, 129 * 80, 2048), (5, 0, MX, 0, 0), (0, 5, NV, 0, 0),
    (1 << 30, 32, MX, 1 << 34, 1 << 32),
])
def test_sizes(rows, cols, fmt, codes, scales):
    assert sizes(rows, cols, fmt) == (dpg.DPG_OK, codes, scales)


@pytest.mark.parametrize("rows,cols,fmt", [(-1, 4, NV), (4, -1, NV), ((1 << 30) + 1, 1, NV), (1, (1 << 30) + 1, MX),
                                           (4, 4, 2), (4, 4, -1)])
def test_sizes_refused(rows, cols, fmt):
    assert sizes(rows, cols, fmt)[0] == INVALID
    assert dpg.lib().dpg_fp4_sizes(1, 1, NV, None, None) == dpg.DPG_OK


def test_plain_form_on_known_blocks():
    # 6 * 448 * 2^0 is the largest magnitude with e = 0
    x = np.zeros((1, 16))
    x[0, 0] = 2688.0
    codes, scales, values = quantized(x, NV)
    assert scales[0, 0] == 0x7E and codes[0, 0] == 7 and values[0, 0] == 2688.0
    x[0, 1] = -448 * 2.5
    codes, _, values = quantized(x, NV)
    assert codes[0, 1] == 8 + 4 and values[0, 1] == -896.0          # a tie goes to the even code
    y = np.zeros((1, 32))
    y[0, 0] = 6.1
    assert quantized(y, MX)[1][0, 0] == 128                        # 6 * 2^0 < 6.1 <= 6 * 2^1
    assert E4M3[0x7E] == 448 and E4M3[8] == 2.0 ** -6


def test_philox_known_answers():
    # Salmon et al. 2011, known answers of Philox4x32-10 for counter and key of zeros
    u = philox(0, 0, 1, 8)[0]
    words = [int(u[2 * j]) | int(u[2 * j + 1]) << 16 for j in range(4)]
    assert words == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def test_layout_of_scales():
    raw = np.zeros((2, 1, 512), np.uint8)
    raw[1, 0, (37 % 32) * 16 + (37 // 32) * 4 + 2] = 9             # row 128 + 37, block 2
    _, s, _, _ = unpacked(np.zeros(200 * 32, np.uint8), raw, 200, 64, NV)
    assert s[165, 2] == 9 and s.sum() == 9


class Q:
    """A quantised matrix at addresses that are never read."""

    def __init__(self, rows=4, cols=64, fmt=NV, codes=BUF, scales=2 * BUF, amax=3 * BUF):
        self.c = dpg.dpg_fp4(codes, scales, amax, rows, cols, fmt)
        self.ref = ctypes.byref(self.c)


def refused(status, text, fn, *args):
    before = dpg.dpg_launch_count()
    assert fn(*args) == status, dpg.lib().dpg_last_error()
    assert text.encode() in dpg.lib().dpg_last_error(), dpg.lib().dpg_last_error()
    assert dpg.dpg_launch_count() == before


@pytest.mark.parametrize("kw,status,text", [
    (dict(row=None), INVALID, "by_row and by_col are NULL"),
    (dict(row=Q(5, 64)), INVALID, "by_row is 5 x 64"),
    (dict(row=Q(64, 4)), INVALID, "by_row is 64 x 4"),
    (dict(row=None, col=Q(4, 64)), INVALID, "by_col is 4 x 64"),
    (dict(row=Q(fmt=7)), INVALID, "format 7"),
    (dict(row=Q(-4)), INVALID, "outside"),
    (dict(row=Q(codes=None)), INVALID, "by_row.codes is NULL"),
    (dict(row=Q(scales=None)), INVALID, "by_row.scales is NULL"),
    (dict(row=Q(amax=None)), INVALID, "by_row.amax is NULL"),
    (dict(row=Q(codes=BUF + 8)), MISALIGNED, "by_row.codes"),
    (dict(row=Q(scales=BUF + 8)), MISALIGNED, "by_row.scales"),
    (dict(row=Q(amax=BUF + 2)), MISALIGNED, "by_row.amax"),
    (dict(col=Q(64, 4, MX, BUF * 4, BUF * 5)), INVALID, "different formats"),
    (dict(col=Q(64, 4, NV, BUF, BUF * 5)), INVALID, "share a buffer"),
    (dict(col=Q(64, 4, NV, BUF * 4, 2 * BUF)), INVALID, "share a buffer"),
    (dict(dtype=2), INVALID, "dtype 2"),
    (dict(x=None), INVALID, "x is NULL"),
    (dict(x=BUF + 1), MISALIGNED, "x misaligned"),
    (dict(x=BUF + 2, dtype=dpg.DPG_F32), MISALIGNED, "x misaligned"),
    (dict(stride=63), INVALID, "row stride 63"),
    (dict(stride=-64), INVALID, "row stride -64"),
    (dict(seed=BUF + 4), MISALIGNED, "seed"),
])
def test_quantize_refusals(kw, status, text):
    row, col = kw.get("row", Q()), kw.get("col")
    refused(status, text, dpg.lib().dpg_fp4_quantize, kw.get("x", BUF), kw.get("dtype", dpg.DPG_BF16), 4, 64,
            kw.get("stride", 64), kw.get("seed"), row and row.ref, col and col.ref, None)


def test_nothing_to_quantize():
    L = dpg.lib()
    before = dpg.dpg_launch_count()
    for r, c in ((0, 64), (64, 0), (0, 0)):
        q, t = Q(r, c, NV, None, None, None), Q(c, r, NV, None, None, None)
        assert L.dpg_fp4_quantize(None, dpg.DPG_F32, r, c, c, None, q.ref, t.ref, None) == dpg.DPG_OK
        assert L.dpg_fp4_dequantize(q.ref, None, dpg.DPG_F32, c, None) == dpg.DPG_OK
    assert dpg.dpg_launch_count() == before


@pytest.mark.parametrize("kw,status,text", [
    (dict(q=None), INVALID, "q is NULL"),
    (dict(q=Q(codes=None)), INVALID, "q.codes"),
    (dict(out=None), INVALID, "out is NULL"),
    (dict(out=BUF + 1), MISALIGNED, "out misaligned"),
    (dict(dtype=5), INVALID, "dtype 5"),
    (dict(stride=10), INVALID, "row stride 10"),
])
def test_dequantize_refusals(kw, status, text):
    q = kw.get("q", Q())
    refused(status, text, dpg.lib().dpg_fp4_dequantize, q and q.ref, kw.get("out", BUF), kw.get("dtype", dpg.DPG_BF16),
            kw.get("stride", 64), None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(a=None), INVALID, "a is NULL"),
    (dict(b=None), INVALID, "b is NULL"),
    (dict(b=Q(7, 64, MX)), INVALID, "different formats"),
    (dict(b=Q(7, 65)), INVALID, "sums over 64 and 65"),
    (dict(a=Q(codes=None)), INVALID, "a.codes"),
    (dict(b=Q(7, 64, scales=2 * BUF + 4)), MISALIGNED, "b.scales"),
    (dict(c=None), INVALID, "c is NULL"),
    (dict(c=BUF + 1), MISALIGNED, "c misaligned"),
    (dict(c=BUF + 2, dtype=dpg.DPG_F32), MISALIGNED, "c misaligned"),
    (dict(dtype=9), INVALID, "dtype 9"),
    (dict(add=1), INVALID, "only an fp32 c"),
    (dict(stride=6), INVALID, "row stride 6"),
])
def test_product_refusals(kw, status, text):
    a, b = kw.get("a", Q()), kw.get("b", Q(7, 64))
    refused(status, text, dpg.lib().dpg_fp4_product, a and a.ref, b and b.ref, kw.get("c", BUF),
            kw.get("dtype", dpg.DPG_BF16), kw.get("stride", 7), kw.get("add", 0), None)


def test_empty_products():
    L = dpg.lib()
    before = dpg.dpg_launch_count()
    none = Q(0, 64, NV, None, None, None)
    assert L.dpg_fp4_product(none.ref, Q(7, 64).ref, None, dpg.DPG_BF16, 7, 0, None) == dpg.DPG_OK
    assert L.dpg_fp4_product(Q().ref, none.ref, None, dpg.DPG_BF16, 0, 0, None) == dpg.DPG_OK
    # a sum over nothing leaves an accumulator as it is
    x, w = Q(4, 0, NV, None, None, None), Q(7, 0, NV, None, None, None)
    assert L.dpg_fp4_product(x.ref, w.ref, BUF, dpg.DPG_F32, 7, 1, None) == dpg.DPG_OK
    assert dpg.dpg_launch_count() == before


def test_allgather_refusals():
    plan = dpg.dpg_plan_buckets([24, 2 * 15], 1 << 30, 1)
    mats = dpg.dpg_plan_matrices(plan, [4, 3], [6, 5])             # 4 x 6, and two of 3 x 5
    L = dpg.lib()

    def arrays(shapes, **kw):
        return (dpg.dpg_fp4 * len(shapes))(*(Q(r, c, **kw).c for r, c in shapes))

    rows, cols = [(4, 6), (3, 5), (3, 5)], [(6, 4), (5, 3), (5, 3)]
    far = dict(codes=8 * BUF, scales=9 * BUF)
    for master, seed, br, bc, n, status, text in (
            (BUF, None, arrays(rows), None, 2, INVALID, "2 matrices, the object has 3"),
            (BUF, None, None, None, 3, INVALID, "by_row and by_col are NULL"),
            (None, None, arrays(rows), None, 3, INVALID, "master is NULL"),
            (BUF + 4, None, arrays(rows), None, 3, MISALIGNED, "master"),
            (BUF, BUF + 1, arrays(rows), None, 3, MISALIGNED, "seed"),
            (BUF, None, arrays(cols), None, 3, INVALID, "by_row is 6 x 4"),
            (BUF, None, arrays(rows[:2] + [(5, 3)]), None, 3, INVALID, "by_row is 5 x 3"),
            (BUF, None, arrays(rows), arrays(cols[:2] + [(3, 5)], **far), 3, INVALID, "by_col is 3 x 5")):
        refused(status, text, L.dpg_allgather_params_fp4, mats.handle, master, seed, br, bc, n, None)
    refused(INVALID, "mats is NULL", L.dpg_allgather_params_fp4, None, BUF, None, arrays(rows), None, 3, None)


def test_binding_refuses_what_it_can_see():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dpg.dpg_fp4_quantize(x, None, stream=0)                    # not on a GPU
    with pytest.raises(TypeError):
        dpg.dpg_fp4_quantize(x.half(), None, stream=0)
    with pytest.raises(ValueError):
        dpg.dpg_fp4_quantize(x[0], None, stream=0)
    with pytest.raises(ValueError):
        dpg.dpg_fp4_quantize(x.t(), None, stream=0)
    q = dpg.Fp4(4, 64, device="cpu")
    with pytest.raises(ValueError):
        dpg.dpg_fp4_dequantize(q, x[:2], stream=0)
    with pytest.raises(ValueError):
        dpg.dpg_fp4_product(q, q, x, stream=0)
    with pytest.raises(dpg.DpgError):
        dpg.Fp4(-1, 4)


def test_buffers_are_not_replaced():
    """The C description holds their addresses."""
    q = dpg.Fp4(4, 40, dpg.DPG_MXFP4, device="cpu")
    for name in ("codes", "scales", "amax"):
        assert getattr(q.c, name) == getattr(q, name).data_ptr()
        with pytest.raises(AttributeError):
            setattr(q, name, getattr(q, name).clone())
