"""4-bit matrices at the upper end of fp32: the few elements whose value is 2^128."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import MX, NV, quantized, values_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def below(x):
    return float(np.nextafter(np.float32(x), np.float32(0)))


# E8M0: codes of 3 and 4 with the scale 2^126 meet at 3.5 * 2^126; with a largest magnitude of
# 1.5 * 2^127 the scale is 2^125.  E4M3: 4 and 6 with the scale 352 * 2^117 meet at 5 * 352 * 2^117, and
# up to 1920 * 2^117 the scale is 320 * 2^117.
MOST = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,top,at,infinite", [
    (MX, MOST, 3.5 * 2.0 ** 126, True), (MX, MOST, below(3.5 * 2.0 ** 126), False), (MX, 1.5 * 2.0 ** 127, 1.5 * 2.0 ** 127, False),
    (NV, MOST, 1761 * 2.0 ** 117, True), (NV, MOST, 1760 * 2.0 ** 117, False), (NV, 1920 * 2.0 ** 117, 1920 * 2.0 ** 117, False),
])
def test_values_beyond_fp32(fmt, top, at, infinite, out_dtype):
    x = torch.zeros(3, 64)
    x[1, 0], x[1, 5], x[1, 6], x[1, 7], x[2, 40] = top, at, -at, top / 5, 1.0
    q = dpg.Fp4(3, 64, fmt)
    dpg.dpg_fp4_quantize(x.cuda(), q)
    want = quantized(x.double().numpy(), fmt)[2]
    np.testing.assert_array_equal(values_of(q), want)
    assert np.isfinite(want).all() and (abs(want[1, 5]) >= 2.0 ** 128) == infinite
    out = torch.empty(3, 64, dtype=out_dtype, device="cuda")
    dpg.dpg_fp4_dequantize(q, out)
    got = out.cpu().double().numpy()
    np.testing.assert_array_equal(got, np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want))
    assert np.isinf(got[1, 5]) == np.isinf(got[1, 6]) == infinite
    assert np.isfinite(np.delete(got[1], [0, 5, 6])).all() and np.isfinite(got[[0, 2]]).all()
