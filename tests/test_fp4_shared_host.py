"""A plan's 4-bit forms that share buffers (no GPU): refused before device work, since
the matrix quantised last would be in the place of the others."""

import pytest

import zero_optimizer_step_gb300 as dpg

BUF = 1 << 20   # aligned addresses that are never read: the calls stop before
NV, MX = dpg.DPG_NVFP4, dpg.DPG_MXFP4


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def forms(shapes, first, fmt=NV):
    return [dpg.dpg_fp4(BUF * (first + 3 * k), BUF * (first + 3 * k + 1), BUF * (first + 3 * k + 2), r, c, fmt)
            for k, (r, c) in enumerate(shapes)]


@pytest.mark.parametrize("side,k,field,other,from_,from_field,fmt", [
    ("row", 2, "codes", "row", 1, "codes", NV), ("row", 2, "scales", "row", 1, "scales", MX),
    ("row", 2, "amax", "row", 1, "amax", NV), ("col", 1, "codes", "col", 0, "codes", NV),
    ("col", 1, "codes", "row", 0, "codes", NV), ("col", 0, "scales", "row", 2, "scales", MX),
    ("col", 0, "amax", "row", 2, "amax", NV), ("row", 0, "codes", "row", 0, "scales", NV),
    ("row", 0, "scales", "col", 1, "codes", MX), ("row", 0, "amax", "col", 1, "codes", NV),
])
def test_refused(side, k, field, other, from_, from_field, fmt):
    plan = dpg.dpg_plan_buckets([24, 2 * 15], 1 << 30, 1)
    mats = dpg.dpg_plan_matrices(plan, [4, 3], [6, 5])             # 4 x 6, and two of 3 x 5
    shapes = [(4, 6), (3, 5), (3, 5)]
    q = {"row": forms(shapes, 8, fmt), "col": forms([s[::-1] for s in shapes], 40, fmt)}
    setattr(q[side][k], field, getattr(q[other][from_], from_field))
    arrays = [(dpg.dpg_fp4 * 3)(*q[s]) for s in ("row", "col")]
    before = dpg.dpg_launch_count()
    for a in (arrays, [arrays[0], None], [None, arrays[1]]):
        needed = {side, other} <= {s for s, v in zip(("row", "col"), a) if v is not None}
        if needed:
            assert dpg.lib().dpg_allgather_params_fp4(mats.handle, BUF, None, a[0], a[1], 3, None) == dpg.DPG_ERR_INVALID_ARG
            assert b"share a buffer" in dpg.lib().dpg_last_error()
    assert dpg.dpg_launch_count() == before


def test_buffers_that_overlap():
    plan = dpg.dpg_plan_buckets([2 * 15], 1 << 30, 1)
    mats = dpg.dpg_plan_matrices(plan, [3], [5])
    for field, offset in (("codes", 32), ("scales", 496), ("amax", 4 * 255)):
        q = forms([(3, 5)] * 2, 8)                                 # 48 bytes, 512 and 256 floats
        setattr(q[1], field, getattr(q[0], field) + offset)
        before = dpg.dpg_launch_count()
        assert dpg.lib().dpg_allgather_params_fp4(mats.handle, BUF, None, (dpg.dpg_fp4 * 2)(*q), None, 2,
                                                  None) == dpg.DPG_ERR_INVALID_ARG
        assert b"share a buffer" in dpg.lib().dpg_last_error()
        assert dpg.dpg_launch_count() == before
