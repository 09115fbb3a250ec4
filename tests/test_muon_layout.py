"""How the matrices of an object are laid out, and the limits of one object, on
the host (no GPU)."""
import pytest

import zero_optimizer_step_gb300 as dpg

GIB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def _mats(rows, cols, count):
    plan = dpg.dpg_plan_buckets([rows * cols * count], 1 << 50, 1)
    return dpg.dpg_plan_matrices(plan, [rows], [cols])


def _tile_bytes(rows, cols, count):
    """The tiles' blocks for a short side of up to 128: four parts of X and three
    of Gram matrices, of fp16, padded to 256."""
    m, n = -(-min(rows, cols) // 256) * 256, -(-max(rows, cols) // 256) * 256
    return count * 2 * (4 * m * n + 3 * m * m)


@pytest.mark.parametrize("rows,cols,count", [(128, 2048, 6000), (2048, 128, 6000), (128, 4096, 3000), (100, 6000, 3000),
                                             (128, 1024, 20000)])
def test_large_lists_take_the_path_of_less_memory(rows, cols, count):
    # (a tenth more for counters, items and row sums)
    tiles = _tile_bytes(rows, cols, count)
    assert tiles > 16 * GIB and _mats(rows, cols, count).workspace_bytes <= 1.1 * tiles


@pytest.mark.parametrize("rows,cols,count", [(16, 64, 1 << 16), (10, 100, 1 << 17), (32, 256, 1 << 15)])
def test_large_lists_of_narrow_matrices_are_not_padded_to_tiles(rows, cols, count):
    tiles = _tile_bytes(rows, cols, count)
    assert tiles > 16 * GIB and _mats(rows, cols, count).workspace_bytes < tiles / 8


def test_rows_of_the_workspace_stay_within_a_copys_coordinate():
    # 129 x 129 is padded to 256 x 256: 5 x 8 blocks of 128 rows each, and a
    # block's first row has to stay below 2^31
    most = ((1 << 31) - 1) // 128 // 40
    assert _mats(129, 129, most).n_matrices == most
    with pytest.raises(dpg.DpgError) as e:
        _mats(129, 129, most + 1)
    assert e.value.status == dpg.DPG_ERR_INVALID_ARG and "large" in str(e.value)


def test_matrices_of_one_object_are_counted():
    most = 1 << 20
    assert _mats(1, 1, most).n_matrices == most
    with pytest.raises(dpg.DpgError) as e:
        _mats(1, 1, most + 1)
    assert e.value.status == dpg.DPG_ERR_INVALID_ARG and "large" in str(e.value)


def test_a_parameter_without_elements_changes_nothing():
    def workspace(numels, rows, cols):
        plan = dpg.dpg_plan_buckets(numels, 1 << 50, 1)
        return dpg.dpg_plan_matrices(plan, rows, cols).workspace_bytes
    alone = workspace([100 * 100 * 30], [100], [100])
    assert workspace([100 * 100 * 30, 0], [100, 100], [100, 1 << 23]) == alone
    assert workspace([0, 100 * 100 * 30], [1 << 23, 100], [1 << 23, 100]) == alone
