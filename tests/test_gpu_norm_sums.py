"""Layer norm's gradient sums where rows are shared out in other ways: few and many
rows, wide ones, both types, and workspaces on a 16-byte boundary."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(40, 64), (700, 256), (2500, 700), (5000, 768), (300, 1024), (1300, 2048),
                                       (512, 4096), (1000, 4000), (400, 8192), (700, 5000), (33, 16384), (320, 9000),
                                       (20, 17000), (1300, 771)])
@pytest.mark.parametrize("offset", [0, 16])
def test_sums(rows, cols, offset, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) + 0.5).to(dtype).cuda()
    dy = torch.randn(rows, cols, generator=g).to(dtype).cuda()
    gain = (1 + 0.1 * torch.randn(cols, generator=g)).to(dtype).cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dpg.dpg_layer_norm(x, gain, None, 1e-5, y, mean, rstd)
    size = dpg.dpg_layer_norm_workspace(rows, cols)
    beside = torch.full((size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = beside[offset:offset + size]
    dx, alone = torch.empty_like(x), torch.empty_like(x)
    dgain, dbias = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, dx, dgain, dbias, ws)
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, alone)
    assert torch.equal(dx, alone)                             # however the rows are shared out
    assert (beside[:offset] == 0xA5).all() and (beside[offset + size:] == 0xA5).all()
    n = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    # one term after the other in a part (fp32 rows: in half as many parts at least), eight warps,
    # 16 threads' parts and their tree, n's own three roundings and the product's
    parts = size // (8 * cols)
    depth = 2 * -(-rows // parts) + 8 + -(-parts // 16) + 4 + 4
    for got, term in ((dgain, dy.double() * n), (dbias, dy.double())):
        assert torch.all((got.double() - term.sum(0)).abs() <= depth * U * term.abs().sum(0) * 1.05 + 1e-37)
    # the same bits again, and added to what is there
    again, held = torch.empty_like(dgain), torch.full_like(dgain, 3.0)
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, None, again, None, ws)
    assert torch.equal(again, dgain)
    dpg.dpg_layer_norm_backward(dy, x, gain, mean, rstd, None, None, held, ws, accumulate=True)
    np.testing.assert_array_equal(held.cpu().numpy(), (dbias + 3.0).cpu().numpy())


def test_offsets_beyond_32_bits():
    rows, cols, last = 530000, 4096, 64
    g = torch.Generator().manual_seed(1)
    x, dy = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, cols, dtype=torch.bfloat16,
                                                                                     device="cuda")
    x[-last:] = torch.randn(last, cols, generator=g).cuda()
    dy[-last:] = torch.randn(last, cols, generator=g).cuda()
    out = []
    for p, q in ((x, dy), (x[-last:], dy[-last:])):
        y, dx, n = torch.empty_like(p), torch.empty_like(p), p.shape[0]
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        dpg.dpg_layer_norm(p, None, None, 1e-5, y, mean, rstd)
        ws = torch.empty(dpg.dpg_layer_norm_workspace(n, cols), dtype=torch.uint8, device="cuda")
        dgain, dbias = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        dpg.dpg_layer_norm_backward(q, p, None, mean, rstd, dx, dgain, dbias, ws)
        out.append((y, dx, dgain, dbias))
    (y, dx, dgain, dbias), (y1, dx1, dgain1, dbias1) = out
    assert torch.equal(y[-last:], y1) and torch.equal(dx[-last:], dx1)
    assert not y[:-last].any() and not dx[:-last].any()
    # 64 terms in another order each, and zeros: at most 70 roundings on either side
    n = (x[-last:].double() - mean.double()[:, None]) * rstd.double()[:, None]
    for a, b, term in ((dgain, dgain1, dy[-last:].double() * n), (dbias, dbias1, dy[-last:].double())):
        assert torch.all((a - b).abs() <= 140 * U * term.abs().sum(0))
