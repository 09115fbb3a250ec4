"""The 4-bit layers and the norm as the example puts them together: that they run
in its training loop, and their gradients against the formulas in 64 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import NV, product_bound, quantized, spread, values_of

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from zero_optimizer_step_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import muon_adam
    finally:
        sys.path.pop(0)
    return muon_adam


def test_example_runs_in_4_bits():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "muon_adam.py"), "--fp4"], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    losses = [float(line.split()[-1]) for line in r.stdout.splitlines() if line.startswith("step")]
    assert len(losses) == 4 and all(np.isfinite(losses)), r.stdout


def test_gradients_of_its_layers(example):
    t, d, h = 60, 48, 80
    group = example.Group([spread(h, d, 1, torch.bfloat16, 0.1).cuda().requires_grad_()])
    w = dpg.Fp4(h, d), dpg.Fp4(d, h)
    mats = dpg.dpg_plan_matrices(group.plan, [h], [d])
    dpg.dpg_allgather_params_fp4(mats, group.master, [w[0]], [w[1]])
    x = spread(t, d, 2, torch.bfloat16, 1.0).cuda().requires_grad_()
    dy = spread(t, h, 3, torch.bfloat16).cuda()
    seed = torch.tensor([9], device="cuda")
    y = example.Linear4.apply(x, w, group.slot(0, 1), seed)
    y.backward(dy)
    x64, dy64 = x.detach().cpu().double().numpy(), dy.cpu().double().numpy()
    for got, a, b in ((y.detach(), quantized(x64, NV)[2], values_of(w[0])),
                      (x.grad, quantized(dy64, NV, 9, 0)[2], values_of(w[1])),
                      (group.slot(0, 1), quantized(dy64.T, NV, 9, 1)[2], quantized(x64.T, NV)[2])):
        want = a @ b.T
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= product_bound(a, b, torch.bfloat16, want))
    assert not group.slot(0, 0).any()


def test_gradients_of_its_norm(example):
    rows, cols = 30, 72
    x = spread(rows, cols, 4, torch.bfloat16, 1.0).cuda().requires_grad_()
    gain, bias = ((1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(k))).to(torch.bfloat16).cuda()
                  for k in (5, 6))
    dgain, dbias = torch.empty_like(gain), torch.empty_like(bias)
    dy = spread(rows, cols, 7, torch.bfloat16).cuda()
    example.Norm.apply(x, gain, bias, dgain, dbias).backward(dy)
    p = x.detach().cpu().double().requires_grad_()
    g, b = gain.cpu().double().requires_grad_(), bias.cpu().double().requires_grad_()
    n = (p - p.mean(1, keepdim=True)) / (p.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    (n * g + b).backward(dy.cpu().double())
    for got, want in ((x.grad, p.grad), (dgain, g.grad), (dbias, b.grad)):
        # half a step of bf16, and fp32 sums of at most 72 terms (under 100 roundings with
        # the products), whose magnitudes add up to at most ten times the largest result
        tol = 2.0 ** -8 * want.abs() + 100 * 2.0 ** -24 * 10 * want.abs().max()
        assert torch.all((got.cpu().double() - want).abs() <= tol)
