"""The 4-bit training loop of the example: where its operators leave gradients, what
its products read after a step, and which random bits it takes."""
import os
import sys

import numpy as np
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import NV, quantized, values_of

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def run(monkeypatch):
    """What two steps of the loop did, call by call."""
    from zero_optimizer_step_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import muon_adam
    finally:
        sys.path.pop(0)
    log = []

    def record(name, note):
        real = getattr(dpg, name)

        def call(*args, **kw):
            log.append((name, note(*args, **kw)))
            return real(*args, **kw)
        monkeypatch.setattr(dpg, name, call)

    record("dpg_fp4_quantize", lambda x, row=None, col=None, *, seed=None: None if seed is None else int(seed))
    record("dpg_fp4_product", lambda a, b, out: (values_of(b), tuple(out.shape), out.data_ptr()))
    record("dpg_layer_norm_backward", lambda dy, x, gain, mean, rstd, dx, dgain, dbias, ws: (dgain.data_ptr(), dbias.data_ptr()))
    record("dpg_muon_step", lambda plan, mats, grads, *rest: (plan, list(grads), rest[2].clone()))
    record("dpg_step", lambda plan, grads, *rest: (plan, list(grads)))
    monkeypatch.setattr(muon_adam, "STEPS", 2)
    muon_adam.main(fp4=True)
    return muon_adam, log


def test_gradients_are_left_where_the_steps_read_them(run):
    example, log = run
    muon = [n for name, n in log if name == "dpg_muon_step"]
    adam = [n for name, n in log if name == "dpg_step"]
    assert len(muon) == len(adam) == 2
    plan, grads, _ = muon[0]
    shapes = [(768, 256), (256, 768)]
    # a replica's backward pass: the second layer's weight first
    want = [grads[r][int(plan.param_offset[k]):].data_ptr() for _ in muon for r in range(example.R) for k in (1, 0)]
    got = [(s, p) for name, n in log if name == "dpg_fp4_product" for s, p in [n[1:]] if s in shapes]
    assert got == [(shapes[1 - i % 2], p) for i, p in enumerate(want)]
    plan, grads = adam[0]
    want = [tuple(grads[r][int(plan.param_offset[k]):].data_ptr() for k in (2, 3)) for _ in adam for r in range(example.R)]
    assert [n for name, n in log if name == "dpg_layer_norm_backward"] == want


def test_products_read_what_the_step_left(run):
    example, log = run
    at = [i for i, (name, _) in enumerate(log) if name == "dpg_muon_step"]
    for start, end in ((0, at[0]), (at[0], at[1])):
        plan, _, master = log[end][1]                           # before that step: as its products read it
        b = [n[0] for name, n in log[start:end] if name == "dpg_fp4_product"]
        assert len(b) == 6 * example.R
        forms = []
        for k, shape in enumerate([(768, 256), (256, 768)]):
            o = int(plan.param_offset[k])
            m = master[o:o + shape[0] * shape[1]].view(shape).cpu().double().numpy()
            forms.append((quantized(m, NV)[2], quantized(m.T, NV)[2]))
        for r in range(example.R):                              # forward; then dx and dW of each layer
            for n, want in ((0, forms[0][0]), (1, forms[1][0]), (2, forms[1][1]), (4, forms[0][1])):
                np.testing.assert_array_equal(b[6 * r + n], want)


def test_every_rounding_has_random_bits_of_its_own(run):
    example, log = run
    seeds = [n for name, n in log if name == "dpg_fp4_quantize" and n is not None]
    assert len(seeds) == 2 * 2 * example.R                      # a layer, a step, a replica
    assert len(set(seeds)) == len(seeds)
