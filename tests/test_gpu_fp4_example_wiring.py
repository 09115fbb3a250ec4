"""The 4-bit training loop of the example: which random bits it takes."""
import os
import sys

import pytest
import torch

import zero_optimizer_step_gb300 as dpg

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
    monkeypatch.setattr(muon_adam, "STEPS", 2)
    muon_adam.main(fp4=True)
    return muon_adam, log


def test_every_rounding_has_random_bits_of_its_own(run):
    example, log = run
    seeds = [n for name, n in log if name == "dpg_fp4_quantize" and n is not None]
    assert len(seeds) == 2 * 2 * example.R                      # a layer, a step, a replica
    assert len(set(seeds)) == len(seeds)
