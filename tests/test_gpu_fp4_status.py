"""The record of a product's wait that ran out, where several streams ask for it."""
import pytest
import torch

import zero_optimizer_step_gb300 as dpg
from fp4_util import NV, spread

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_optimizer_step_gb300 import build
    build.build()


def told(stream=None):
    """Whether the stream is told of a wait that ran out."""
    try:
        dpg.dpg_fp4_status(stream)
    except dpg.DpgError as e:
        assert e.status == dpg.DPG_ERR_DEVICE_TIMEOUT
        return True
    return False


@pytest.fixture(autouse=True)
def default_stream_has_asked():
    yield
    told()
    assert not told()


@pytest.fixture
def operands():
    a, b = dpg.Fp4(8, 3000, NV), dpg.Fp4(300, 3000, NV)
    for q, seed in ((a, 1), (b, 2)):
        dpg.dpg_fp4_quantize(spread(q.rows, q.cols, seed, torch.bfloat16).cuda(), q)
    torch.cuda.synchronize()
    return a, b, torch.empty(8, 300, device="cuda")


@pytest.fixture
def streams():
    """Two streams that have been told of whatever came before."""
    two = torch.cuda.Stream(), torch.cuda.Stream()
    assert two[0].cuda_stream != two[1].cuda_stream
    for s in two:
        told(s)
        assert not told(s)
    return two


def one_that_runs_out(a, b, out, stream, monkeypatch):
    monkeypatch.setenv("DPG_TEST_HOOKS", "1")
    assert dpg.lib().dpg_set_staged_fault(1, 20_000_000) == dpg.DPG_OK
    dpg.dpg_fp4_product(a, b, out, stream=stream)


def test_no_stream_takes_the_record_of_another(operands, streams, monkeypatch):
    one_that_runs_out(*operands, streams[1], monkeypatch)
    streams[1].synchronize()
    assert told(streams[0])                    # a product on the device
    assert told(streams[1])                    # whose result is incomplete
    assert not told(streams[0]) and not told(streams[1])
    one_that_runs_out(*operands, streams[0], monkeypatch)
    assert told(streams[0]) and not told(streams[0])
    assert told(streams[1]) and not told(streams[1])


def test_two_failures_before_a_stream_asks(operands, streams, monkeypatch):
    for s in streams:
        one_that_runs_out(*operands, s, monkeypatch)
        s.synchronize()
    for s in streams:
        assert told(s) and not told(s)
    dpg.dpg_fp4_product(*operands, stream=streams[0])
    assert not told(streams[0])


def test_a_graph_replayed_on_another_stream(operands, streams, monkeypatch):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        one_that_runs_out(*operands, streams[0], monkeypatch)
    assert not told(streams[0]) and not told(streams[1])
    with torch.cuda.stream(streams[1]):
        graph.replay()
    assert told(streams[1]) and told(streams[0])
    assert not told(streams[0]) and not told(streams[1])
