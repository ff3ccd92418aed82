"""Captured attention calls whose workspace was never made before the capture, or was grown out of after it: every
replay against the same eager calls."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg

from attn_problem import Paged, to_torch
from test_gpu_attn import DEV, _say, _values

pytestmark = pytest.mark.gpu

H, KV, D, ACT = 8, 2, 128, "f16"
LENS, NEW = [900, 130, 64], [5, 9, 1]


@pytest.fixture(autouse=True)
def _parts():
    qg.set_attn_splits(6)
    yield
    qg.set_attn_splits(0)


class Calls:
    def __init__(self, rng):
        self.pg = Paged(rng, LENS, KV, D, ACT, 16, DEV)
        self.q = to_torch(_values(rng, (sum(NEW), H, D), ACT)[0], ACT, DEV)
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(NEW)]), dtype=torch.int32, device=DEV)

    def __call__(self, ws, out=None):
        pg, (one, many) = self.pg, out or (None, None)
        return (qg.attn_decode(self.q[:3], pg.cache, pg.table_dev, pg.lens_dev, 900, workspace=ws, out=one),
                qg.attn_prefill(self.q, pg.cache, pg.table_dev, self.start, pg.lens_dev, 9, 900, workspace=ws, out=many))

    def captured(self, ws, stream):
        out = torch.zeros_like(self.q[:3]), torch.zeros_like(self.q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self(ws, out)
        return graph, out

    def check(self, graph, out, rng, what):
        for i in range(3):
            self.q.copy_(to_torch(_values(rng, tuple(self.q.shape), ACT)[0], ACT, DEV))
            want = self(qg.Workspace())
            for o in out:
                o.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (what, i)


def test_graphs_captured_without_a_workspace():
    _say("capture without a workspace")
    rng = np.random.default_rng(50)
    calls, ws, side = Calls(rng), qg.Workspace(), torch.cuda.Stream()
    first, second = calls.captured(ws, side), calls.captured(ws, side)
    # the later one first: neither counts on what the other cleared
    calls.check(*second, rng, "second")
    calls.check(*first, rng, "first")
    with torch.cuda.stream(side):
        got = calls(ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, calls(qg.Workspace())))


def test_a_graph_outlives_the_growth_of_its_workspace():
    _say("workspace grown after the capture")
    rng = np.random.default_rng(51)
    calls, ws, side = Calls(rng), qg.Workspace(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(ws)
    side.synchronize()
    graph, out = calls.captured(ws, side)
    calls.check(graph, out, rng, "before")
    with torch.cuda.stream(side):
        ws.get(32 << 20, DEV)
        # whatever the allocator has free on that stream is in use and not zero
        held = [torch.full((n << 20,), 0xA5, dtype=torch.uint8, device=DEV) for n in (1, 1, 2, 4, 8)]
    side.synchronize()
    calls.check(graph, out, rng, "after")
    assert all(bool((t == 0xA5).all()) for t in held)
