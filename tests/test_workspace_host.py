"""Host logic of qg.Workspace: what a captured graph was given stays where it is, and a buffer that only a capture would
clear is not handed to other calls. CPU tensors stand in for device memory."""

import gc
import weakref

import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg

MB = 1 << 20


@pytest.fixture
def stream(monkeypatch):
    """The current stream's handle, and whether it captures."""
    s = {"handle": 7, "capturing": False}
    monkeypatch.setattr(qg, "_raw_stream", lambda index: s["handle"])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s["capturing"])
    return s


def test_one_buffer_per_stream_serves_every_smaller_call(stream):
    ws = qg.Workspace()
    a, n = ws.get(5000, "cpu")
    assert n == a.numel() == MB and not bool(a.any())
    assert ws.get(100, "cpu")[0] is a and ws.get(MB, "cpu")[0] is a
    assert ws.get(0, "cpu") == (None, 0)
    stream["handle"] = 8
    assert ws.get(100, "cpu")[0] is not a


def test_a_buffer_that_was_grown_out_of_stays_allocated(stream):
    ws = qg.Workspace()
    first = weakref.ref(ws.get(5000, "cpu")[0])
    at = first().data_ptr()
    second, n = ws.get(MB + 1, "cpu")
    gc.collect()
    assert n >= MB + 1 and first() is not None and second.data_ptr() != at
    # so that calls of slowly growing sizes do not pile up buffers: each at least doubles
    assert n >= 2 * MB
    third, n = ws.get(5 * MB, "cpu")
    assert n == 5 * MB and ws.get(3 * MB, "cpu")[0] is third


def test_a_buffer_made_inside_a_capture_serves_that_call_alone(stream):
    ws = qg.Workspace()
    stream["capturing"] = True
    a, n = ws.get(5000, "cpu")   # the graph clears it at each replay
    assert n >= 5000 and not bool(a.any())
    stream["capturing"] = False
    b, _ = ws.get(5000, "cpu")
    assert b is not a
    stream["capturing"] = True
    assert ws.get(5000, "cpu")[0] is b   # one that is there and clear is taken
    assert ws.get(2 * MB, "cpu")[0] is not b
    stream["capturing"] = False
    assert ws.get(5000, "cpu")[0] is b
