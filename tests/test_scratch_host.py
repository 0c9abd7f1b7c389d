"""Whose scratch a call without ``ws`` counts in (no GPU: streams, capture and allocation are stand-ins)."""

import contextlib
import ctypes
import threading
from types import SimpleNamespace

import pytest
import torch

import sparse_mixture_experts_expert_b200 as moe
import sparse_mixture_experts_expert_b200.autograd as ag


@pytest.fixture
def gpu(monkeypatch):
    """One device, a current stream that the test sets, and buffers that stay alive, so that no address is used twice."""
    state = SimpleNamespace(stream=7, capturing=False, kept=[])
    real_empty = torch.empty

    def empty(*sh, device=None, **kw):
        state.kept.append(real_empty(*sh, **kw))
        return state.kept[-1]
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(moe, "_device", lambda: 0)
    monkeypatch.setattr(moe, "_capturing", lambda: state.capturing)
    monkeypatch.setattr(moe, "_raw_stream", lambda dev: state.stream)
    monkeypatch.setattr(moe, "_held", type(moe._held)())
    monkeypatch.setattr(moe, "moe_workspace_size", lambda shape: 1024 * shape.T)
    return state


def _shape(T=4):
    return moe.MoeShape(T=T, d=64, E=8, k=2, H=16)


def _addr(T=4):
    return moe.workspace(_shape(T), "cuda").data_ptr()


def test_one_stream_keeps_its_buffer_and_grows_it(gpu):
    a = _addr()
    assert _addr() == a and _addr(T=2) == a
    b = _addr(T=9)
    assert b != a and _addr(T=9) == b and _addr() == b


def test_streams_captures_and_threads_share_nothing(gpu):
    seen = {_addr()}

    def new(what):
        a = _addr()
        assert a not in seen, what
        seen.add(a)
    gpu.stream = 8
    new("another stream")
    gpu.stream = 7
    new("back on the first stream, whose old buffer was given up")
    gpu.capturing = True
    new("a captured call")
    new("the next captured call, perhaps of another graph")
    gpu.capturing = False
    t = threading.Thread(target=lambda: new("another host thread"))
    t.start()
    t.join()
    assert len(seen) == 6


def test_dispatch_on_two_streams_counts_in_two_buffers(gpu, monkeypatch):
    used = []

    def moe_permute(shape, x, idx, slot, drop, counts, kept, offsets, row_src, x_perm, ws, n, stream):
        used.append((stream, ws))
        return 0
    monkeypatch.setattr(moe, "_L", lambda: SimpleNamespace(moe_permute=moe_permute))
    monkeypatch.setattr(moe, "_ptr", lambda t: t.data_ptr())
    monkeypatch.setattr(moe, "_on", lambda *a: contextlib.nullcontext())
    x, idx = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    monkeypatch.setattr(moe, "permute_outputs", lambda shape, dev: {k: torch.zeros(1) for k in (
        "slot_pos", "drop_mask", "counts", "kept", "offsets", "row_src", "x_perm")})
    for gpu.stream in (7, 8):
        ag.dispatch(_shape(), x, idx)
    (s0, w0), (s1, w1) = used
    assert (s0, s1) == (7, 8) and w0 != w1
