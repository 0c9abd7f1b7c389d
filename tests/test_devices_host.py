"""The grouping and the combine run on their tensors' device and, where one is given, on their stream (no GPU: tensors
and devices are stand-ins)."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

import sparse_mixture_experts_expert_b200 as moe


class Fake:
    """A tensor of a device that is not there."""

    def __init__(self, dev, shape, dtype):
        self.device, self.shape, self.dtype, self.is_cuda = torch.device(dev), torch.Size(shape), dtype, True

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 4096

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()


@pytest.fixture
def calls(monkeypatch):
    now = SimpleNamespace(dev=0, stream=None, log=[])

    @contextlib.contextmanager
    def device(d):
        old, now.dev = now.dev, torch.device(d).index
        yield
        now.dev = old

    @contextlib.contextmanager
    def on_stream(st):
        old, now.stream = now.stream, st
        yield
        now.stream = old
    monkeypatch.setattr(moe, "_device", lambda: now.dev)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(moe, "_capturing", lambda: False)
    monkeypatch.setattr(moe, "_raw_stream", lambda dev: 100 + dev if now.stream is None else now.stream.cuda_stream)
    made = lambda *sh, dtype=None, device=None: (now.log.append(("made", now.dev, now.stream)),     # noqa: E731
                                                 Fake(device, sh, dtype))[1]
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, made)
    monkeypatch.setattr(torch, "full", lambda sh, v, dtype=None, device=None: made(*sh, dtype=dtype, device=device))
    monkeypatch.setattr(moe, "moe_workspace_size", lambda shape: 512)
    monkeypatch.setattr(moe, "_held", type(moe._held)())
    run = lambda *a: (now.log.append(("ran", now.dev, a[-1])), 0)[1]                                 # noqa: E731
    fwd = lambda *a: (now.log.append(("ran", now.dev, a[-2])), 0)[1]                                 # noqa: E731
    monkeypatch.setattr(moe, "_L", lambda: SimpleNamespace(moe_permute=run, moe_combine=run, moe_route=run,
                                                                 moe_route_from_logits=run, moe_forward=fwd))
    return now


def _args(dev, T=4, k=2, d=64):
    f = lambda sh, dt: Fake(dev, sh, dt)  # noqa: E731
    return (moe.MoeShape(T=T, d=d, E=8, k=k, H=16), f((T, d), torch.bfloat16), f((T, k), torch.int32),
            f((T * k, d), torch.bfloat16), f((T, k), torch.float32))


def test_tensors_of_another_device_run_there(calls):
    s, x, idx, y, w = _args("cuda:1")
    moe.moe_permute(s, x, idx)
    moe.moe_combine(s, y, idx, w)
    assert [e for e in calls.log if e[0] == "ran"] == [("ran", 1, 101)] * 2
    assert all(e[1] == 1 for e in calls.log) and calls.dev == 0


def test_tensors_of_two_devices_are_refused(calls):
    s, x, idx, y, w = _args("cuda:1")
    other = Fake("cuda:0", idx.shape, idx.dtype)
    with pytest.raises(ValueError, match="cuda:0"):
        moe.moe_permute(s, x, other)
    with pytest.raises(ValueError, match="cuda:0"):
        moe.moe_combine(s, y, other, w)
    with pytest.raises(ValueError, match="cuda:0"):
        moe.moe_combine(s, y, idx, w, out=Fake("cuda:0", (4, 64), torch.bfloat16))
    assert not [e for e in calls.log if e[0] == "ran"]


def test_outputs_are_prepared_on_the_given_stream(calls):
    # row_src and x_perm are filled before the rows are moved: on the same stream, or the fill may come after
    s, x, idx, y, w = _args("cuda:0")
    st = SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=55)
    moe.moe_permute(s, x, idx, stream=st)
    made = [e for e in calls.log if e[0] == "made"]
    assert len(made) == 8 and all(e[2] is st for e in made) and ("ran", 0, 55) in calls.log


def _layer(dev, T=4, d=64, E=8):
    f = lambda sh, dt: Fake(dev, sh, dt)  # noqa: E731
    i8, f32 = torch.int8, torch.float32
    s = moe.MoeShape(T=T, d=d, E=E, k=2, H=16, wfmt=moe.WFMT_INT8)
    return (s, f((T, d), torch.bfloat16), f((E, d), f32), f((E, 32, d), i8), f((E, d, 16), i8),
            dict(s13=f((E, 32), f32), s2=f((E, d), f32)))


def test_the_layer_and_the_router_run_on_their_tensors_device(calls):
    s, x, wr, w13, w2, scales = _layer("cuda:1")
    moe.moe_forward(s, x, wr, w13, w2, **scales)
    moe.moe_route(s, x, wr)
    moe.moe_route_from_logits(s, Fake("cuda:1", (4, 8), torch.float32))
    assert [e for e in calls.log if e[0] == "ran"] == [("ran", 1, 101)] * 3
    assert all(e[1] == 1 for e in calls.log) and calls.dev == 0
    other = Fake("cuda:0", wr.shape, wr.dtype)
    for call in (lambda: moe.moe_forward(s, x, other, w13, w2, **scales), lambda: moe.moe_route(s, x, other),
                 lambda: moe.moe_forward(s, x, wr, w13, w2, s13=Fake("cuda:0", (8, 32), torch.float32), s2=scales["s2"])):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    assert len([e for e in calls.log if e[0] == "ran"]) == 3


def test_scratch_that_a_call_frees_belongs_to_the_given_stream(calls, monkeypatch):
    # freed at the end of the call: memory of the current stream could be handed out while the call still runs
    def size(*a):
        a[-1]._obj.value = 1024
        return 0
    ran = lambda *a: 0  # noqa: E731
    monkeypatch.setattr(moe, "_L", lambda: SimpleNamespace(
        moe_backward_workspace_size=size, moe_route_tree_workspace_size=size, moe_transpose_experts=ran, moe_backward=ran,
        moe_backward_x=ran, moe_route_tree=ran))
    st = SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=55)
    f = lambda *sh, dt=torch.bfloat16: Fake("cuda:0", sh, dt)  # noqa: E731
    s = moe.MoeShape(T=4, d=64, E=8, k=2, H=16)
    made = []
    monkeypatch.setattr(torch, "empty", lambda *sh, dtype=None, device=None: (made.append((dtype, calls.stream)),
                                                                             f(*sh, dt=dtype))[1])
    args = (s, f(4, 64), f(8, 64, dt=torch.float32), f(8, 32, 64), f(8, 64, 16), f(4, 64))
    for call in (moe.moe_backward, moe.moe_backward_x):
        made.clear()
        call(*args, stream=st)
        temp = [e for e in made if e[0] in (torch.uint8, torch.bfloat16)]      # workspace and transposed weights
        assert len(temp) == 3 and all(e[1] is st for e in temp)
    made.clear()
    moe.moe_route_tree(moe.MoeShape(T=4, d=64, E=64, k=2, H=16), 8, 2, f(4, 64), f(16, 64, dt=torch.float32), stream=st)
    assert [e[1] for e in made if e[0] == torch.uint8] == [st]
