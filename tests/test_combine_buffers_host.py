"""What moe_combine takes for its buffers: larger ones and other leading dimensions, as long as the values it reads and
writes are there; anything else is refused before the call (no GPU: the call is a stand-in)."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

import sparse_mixture_experts_expert_b200 as moe
import sparse_mixture_experts_expert_b200.autograd as ag

bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture
def ran(monkeypatch):
    log = []
    monkeypatch.setattr(moe, "_L", lambda: SimpleNamespace(moe_combine=lambda *a: (log.append(a), 0)[1]))
    monkeypatch.setattr(moe, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(moe, "_on", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_stream", lambda *a: None)
    return log


def _args(**kw):
    a = dict(y_perm=torch.zeros(24, 64, dtype=bf), slot_pos=torch.zeros(4, 2, dtype=i32), topk_w=torch.zeros(4, 2))
    a.update(kw)
    return a


S = moe.MoeShape(T=4, d=64, E=8, k=2, H=16, capacity=3)


@pytest.mark.parametrize("kw", [{}, dict(y_perm=torch.zeros(30, 64, dtype=bf)), dict(y_perm=torch.zeros(8, 3, 64, dtype=bf)),
                                dict(y_perm=torch.zeros(24 * 64, dtype=bf)), dict(slot_pos=torch.zeros(8, dtype=i32)),
                                dict(topk_w=torch.zeros(8)), dict(topk_w=torch.zeros(2, 2, 2)),
                                dict(slot_pos=torch.zeros(9, 2, dtype=i32)),
                                dict(out=torch.zeros(2, 2, 64, dtype=bf)), dict(out=torch.zeros(7, 64, dtype=bf)),
                                dict(y_shared=torch.zeros(2, 2, 64, dtype=bf))])
def test_larger_buffers_and_other_leading_dimensions(ran, kw):
    a = _args(**kw)
    out = moe.moe_combine(S, **a)
    assert len(ran) == 1 and ran[0][1] == a["y_perm"].data_ptr()
    assert out is a["out"] if "out" in a else out.shape == (4, 64)


@pytest.mark.parametrize("err,name,kw", [(ValueError, "y_perm", dict(y_perm=torch.zeros(23, 64, dtype=bf))),
                                         (ValueError, "slot_pos", dict(slot_pos=torch.zeros(3, 2, dtype=i32))),
                                         (ValueError, "topk_w", dict(topk_w=torch.zeros(7))),
                                         (TypeError, "slot_pos", dict(slot_pos=torch.zeros(4, 2, dtype=torch.int64))),
                                         (ValueError, "y_shared", dict(y_shared=torch.zeros(8, 64, dtype=bf))),
                                         (TypeError, "out", dict(out=torch.zeros(4, 64))),
                                         (ValueError, "out", dict(out=torch.zeros(3, 64, dtype=bf)))])
def test_missing_values_and_other_types_are_refused(ran, err, name, kw):
    with pytest.raises(err, match=name):
        moe.moe_combine(S, **_args(**kw))
    assert not ran


def test_differentiable_combine_takes_the_grouped_rows_alone(ran):
    # its gradient has y_perm's own rows
    for kw in (dict(y_perm=torch.zeros(30, 64, dtype=bf)), dict(slot_pos=torch.zeros(8, dtype=i32)), dict(topk_w=torch.zeros(8))):
        a = _args(**kw)
        with pytest.raises(ValueError, match=next(iter(kw))):
            ag.combine(S, a["y_perm"], a["slot_pos"], a["topk_w"], kept=torch.zeros(8, dtype=i32))
    assert not ran
