"""combine with frozen rows: the gates' gradient alone, without a gradient buffer for the rows."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

import oracle as O
import sparse_mixture_experts_expert_b200 as moe
import sparse_mixture_experts_expert_b200.autograd as ag
import synth
from helpers import np64


@pytest.mark.parametrize("frozen", [True, False])
def test_frozen_rows_ask_for_no_gradient(monkeypatch, frozen):
    asked = {}

    def combine_backward(shape, dout, y, slot, w, *, kept=None, want_dw=True, want_dy=True):
        asked.update(want_dy=want_dy, want_dw=want_dw, kept=kept)
        return dict(dy_perm=torch.zeros_like(y) if want_dy else None, dtopk_w=torch.ones_like(w))
    monkeypatch.setattr(ag, "moe_combine", lambda shape, y, slot, w, ysh=None: y[:shape.T] + w.sum())
    monkeypatch.setattr(ag, "moe_combine_backward", combine_backward)
    s = moe.MoeShape(T=3, d=16, E=4, k=2, H=16, capacity=2)
    y, w = torch.zeros(8, 16), torch.zeros(3, 2).requires_grad_(True)
    kept = torch.zeros(4, dtype=torch.int32)
    ag.combine(s, y.requires_grad_(not frozen), torch.zeros(3, 2, dtype=torch.int32), w, kept=kept).sum().backward()
    assert asked["want_dy"] is not frozen and asked["want_dw"] and (asked["kept"] is None) == frozen
    assert torch.equal(w.grad, torch.ones(3, 2)) and (y.grad is None) == frozen


def test_no_gradient_at_all_is_refused(monkeypatch):
    monkeypatch.setattr(moe, "_L", lambda: SimpleNamespace(moe_combine_backward=lambda *a: 0))
    s = moe.MoeShape(T=4, d=64, E=8, k=2, H=16)
    with pytest.raises(ValueError, match="want_dy"):
        moe.moe_combine_backward(s, torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16),
                                 torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), want_dw=False, want_dy=False)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0, 30])
def test_gate_gradient_with_frozen_rows(lib, cap):
    T, E, k, d = 500, 24, 3, 192
    s = lib.MoeShape(T=T, d=d, E=E, k=k, H=16, capacity=cap)
    p = O.permute(synth.draw_topk_idx(T, E, k, seed=2, skew=0.7).numpy(), E, cap)
    g = torch.Generator().manual_seed(4)
    y, G = torch.randn(s.R, d, generator=g).bfloat16(), torch.randn(T, d, generator=g).bfloat16()
    w = torch.rand(T, k, generator=g)
    slot = torch.from_numpy(p["slot_pos"].astype(np.int32)).cuda()
    W = w.cuda().requires_grad_(True)
    torch.cuda.synchronize()
    out = ag.combine(s, y.cuda(), slot, W)
    G = G.cuda()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out.backward(G)
    torch.cuda.synchronize()
    if s.R * d * 2 > 1 << 19:   # no buffer of the rows' size
        assert torch.cuda.max_memory_allocated() - before < s.R * d
    dw = O.combine_backward(np64(G), np64(y), p["slot_pos"], np64(w))[1]
    mag = O.combine_backward(np.abs(np64(G)), np.abs(np64(y)), p["slot_pos"], np64(w))[1]
    assert (np.abs(np64(W.grad) - dw) <= d * 2.0 ** -24 * mag).all()   # an fp32 dot product of d terms
    # the same bits as with the rows' gradient
    r = lib.moe_combine_backward(s, G, y.cuda(), slot, w.cuda())
    assert torch.equal(r["dtopk_w"], W.grad) and r["dy_perm"].shape == y.shape
