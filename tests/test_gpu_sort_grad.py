"""GPU parity of the sorting gradients (moe_permute_backward, moe_combine_backward) and of the differentiable
``dispatch`` / ``combine`` against float64.

Tolerances, from the arithmetic: a bf16 output is one rounding of the fp32 value (2^-8 of it, half a step of an
8-bit significand at its worst), an fp32 dot product of n terms is within n 2^-24 of the sum of magnitudes, and a sum
of k rows within k 2^-24 of theirs.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle as O
import synth
from helpers import np64, npi

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(T, E, k, d, cap, seed=0, dtype=torch.bfloat16, skew=0.0):
    idx = synth.draw_topk_idx(T, E, k, seed=seed, skew=skew).numpy()
    p = O.permute(idx, E, cap)
    g = torch.Generator().manual_seed(seed)
    R = E * cap if cap else T * k
    rows = torch.randn(R, d, generator=g).to(dtype)
    filled = np.zeros(R, bool)
    slot = p["slot_pos"]
    filled[slot[slot >= 0]] = True
    rows[~torch.from_numpy(filled)] = float("nan")          # what no token fills must not be read
    return dict(slot=torch.from_numpy(slot.astype(np.int32)), kept=torch.from_numpy(p["kept"].astype(np.int32)),
                rows=rows, filled=filled, R=R, dout=torch.randn(T, d, generator=g).to(torch.bfloat16),
                w=torch.rand(T, k, generator=g), add=torch.randn(T, d, generator=g))


def _shape(moe, T, E, k, d, cap):
    return moe.MoeShape(T=T, d=d, E=E, k=k, H=16, capacity=cap)


# one token and one slot; a narrow and an odd width; k of every kernel width (2, 4, 8, 16); tokens few enough for a
# CTA each (narrow and wide rows) and many; capacities with drops, with empty experts, with padding longer than the
# rows one CTA clears
SIZES = [(1, 1, 1, 16, 0), (1, 8, 2, 64, 0), (3, 5, 3, 784, 0), (70, 16, 16, 272, 0), (300, 33, 5, 48, 20),
         (1000, 192, 4, 768, 27), (2500, 8, 2, 256, 0), (1500, 12, 7, 1040, 700), (64, 512, 8, 7168, 0),
         (9, 4, 2, 7168, 1)]


@pytest.mark.parametrize("T,E,k,d,cap", SIZES)
def test_combine_backward_matches_the_oracle(lib, T, E, k, d, cap):
    moe = lib
    c = _case(T, E, k, d, cap, seed=T, skew=1.0 if cap else 0.0)
    s = _shape(moe, T, E, k, d, cap)
    r = moe.moe_combine_backward(s, c["dout"].to(DEV), c["rows"].to(DEV), c["slot"].to(DEV), c["w"].to(DEV),
                                 kept=c["kept"].to(DEV))
    clean = np.where(c["filled"][:, None], np64(c["rows"]), 0.0)
    dy, dw = O.combine_backward(np64(c["dout"]), clean, npi(c["slot"]), np64(c["w"]))
    got = np64(r["dy_perm"])
    assert (np.abs(got - dy) <= 2.0 ** -8 * np.abs(dy)).all()
    if cap:
        assert (got[~c["filled"]] == 0).all()
    mag = O.combine_backward(np.abs(np64(c["dout"])), np.abs(clean), npi(c["slot"]), np64(c["w"]))[1]
    assert (np.abs(np64(r["dtopk_w"]) - dw) <= d * 2.0 ** -24 * mag).all()
    assert (npi(r["dtopk_w"])[npi(c["slot"]) < 0] == 0).all()
    again = moe.moe_combine_backward(s, c["dout"].to(DEV), c["rows"].to(DEV), c["slot"].to(DEV), c["w"].to(DEV),
                                     kept=c["kept"].to(DEV))
    assert torch.equal(again["dy_perm"], r["dy_perm"]) and torch.equal(again["dtopk_w"], r["dtopk_w"])


@pytest.mark.parametrize("T,E,k,d,cap", SIZES)
@pytest.mark.parametrize("tin,tout,add", [(torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, True),
                                          (torch.float32, torch.bfloat16, True), (torch.float32, torch.float32, False)])
def test_permute_backward_matches_the_oracle(lib, T, E, k, d, cap, tin, tout, add):
    moe = lib
    c = _case(T, E, k, d, cap, seed=T + 1, dtype=tin, skew=1.0 if cap else 0.0)
    s = _shape(moe, T, E, k, d, cap)
    a = c["add"].to(tout) if add else None
    got = moe.moe_permute_backward(s, c["rows"].to(DEV), c["slot"].to(DEV), add=a.to(DEV) if add else None, dtype=tout)
    assert got.dtype == tout
    clean = np.where(c["filled"][:, None], np64(c["rows"]), 0.0)
    want = O.permute_backward(clean, npi(c["slot"]), np64(a) if add else None)
    mag = O.permute_backward(np.abs(clean), npi(c["slot"]), np.abs(np64(a)) if add else None)
    tol = (k + 1) * 2.0 ** -24 * mag
    if tout == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(np64(got) - want) <= tol).all()


def test_permute_backward_accumulates_in_place(lib):
    moe = lib
    c = _case(500, 16, 4, 208, 0)
    s = _shape(moe, 500, 16, 4, 208, 0)
    acc = c["add"].to(DEV)
    want = moe.moe_permute_backward(s, c["rows"].to(DEV), c["slot"].to(DEV), add=acc)
    got = moe.moe_permute_backward(s, c["rows"].to(DEV), c["slot"].to(DEV), add=acc, out=acc)
    assert got.data_ptr() == acc.data_ptr() and torch.equal(got, want)


def test_dropped_slots_take_nothing_from_infinite_gradients(lib):
    # a token whose slots were all dropped, and one with one left: an infinite dout stays out of their dw and rows
    moe = lib
    s = _shape(moe, 3, 2, 2, 32, 2)
    slot = torch.tensor([[0, 2], [1, -1], [-1, -1]], dtype=torch.int32, device=DEV)
    dout = torch.full((3, 32), float("inf"), dtype=torch.bfloat16, device=DEV)
    dout[0] = 1.0
    y = torch.ones(4, 32, dtype=torch.bfloat16, device=DEV)
    kept = torch.tensor([2, 1], dtype=torch.int32, device=DEV)
    r = moe.moe_combine_backward(s, dout, y, slot, torch.ones(3, 2, device=DEV), kept=kept)
    assert r["dtopk_w"].tolist() == [[32.0, 32.0], [float("inf"), 0.0], [0.0, 0.0]]
    assert r["dy_perm"][0].eq(1).all() and r["dy_perm"][1].isinf().all() and r["dy_perm"][3].eq(0).all()
    # rows outside the buffer count as dropped
    wild = torch.tensor([[0, 4], [2147483647, 1], [-7, 3]], dtype=torch.int32, device=DEV)
    dx = moe.moe_permute_backward(s, y, wild)
    assert dx[:, 0].tolist() == [1.0, 1.0, 1.0]
    assert moe.moe_combine_backward(s, y[:3], y, wild, torch.ones(3, 2, device=DEV))["dtopk_w"].tolist() == \
        [[32.0, 0.0], [0.0, 32.0], [0.0, 32.0]]


def test_combine_backward_one_output_at_a_time(lib):
    """Through the C ABI: dy alone (no y needed), dw alone, and rows that no slot fills untouched without kept."""
    moe = lib
    L = moe.load()
    T, E, k, d, cap = 40, 6, 2, 96, 9
    c = {k_: v.to(DEV) if isinstance(v, torch.Tensor) else v for k_, v in _case(T, E, k, d, cap, skew=0.7).items()}
    s = _shape(moe, T, E, k, d, cap)
    full = moe.moe_combine_backward(s, c["dout"], c["rows"], c["slot"], c["w"], kept=c["kept"])
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    dy = torch.full((c["R"], d), 7.0, dtype=torch.bfloat16, device=DEV)
    assert L.moe_combine_backward(ctypes.byref(s), P(c["dout"]), None, P(c["slot"]), P(c["w"]), None, P(dy), None, st) == 0
    dw = torch.full((T, k), 7.0, device=DEV)
    assert L.moe_combine_backward(ctypes.byref(s), P(c["dout"]), P(c["rows"]), P(c["slot"]), P(c["w"]), None, None, P(dw),
                                  st) == 0
    torch.cuda.synchronize()
    filled = torch.from_numpy(c["filled"])
    assert torch.equal(dy.cpu()[filled], full["dy_perm"].cpu()[filled]) and (dy.cpu()[~filled] == 7.0).all()
    assert torch.equal(dw, full["dtopk_w"])


@pytest.mark.parametrize("cap", [0, 13])
def test_training_step_through_dispatch_and_combine(lib, cap):
    """Own experts (a scaled tanh per expert) between dispatch and combine: gradients of x, the gates, the experts and
    the shared output against float64 autograd of the same formula."""
    from sparse_mixture_experts_expert_b200.autograd import combine, dispatch
    moe = lib
    T, E, k, d = 90, 16, 3, 64
    s = _shape(moe, T, E, k, d, cap)
    idx = synth.draw_topk_idx(T, E, k, seed=5, skew=0.8)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, d, generator=g).bfloat16()
    w, ysh = torch.rand(T, k, generator=g), torch.randn(T, d, generator=g).bfloat16()
    a, G = torch.rand(E, d, generator=g) + 0.5, torch.randn(T, d, generator=g).bfloat16()
    p = O.permute(idx.numpy(), E, cap)
    slot = torch.from_numpy(p["slot_pos"].astype(np.int64))

    leaf = lambda t: t.to(DEV).requires_grad_(True)  # noqa: E731
    X, W, S, A = leaf(x), leaf(w), leaf(ysh), leaf(a)
    xp, sl, kept, offs = dispatch(s, X, idx.to(DEV))
    assert (npi(sl) == p["slot_pos"]).all() and (npi(kept) == p["kept"]).all()
    rows = torch.arange(xp.shape[0], device=DEV)
    e_of = torch.searchsorted(offs[1:].long(), rows, right=True).clamp(max=E - 1)
    y = torch.tanh(xp.float() * A[e_of]).bfloat16()
    out = combine(s, y, sl, W, S, kept=kept if cap else None)
    out.backward(G.to(DEV))

    x64, w64, s64, a64 = (t.double().requires_grad_(True) for t in (x, w, ysh, a))
    keep = (slot >= 0).double()
    y64 = torch.tanh(x64[:, None] * a64[idx.long()])
    ((w64 * keep)[..., None] * y64).sum(1).add(s64).mul(G.double()).sum().backward()
    # bf16 steps on the way: y (2^-8), dy (2^-8), the row gradient handed back as bf16 (2^-8), dx (2^-8)
    for got, want, n in ((X.grad, x64.grad, 4), (W.grad, w64.grad, 1), (A.grad, a64.grad, 2)):
        d_, w_ = np64(got) - want.numpy(), want.numpy()
        assert np.linalg.norm(d_) <= n * 2.0 ** -8 * np.linalg.norm(w_)
    assert torch.equal(S.grad.cpu(), G)
    assert moe.moe_get_status()[0] == 0


def test_gradients_on_another_stream_and_in_a_graph(lib):
    moe = lib
    T, E, k, d = 400, 24, 4, 128
    c = {k_: v.to(DEV) if isinstance(v, torch.Tensor) else v for k_, v in _case(T, E, k, d, 0).items()}
    s = _shape(moe, T, E, k, d, 0)

    def step(stream=None):
        r = moe.moe_combine_backward(s, c["dout"], c["rows"], c["slot"], c["w"], stream=stream)
        return r["dy_perm"], r["dtopk_w"], moe.moe_permute_backward(s, r["dy_perm"], c["slot"], stream=stream)
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    c["dout"].mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], 2 * want[1]) and torch.equal(outs[0].float(), 2 * want[0].float())
    assert torch.equal(outs[2], 2 * want[2])
