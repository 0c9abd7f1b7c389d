"""Refusals of the 8-bit integer entry points and of the sorting gradients (no GPU): the C ABI returns its status
before touching the device, and the Python binding raises on types, shapes and devices; and the plumbing of the
differentiable ``dispatch`` and ``combine`` with stand-in entry points."""

import ctypes

import pytest
import torch

import oracle as O
import sparse_mixture_experts_expert_b200 as moe
import sparse_mixture_experts_expert_b200.autograd as ag

P = ctypes.c_void_p
FAKE = P(4096)     # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def L():
    from sparse_mixture_experts_expert_b200 import _build
    _build.build()
    return moe.load()


def _shape(**kw):
    base = dict(T=256, d=64, E=8, k=2, H=128, wfmt=moe.WFMT_INT8)
    base.update(kw)
    return moe.MoeShape(**base)


@pytest.mark.parametrize("kw,code", [({}, 0), ({"d": 80, "H": 48}, 0), ({"d": 60}, 2), ({"H": 8}, 2), ({"wfmt": 3}, 1),
                                     ({"H_s": 24}, 2), ({"H_s": 32, "capacity": 7}, 0)])
def test_int8_shape_validation(L, kw, code):
    n = ctypes.c_size_t(0)
    s = _shape(**kw)
    assert L.moe_workspace_size(ctypes.byref(s), ctypes.byref(n)) == code
    if code == 0:
        assert n.value > 0 and n.value % 256 == 0


def test_quantize_int8_refusals(L):
    q = lambda x=FAKE, dt=0, rows=4, K=64, c=FAKE, s=FAKE: L.moe_quantize_int8(x, dt, rows, K, c, s, None)
    assert q(dt=2) == 1 and q(dt=-1) == 1
    assert q(K=24) == 2 and q(K=0) == 2 and q(rows=-1) == 2 and q(rows=1 << 31) == 2
    assert q(x=None) == 1 and q(c=None) == 1 and q(s=None) == 1
    assert q(x=P(4104)) == 1 and q(c=P(4100)) == 1 and q(s=P(4098)) == 1
    assert q(x=None, rows=0) == 0          # nothing to do


def test_permute_int8_refusals(L):
    s = _shape()
    n = ctypes.c_size_t(0)
    assert L.moe_workspace_size(ctypes.byref(s), ctypes.byref(n)) == 0

    def call(sh=s, x=FAKE, xq=FAKE, xs=FAKE, ws=FAKE, nb=None):
        return L.moe_permute_int8(ctypes.byref(sh), x, FAKE, FAKE, None, None, FAKE, FAKE, None, xq, xs, ws,
                                  n.value if nb is None else nb, None)
    assert call(x=None) == 1 and call(xq=None) == 1 and call(xs=None) == 1 and call(ws=None) == 1
    assert call(x=P(4100)) == 1 and call(xq=P(4100)) == 1
    assert call(nb=n.value - 1) == 3
    assert call(sh=_shape(k=9)) == 1


def test_expert_ffn_int8_refusals(L):
    s = _shape()
    n = ctypes.c_size_t(0)
    size = lambda sh, hidden, R: L.moe_expert_ffn_int8_workspace_size(ctypes.byref(sh), hidden, R, ctypes.byref(n))
    assert size(_shape(wfmt=0), 128, 64) == 1 and size(s, 100, 64) == 2 and size(s, 0, 64) == 2
    assert size(s, 65552, 64) == 2 and size(s, 128, -1) == 1
    assert size(s, 128, 0) == 0
    assert size(s, 128, 64) == 0 and n.value >= 64 * (3 * 128 + 4)

    def call(sh=s, groups=8, hidden=128, R=64, gs=FAKE, gr=FAKE, xq=FAKE, xs=FAKE, s13=FAKE, y=FAKE, ws=FAKE, nb=None):
        return L.moe_expert_ffn_int8(ctypes.byref(sh), groups, hidden, R, xq, xs, gs, gr, FAKE, s13, FAKE, FAKE, y, ws,
                                     n.value if nb is None else nb, None)
    assert call(sh=_shape(wfmt=0)) == 1 and call(groups=0) == 1 and call(groups=513) == 1 and call(R=-1) == 1
    assert call(hidden=24) == 2
    assert call(gr=None) == 1 and call(gs=None, gr=None) == 1       # no table: one group only
    assert call(xq=None) == 1 and call(xs=None) == 1 and call(s13=None) == 1 and call(y=None) == 1
    assert call(xq=P(4104)) == 1 and call(y=P(4104)) == 1 and call(ws=P(4096 + 16)) == 1
    assert call(nb=n.value - 1) == 3
    assert call(R=0) == 0
    # the scratch-free expert step takes no 8-bit experts, nor does the backward
    assert L.moe_expert_ffn(ctypes.byref(s), 8, 128, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == 1
    b = [ctypes.byref(s), FAKE, FAKE, None, FAKE, FAKE, FAKE, None, None, None, FAKE, ctypes.c_float(0.0), FAKE]
    assert L.moe_backward_x(*b, FAKE, 1 << 40, None) == 2


def test_int8_forward_needs_its_scales(L):
    s = _shape(H_s=64)
    n = ctypes.c_size_t(0)
    assert L.moe_workspace_size(ctypes.byref(s), ctypes.byref(n)) == 0

    def call(s13=FAKE, s2=FAKE, s13s=FAKE, s2s=FAKE, nb=None):
        return L.moe_forward(ctypes.byref(s), FAKE, FAKE, None, FAKE, s13, FAKE, s2, FAKE, s13s, FAKE, s2s, FAKE, None,
                             None, None, None, None, None, None, FAKE, n.value if nb is None else nb, None, None)
    assert call(s13=None) == 1 and call(s2=None) == 1 and call(s13s=None) == 1 and call(s2s=None) == 1
    assert call(nb=n.value - 256) == 3


def test_sorting_gradient_refusals(L):
    s, cap = _shape(wfmt=0), _shape(wfmt=0, capacity=16)

    def cb(sh=s, dout=P(8192), y=P(8192), slot=FAKE, w=FAKE, kept=None, dy=FAKE, dw=FAKE):
        return L.moe_combine_backward(ctypes.byref(sh), dout, y, slot, w, kept, dy, dw, None)
    assert cb(dout=None) == 1 and cb(slot=None) == 1 and cb(w=None) == 1
    assert cb(y=None) == 1 and cb(dy=None, dw=None) == 1
    assert cb(kept=FAKE) == 1 and cb(sh=cap, kept=FAKE, dy=None) == 1
    assert cb(dout=P(4104)) == 1 and cb(y=P(4104)) == 1 and cb(dy=P(4104)) == 1
    assert cb(sh=_shape(d=72)) == 2
    assert cb(dout=P(8192), y=FAKE, dy=FAKE) == 1 and cb(dout=FAKE, y=P(8192), dy=FAKE) == 1     # in place

    def pb(g=P(8192), ti=0, slot=FAKE, add=None, dx=FAKE, to=0):
        return L.moe_permute_backward(ctypes.byref(s), g, ti, slot, add, dx, to, None)
    assert pb(g=None) == 1 and pb(slot=None) == 1 and pb(dx=None) == 1
    assert pb(ti=2) == 1 and pb(to=-1) == 1
    assert pb(g=FAKE, dx=FAKE) == 1                                                               # in place
    assert pb(g=P(4104)) == 1 and pb(add=P(4104)) == 1 and pb(dx=P(4104)) == 1


def test_binding_refuses_types_shapes_and_host_tensors():
    s = _shape(T=4, wfmt=0)
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = lambda *sh, dt=bf: torch.zeros(*sh, dtype=dt)
    with pytest.raises(TypeError):
        moe.moe_quantize_int8(z(4, 64, dt=torch.float16))
    with pytest.raises(ValueError):
        moe.moe_quantize_int8(torch.zeros((), dtype=bf))
    with pytest.raises(ValueError, match="device"):
        moe.moe_quantize_int8(z(4, 64))
    with pytest.raises(TypeError):
        moe.moe_combine_backward(s, z(4, 64, dt=f32), z(8, 64), z(4, 2, dt=i32), z(4, 2, dt=f32))
    with pytest.raises(ValueError):
        moe.moe_combine_backward(s, z(4, 64), z(9, 64), z(4, 2, dt=i32), z(4, 2, dt=f32))
    with pytest.raises(ValueError, match="device"):
        moe.moe_combine_backward(s, z(4, 64), z(8, 64), z(4, 2, dt=i32), z(4, 2, dt=f32))
    with pytest.raises(TypeError):
        moe.moe_permute_backward(s, z(8, 64, dt=torch.float16), z(4, 2, dt=i32))
    with pytest.raises(TypeError):
        moe.moe_permute_backward(s, z(8, 64), z(4, 2, dt=i32), add=z(4, 64), dtype=f32)   # addend of another type
    with pytest.raises(ValueError, match="device"):
        moe.moe_permute_backward(s, z(8, 64), z(4, 2, dt=i32))
    q = _shape(T=4, E=2, H=16)
    w = lambda *sh: torch.zeros(*sh, dtype=torch.int8)
    a = dict(xq=w(8, 64), xs=z(8, dt=f32), w13=w(2, 32, 64), s13=z(2, 32, dt=f32), w2=w(2, 64, 16), s2=z(2, 64, dt=f32))
    call = lambda **kw: moe.moe_expert_ffn_int8(q, *{**a, **kw}.values(), group_start=z(2, dt=i32), group_rows=z(2, dt=i32))
    with pytest.raises(ValueError, match="device"):
        call()
    with pytest.raises(TypeError):
        call(s13=z(2, 32))
    with pytest.raises(ValueError):
        call(s2=z(2, 32, dt=f32))
    with pytest.raises(ValueError):
        moe.moe_expert_ffn_int8(q, *a.values(), group_start=z(1, dt=i32), group_rows=z(2, dt=i32))
    with pytest.raises(ValueError):
        moe.moe_expert_ffn(q, z(8, 64), a["w13"], a["w2"], s13=a["s13"], s2=a["s2"], h=z(8, 16))


def test_layer_and_combine_refuse_other_types_and_shapes():
    s = _shape(T=4, E=2, H=16, H_s=32)
    x, wr = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64)
    a = dict(w13=torch.zeros(2, 32, 64, dtype=torch.int8), w2=torch.zeros(2, 64, 16, dtype=torch.int8),
             s13=torch.zeros(2, 32), s2=torch.zeros(2, 64), w13_sh=torch.zeros(1, 64, 64, dtype=torch.int8),
             s13_sh=torch.zeros(1, 64), w2_sh=torch.zeros(1, 64, 32, dtype=torch.int8), s2_sh=torch.zeros(1, 64))
    call = lambda **kw: moe.moe_forward(s, x, wr, **{**a, **kw})
    with pytest.raises(TypeError, match="s13"):
        call(s13=a["s13"].bfloat16())           # half the bytes the kernels would read
    with pytest.raises(TypeError, match="w13"):
        call(w13=a["w13"].bfloat16())
    with pytest.raises(ValueError, match="s2_sh"):
        call(s2_sh=torch.zeros(1, 32))
    with pytest.raises(ValueError, match="w2_sh: missing"):
        call(w2_sh=None)
    f = _shape(T=4, wfmt=0)
    y, p, w = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(TypeError, match="y_perm"):
        moe.moe_combine(f, y.float(), p, w)
    with pytest.raises(ValueError, match="y_perm"):
        moe.moe_combine(f, y[:7], p, w)
    with pytest.raises(TypeError, match="topk_w"):
        moe.moe_combine(f, y, p, w.bfloat16())
    with pytest.raises(ValueError, match="y_shared"):
        moe.moe_combine(f, y, p, w, y)


# ------------------------------------------------------------------ dispatch and combine with stand-ins


def _stand_ins(monkeypatch, calls):
    def permute(shape, x, idx):
        p = O.permute(idx.numpy(), shape.E, shape.capacity)
        slot = torch.from_numpy(p["slot_pos"].astype("int32"))
        rows = torch.zeros(shape.R, shape.d, dtype=x.dtype)
        for t in range(shape.T):
            for j in range(shape.k):
                if slot[t, j] >= 0:
                    rows[slot[t, j]] = x[t]
        return dict(x_perm=rows, slot_pos=slot, kept=torch.from_numpy(p["kept"].astype("int32")),
                    offsets=torch.from_numpy(p["offsets"].astype("int32")))

    def combine(shape, y, slot, w, ysh=None):
        return torch.from_numpy(O.combine(y.double().numpy(), slot.numpy(), w.double().numpy(),
                                          None if ysh is None else ysh.double().numpy())).to(y.dtype)

    def combine_backward(shape, dout, y, slot, w, *, kept=None, want_dw=True):
        calls["kept"], calls["want_dw"] = kept, want_dw
        dy, dw = O.combine_backward(dout.double().numpy(), y.double().numpy(), slot.numpy(), w.double().numpy())
        return dict(dy_perm=torch.from_numpy(dy).to(y.dtype), dtopk_w=torch.from_numpy(dw).to(w.dtype) if want_dw else None)

    def permute_backward(shape, g, slot, *, dtype):
        calls["dtype"] = dtype
        return torch.from_numpy(O.permute_backward(g.double().numpy(), slot.numpy())).to(g.dtype)
    for name, f in (("moe_permute", permute), ("moe_combine", combine), ("moe_combine_backward", combine_backward),
                    ("moe_permute_backward", permute_backward)):
        monkeypatch.setattr(ag, name, f)


@pytest.mark.parametrize("cap", [0, 3])
def test_gradients_through_dispatch_and_combine(monkeypatch, cap):
    calls = {}
    _stand_ins(monkeypatch, calls)
    T, E, k, d = 6, 4, 2, 16
    s = moe.MoeShape(T=T, d=d, E=E, k=k, H=16, capacity=cap)
    g = torch.Generator().manual_seed(0)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    mk = lambda *sh: torch.randn(*sh, generator=g, dtype=torch.float64).requires_grad_(True)
    x, w, ysh = mk(T, d), mk(T, k), mk(T, d)

    def run(x, w, ysh):
        xp, slot, kept, _ = ag.dispatch(s, x, idx)
        return ag.combine(s, torch.tanh(xp), slot, w, ysh, kept=kept if cap else None)
    assert torch.autograd.gradcheck(run, (x, w, ysh))
    assert (calls["kept"] is not None) == bool(cap) and calls["want_dw"] and calls["dtype"] == torch.bfloat16
    with pytest.raises(RuntimeError):           # no second derivatives
        g1, = torch.autograd.grad(run(x, w, ysh).sum(), x, create_graph=True)
        g1.sum().backward()
    xp, slot, kept, offs = ag.dispatch(s, x, idx)
    assert xp.requires_grad and not slot.requires_grad and not kept.requires_grad and not offs.requires_grad
    ag.combine(s, torch.tanh(xp), slot, w.detach(), None, kept=kept if cap else None).sum().backward()
    assert calls["want_dw"] is False
    if cap:
        with pytest.raises(ValueError, match="kept"):
            ag.combine(s, xp, slot, w)
