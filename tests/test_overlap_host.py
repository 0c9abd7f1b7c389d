"""Outputs that overlap an input where that would race are refused (no GPU: the check comes before the device; the
pointers are never dereferenced)."""

import ctypes

import pytest

import sparse_mixture_experts_expert_b200 as moe

P = ctypes.c_void_p
AT = 1 << 30
FAR = P(1 << 20)
T, d, E, k = 256, 64, 8, 2


@pytest.fixture(scope="module")
def L():
    from sparse_mixture_experts_expert_b200 import _build
    _build.build()
    return moe.load()


@pytest.mark.parametrize("shift", [0, 4, T * k * 4 - 4, -(T * k * 4 - 4)])
@pytest.mark.parametrize("tokens", [T, 64 * T])      # one launch for few pairs, several for many
def test_permute_int8_refuses_slots_over_the_choices(L, shift, tokens):
    # every block of the one-launch form counts all choices while others write their slots
    s = moe.MoeShape(T=tokens, d=d, E=E, k=k, H=128, wfmt=moe.WFMT_INT8)
    n = ctypes.c_size_t(0)
    assert L.moe_workspace_size(ctypes.byref(s), ctypes.byref(n)) == 0
    assert L.moe_permute_int8(ctypes.byref(s), FAR, P(AT), P(AT + shift), None, None, FAR, FAR, None, FAR, FAR, FAR, n.value,
                              None) == 1


ROWS, TOK = T * k * d * 2, T * d * 2     # bytes of [R, d] and of [T, d] in bf16


@pytest.mark.parametrize("shift", [16, ROWS - 16, -16, -(TOK - 16)])
def test_sorting_gradients_refuse_partly_overlapping_outputs(L, shift):
    s = moe.MoeShape(T=T, d=d, E=E, k=k, H=16)

    def cb(dout=FAR, y=FAR, dy=FAR):
        return L.moe_combine_backward(ctypes.byref(s), dout, y, P(64), P(64), None, dy, P(64), None)
    assert cb(y=P(AT), dy=P(AT + shift)) == 1
    if -ROWS < shift < TOK:
        assert cb(dout=P(AT), dy=P(AT + shift)) == 1

    def pb(g=FAR, add=None, dx=P(AT), ti=0, to=0):
        return L.moe_permute_backward(ctypes.byref(s), g, ti, P(64), add, dx, to, None)
    assert pb(g=P(AT - shift)) == 1
    assert pb(add=P(AT + 16)) == 1 and pb(add=P(AT - TOK + 16)) == 1
    assert pb(add=P(AT + 2 * TOK - 16), to=1) == 1                     # fp32: twice the bytes
    assert pb(g=P(AT - 2 * ROWS + 16), ti=1) == 1
