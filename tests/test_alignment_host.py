"""Misaligned weights and scales are refused before anything is enqueued (no GPU: the check comes before the device)."""

import ctypes

import pytest

import sparse_mixture_experts_expert_b200 as moe

P = ctypes.c_void_p
FAKE, OFF = P(1 << 20), P((1 << 20) + 4)     # never dereferenced


@pytest.fixture(scope="module")
def L():
    from sparse_mixture_experts_expert_b200 import _build
    _build.build()
    return moe.load()


@pytest.mark.parametrize("wfmt", [moe.WFMT_BF16, moe.WFMT_INT4_G128, moe.WFMT_INT8])
@pytest.mark.parametrize("name", ["w13", "s13", "w2", "s2", "w13_sh", "s13_sh", "w2_sh", "s2_sh"])
def test_forward_refuses_misaligned_weights_and_scales(L, wfmt, name):
    if wfmt == moe.WFMT_BF16 and name[0] == "s":
        pytest.skip("bf16 experts have no scales")
    if wfmt == moe.WFMT_INT4_G128 and name in ("s13_sh", "s2_sh"):
        pytest.skip("read one bf16 at a time: any place will do")
    s = moe.MoeShape(T=256, d=128, E=8, k=2, H=128, H_s=128, wfmt=wfmt)
    n = ctypes.c_size_t(0)
    assert L.moe_workspace_size(ctypes.byref(s), ctypes.byref(n)) == 0
    w = {k: FAKE for k in ("w13", "s13", "w2", "s2", "w13_sh", "s13_sh", "w2_sh", "s2_sh")}
    w[name] = OFF
    assert L.moe_forward(ctypes.byref(s), FAKE, FAKE, None, *w.values(), FAKE, None, None, None, None, None, None, None,
                         FAKE, n.value, None, None) == 1
