"""A tensor that a call cannot do without is named when it is missing."""

import pytest
import torch

import sparse_mixture_experts_expert_b200 as moe


def _int8(**kw):
    a = dict(xq=torch.zeros(8, 64, dtype=torch.int8), xs=torch.zeros(8), w13=torch.zeros(2, 32, 64, dtype=torch.int8),
             s13=torch.zeros(2, 32), w2=torch.zeros(2, 64, 16, dtype=torch.int8), s2=torch.zeros(2, 64))
    a.update(kw)
    return a


S = moe.MoeShape(T=8, d=64, E=2, k=1, H=16, wfmt=moe.WFMT_INT8)


@pytest.mark.parametrize("name", ["xq", "xs", "w13", "s13", "w2", "s2"])
def test_int8_experts(name):
    with pytest.raises(ValueError, match=f"{name}: missing"):
        moe.moe_expert_ffn_int8(S, **_int8(**{name: None}))


@pytest.mark.parametrize("name", ["w13", "s13", "w2", "s2"])
def test_int8_experts_on_bf16_rows(name):
    # before the rows are quantised
    a = _int8(**{name: None})
    with pytest.raises(ValueError, match=f"{name}: missing"):
        moe.moe_expert_ffn(S, torch.zeros(8, 64, dtype=torch.bfloat16), a["w13"], a["w2"], s13=a["s13"], s2=a["s2"])


def test_sorting_gradients():
    z, i, w = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(8, 1, dtype=torch.int32), torch.zeros(8, 1)
    for args, name in (((None, z, i, w), "dout"), ((z, None, i, w), "y_perm"), ((z, z, None, w), "slot_pos"),
                       ((z, z, i, None), "topk_w")):
        with pytest.raises(ValueError, match=f"{name}: missing"):
            moe.moe_combine_backward(S, *args)
    for args, name in (((None, i), "dx_perm"), ((z, None), "slot_pos")):
        with pytest.raises(ValueError, match=f"{name}: missing"):
            moe.moe_permute_backward(S, *args)
