"""8-bit integer experts on rows whose gates all lie deep in the activation's negative tail.

The row scale of h lifts such a row back to full size, so there the activation's relative error counts, not its absolute
one.  With g = sum s_row s_col formed by two fp32 products (2^-23 of g, which the tail multiplies by 1 + g^2), the
exponent g^2 / 2 off by three roundings (1.5 g^2 2^-24) and 2^-20 for the rest of the formula, an element of h is off by
at most delta = 2^-20 + g^2 2^-22 before it is rounded to bf16.  A rounding then falls the other way with probability
2^9 delta at most (2^-6 for |g| = 10) and moves the element by 2^-7 of itself, its code by a step hs more: in the norm
of a row 2^-3 (2^-7 + hs / rms h), hs / rms h = 1/40 in rows of these spreads: 4.1e-3, but of |g| = 10 alone and for
flips that are all of full size; their mean square is a third, 2.4e-3.  With the rounding of y (2^-8 / sqrt 3 = 2.3e-3
in the norm) that is 3.3e-3, inside the layer's 5e-3.
"""

import numpy as np
import pytest
import torch

import oracle as O
from helpers import REL_FROB, np64

pytestmark = pytest.mark.gpu
DEV = "cuda"


# hidden widths of the fused kernel (128) and of the separate ones (320)
@pytest.mark.parametrize("H", [128, 320])
@pytest.mark.parametrize("act", [0, 1])
def test_rows_deep_in_the_negative_tail(lib, act, H):
    moe = lib
    d = 256
    g = torch.Generator().manual_seed(H + act)
    level = torch.arange(2, 11).float()                       # |g| of a row, within 5 %
    x = level[:, None].expand(-1, d).bfloat16().contiguous()
    w13 = torch.randint(-127, 128, (1, 2 * H, d), generator=g)
    w13[:, :H] = -127 + torch.randint(0, 13, (1, H, 1), generator=g)
    s13 = torch.full((1, 2 * H), 1.0 / (127 * d))
    w2 = torch.randint(-127, 128, (1, d, H), generator=g)
    s2 = torch.full((1, d), 2.0 ** -7)
    q, sc = O.quantize_rows_int8(np64(x))
    want, h, _, hs = O.expert_ffn_int8(q, sc, w13[0].numpy(), np64(s13)[0], w2[0].numpy(), np64(s2)[0], act)
    assert (hs > 0).all() and np.isfinite(want).all()
    s = moe.MoeShape(T=x.shape[0], d=d, E=1, k=1, H=H, act=act, wfmt=moe.WFMT_INT8)
    got = np64(moe.moe_expert_ffn_int8(s, torch.from_numpy(q.astype(np.int8)).to(DEV), torch.from_numpy(sc).to(DEV),
                                       w13.to(torch.int8).to(DEV), s13.to(DEV), w2.to(torch.int8).to(DEV), s2.to(DEV)))
    err = np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)
    assert (err <= REL_FROB).all(), dict(zip(level.tolist(), err.tolist()))
