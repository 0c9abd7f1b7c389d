"""GPU parity of the 8-bit integer experts against the float64 oracle.

Codes and scales are compared bit for bit.  The products are integer sums, exact on both sides, so y differs from the
oracle by (a) the rounding of y to bf16, 2^-8 of it, and (b) elements of h whose bf16 rounding falls the other way
because the fp32 activation is off by about 2^-20: such an element moves by at most 2^-7 of itself and its code by at
most one step hs more than that.  The bound of one output is therefore
  2^-8 |y| + sum_i |w2_i| s2 (2^-7 |h_i| + hs)                                                             (always)
and, since a rounding falls the other way with probability 2^-20 / 2^-9 = 2^-11 at most, in the 2-norm over a whole
output (rms rounding of bf16 at most 2^-8 / sqrt(3) = 2.3e-3, flips 2^-5.5 (2^-7 + hs / rms h) with hs / rms h below
1/8, 2.9e-3) the layer's own 5e-3.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle as O
import synth
from helpers import REL_FROB, assert_out_close, np64, npi, rel_frob

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------- codes


# one row; widths under, at and past what a warp and a CTA hold in registers (1024, 8192), odd multiples of 16, and
# the widest row; more rows than a CTA's
@pytest.mark.parametrize("rows,K", [(1, 16), (9, 48), (37, 784), (300, 1024), (17, 1040), (5, 8192), (3, 8208), (2, 65536)])
def test_bf16_codes_and_scales_bit_exact(lib, rows, K):
    moe = lib
    g = torch.Generator().manual_seed(K)
    x = (torch.randn(rows, K, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).bfloat16()
    x[0, 0], x[0, 1] = 4.0 * x[0].abs().max(), -2.0 * x[0].abs().max()      # a tie at 63.5 both ways
    q, s = moe.moe_quantize_int8(x.to(DEV))
    wq, ws = O.quantize_rows_int8(np64(x))
    assert (npi(q) == wq).all() and (npi(s) == ws).all()


def test_ties_special_rows_and_subnormals(lib):
    moe = lib
    n = torch.arange(-128, 128).float()
    rows = [n / 2 * (127 / 127.0),                    # max 64: quotients 127 n / 128
            torch.where(n.abs() < 127, n + 0.5, torch.full_like(n, 127.0)),     # max 127: every quotient a tie
            torch.where(n.abs() < 127, (n + 0.5) * 2, torch.full_like(n, 254.0)),
            torch.zeros(256), torch.full((256,), 2.0 ** -120), torch.full((256,), 2.0 ** -119),
            n * 2.0 ** 120, n * 1e-38]
    x = torch.stack(rows).bfloat16()
    q, s = moe.moe_quantize_int8(x.to(DEV))
    wq, ws = O.quantize_rows_int8(np64(x))
    assert (npi(q) == wq).all() and (npi(s) == ws).all()
    # a row with an infinity or a NaN says so in its scale, and its neighbours are untouched
    y = torch.ones(4, 256).bfloat16()
    y[1, 7], y[2, 200] = float("-inf"), float("nan")
    for t in (y, y.float()):
        q, s = moe.moe_quantize_int8(t.to(DEV))
        assert s[1].isinf() and s[2].isnan() and (q[0] == 127).all() and (q[3] == 127).all()
        assert s[0] == np.float32(1) / np.float32(127)


@pytest.mark.parametrize("rows,K", [(1, 16), (50, 784), (3, 2048), (2, 20000)])
def test_fp32_codes(lib, rows, K):
    moe = lib
    x = torch.randn(rows, K, generator=torch.Generator().manual_seed(rows))
    q, s = moe.moe_quantize_int8(x.to(DEV))
    wq, ws = O.quantize_rows_int8(np64(x))
    assert (npi(s) == ws).all()
    # r = 127 / m is off by at most 2^-23 of itself: quotients within 127 2^-23 of a tie may go either way
    quot = 127.0 * np64(x) / np.abs(np64(x)).max(axis=1, keepdims=True)
    free = np.abs(np.abs(quot - np.floor(quot)) - 0.5) > 2.0 ** -16
    assert (npi(q) == wq)[free].all() and (np.abs(npi(q) - wq) <= 1).all()


def test_leading_dimensions_and_given_outputs(lib):
    moe = lib
    w = torch.randn(3, 10, 64, generator=torch.Generator().manual_seed(0))
    q, s = moe.moe_quantize_int8(w.to(DEV))
    assert q.shape == (3, 10, 64) and s.shape == (3, 10)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    moe.moe_quantize_int8(w.to(DEV), q=q2, scales=s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert moe.moe_quantize_int8(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))[0].shape == (0, 64)


# ---------------------------------------------------------------- grouping with codes


@pytest.mark.parametrize("T,E,k,d,cap,skew", [(1, 8, 2, 64, 0, 0.0), (300, 8, 2, 80, 0, 0.0), (1000, 192, 4, 768, 27, 1.2),
                                              (70, 33, 5, 1040, 0, 1.0), (40, 16, 16, 16, 3, 0.0), (9, 48, 8, 7168, 0, 0.0),
                                              # either side of the one-launch form's 4096 pairs, its three widths
                                              (4096, 512, 1, 64, 0, 0.5), (4097, 512, 1, 64, 0, 0.5),
                                              (256, 20, 16, 528, 60, 0.6), (257, 20, 16, 528, 60, 0.6),
                                              (100, 7, 5, 1056, 0, 0.0), (256, 384, 8, 256, 2, 1.0),
                                              (600, 16, 8, 1056, 250, 0.5)])
def test_permute_int8_matches_the_oracle(lib, T, E, k, d, cap, skew):
    moe = lib
    s = moe.MoeShape(T=T, d=d, E=E, k=k, H=16, capacity=cap, wfmt=moe.WFMT_INT8)
    idx = synth.draw_topk_idx(T, E, k, seed=T, skew=skew)
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).bfloat16()
    r = moe.moe_permute_int8(s, x.to(DEV), idx.to(DEV), full=True)
    ref = O.permute(idx.numpy(), E, cap)
    for key in ("slot_pos", "kept", "offsets", "row_src", "counts"):
        assert (npi(r[key]) == ref[key]).all(), key
    assert (npi(r["drop_mask"]) == ref["drop"]).all()
    q, sc = O.quantize_rows_int8(np64(x))
    f = ref["row_src"] >= 0
    assert (npi(r["xq_perm"])[f] == q[ref["row_src"][f] // k]).all()
    assert (npi(r["xs_perm"])[f] == sc[ref["row_src"][f] // k]).all()


# ---------------------------------------------------------------- the expert step


def _experts(n, d, H, seed=0):
    g = torch.Generator().manual_seed(seed)
    w13 = torch.randn(n, 2 * H, d, generator=g) / d ** 0.5
    w2 = torch.randn(n, d, H, generator=g) / H ** 0.5
    out = {}
    for name, w in (("w13", w13), ("w2", w2)):
        q, s = O.quantize_rows_int8(np64(w).reshape(-1, w.shape[-1]))
        out[name] = torch.from_numpy(q.astype(np.int8)).view(w.shape)
        out["s" + name[1:]] = torch.from_numpy(s).view(w.shape[:-1])
    return out


def _check_rows(got, xq, xs, w, e, act, what):
    y, h, hq, hs = O.expert_ffn_int8(xq, xs, np64(w["w13"][e]), np64(w["s13"][e]), np64(w["w2"][e]), np64(w["s2"][e]), act)
    slack = (2.0 ** -7 * np.abs(h) + hs.astype(np.float64)[:, None]) @ (np.abs(np64(w["w2"][e])) * np64(w["s2"][e])[:, None]).T
    assert np.isfinite(got).all(), what
    assert (np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + slack).all(), what
    return y


def _ffn_case(moe, d, H, act, rows, starts=None, R=None, seed=0, flags=0, check=True):
    n = len(rows)
    rows = np.asarray(rows)
    starts = np.cumsum(rows) - rows if starts is None else np.asarray(starts)
    R = int((starts + rows).max()) if R is None else R
    x = torch.randn(max(R, 1), d, generator=torch.Generator().manual_seed(seed + 1)).bfloat16()[:R]
    w = _experts(n, d, H, seed)
    s = moe.MoeShape(T=max(R, 1), d=d, E=n, k=1, H=H, act=act, wfmt=moe.WFMT_INT8, flags=flags)
    q, sc = O.quantize_rows_int8(np64(x))
    dv = {k: v.to(DEV) for k, v in w.items()}
    xq, xs = torch.from_numpy(q.astype(np.int8)).to(DEV), torch.from_numpy(sc).to(DEV)
    y0 = torch.full((R, d), 3.0, dtype=torch.bfloat16, device=DEV)
    i32 = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).to(DEV)  # noqa: E731
    y = moe.moe_expert_ffn_int8(s, xq, xs, dv["w13"], dv["s13"], dv["w2"], dv["s2"], group_start=i32(starts),
                                group_rows=i32(rows), y=y0)
    torch.cuda.synchronize()
    assert moe.moe_get_status()[0] == 0
    got = np64(y)
    inside = np.zeros(R, bool)
    for e in range(n):
        a, b = int(starts[e]), int(starts[e] + rows[e])
        inside[a:b] = True
        if b > a and check:
            want = _check_rows(got[a:b], q[a:b], sc[a:b], w, e, act, f"group {e}")
            if b - a >= 64 and d * (b - a) >= 4096:
                assert rel_frob(got[a:b], want) <= REL_FROB
    assert (got[~inside] == 3.0).all(), "rows outside every group were written"
    return s, x, dv, starts, rows, y


# narrow and wide column tiles; reductions under, at and past one 128-code step; widths that are no multiple of a
# tile; empty groups, groups of one row, of a whole tile, past it, and past two; both hidden widths of the bf16
# fused kernel; both activations
@pytest.mark.parametrize("d,H,act,rows", [(16, 16, 0, [1]), (16, 16, 1, [0, 3, 0, 1]), (80, 48, 0, [5, 0, 128, 129]),
                                          (64, 128, 0, [70, 33, 0, 257]), (272, 256, 0, [300, 1, 31, 32, 33]),
                                          (2064, 128, 0, [5, 200]), (784, 256, 1, [9] * 45),
                                          (768, 256, 0, [700, 512, 64, 0, 90]), (768, 128, 1, [400, 300]),
                                          (128, 1040, 1, [17, 140]), (1040, 80, 0, [1, 2, 0, 4]), (256, 2048, 1, [130, 260])])
def test_expert_ffn_matches_the_oracle(lib, d, H, act, rows):
    _ffn_case(lib, d, H, act, rows, seed=d + H)


# more row tiles than the GPU has SMs, so that every CTA (pair) takes several: the fused kernel on pairs and single CTAs
# (hidden 128 and 256, one to three jobs of 256 output columns), the two kernels on both, ragged groups throughout
@pytest.mark.parametrize("d,H,act,groups,rows,flags", [(272, 256, 0, 5, 9000, 0), (528, 128, 1, 4, 11000, 0),
                                                       (768, 256, 0, 3, 15000, 0), (48, 256, 1, 6, 7000, 1),
                                                       (64, 128, 0, 500, 3, 0), (336, 256, 0, 400, 5, 0),
                                                       (64, 320, 0, 6, 7000, 0), (80, 192, 1, 450, 2, 0)])
def test_several_tiles_per_cta(lib, d, H, act, groups, rows, flags):
    moe = lib
    g = torch.Generator().manual_seed(d)
    sizes = torch.randint(rows // 2, rows + 1, (groups,), generator=g).tolist()
    sizes[1] = 0
    s, x, dv, starts, ro, y = _ffn_case(moe, d, H, act, sizes, seed=H, flags=flags, check=False)
    q, sc = O.quantize_rows_int8(np64(x))
    w = {k_: v.cpu() for k_, v in dv.items()}
    got = np64(y)
    for e in range(groups):
        a, b = int(starts[e]), int(starts[e] + ro[e])
        if b > a:
            _check_rows(got[a:b], q[a:b], sc[a:b], w, e, act, f"group {e}")


def test_pair_and_single_tiles_give_the_same_bits(lib):
    moe = lib
    kw = dict(d=400, H=256, act=0, rows=[500, 260, 129, 1000], seed=3)
    a, b = _ffn_case(moe, **kw)[5], _ffn_case(moe, flags=moe.FLAG_SINGLE_CTA_GEMM, **kw)[5]
    assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [100, 200])
@pytest.mark.parametrize("act", [0, 1])
def test_fused_and_separate_kernels_give_the_same_bits(lib, rows, act):
    """One expert of 768 x 256 alone is run by separate kernels, 60 copies of it with the same rows by the fused one, on
    single CTAs (100 rows a group) and on pairs (200)."""
    moe = lib
    d, H, n = 768, 256, 60
    w = _experts(1, d, H, 7)
    x = torch.randn(rows, d, generator=torch.Generator().manual_seed(rows)).bfloat16().to(DEV)
    xq, xs = moe.moe_quantize_int8(x)
    s = moe.MoeShape(T=n * rows, d=d, E=n, k=1, H=H, act=act, wfmt=moe.WFMT_INT8)
    one = {k_: v.to(DEV) for k_, v in w.items()}
    many = {k_: v.to(DEV).repeat(n, *[1] * (v.dim() - 1)).contiguous() for k_, v in w.items()}
    st = (torch.arange(n, dtype=torch.int32) * rows).to(DEV)
    ro = torch.full((n,), rows, dtype=torch.int32, device=DEV)
    before = moe.moe_launch_count()
    a = moe.moe_expert_ffn_int8(s, xq, xs, **one)
    mid = moe.moe_launch_count()
    b = moe.moe_expert_ffn_int8(s, xq.repeat(n, 1), xs.repeat(n), **many, group_start=st, group_rows=ro)
    assert (mid - before, moe.moe_launch_count() - mid) == (3, 1)
    assert torch.equal(b.view(n, rows, d), a.expand(n, rows, d))


@pytest.mark.parametrize("R,d,H,act", [(3000, 192, 512, 0), (129, 1040, 320, 1), (1, 4096, 1024, 0)])
def test_one_dense_group_without_a_table(lib, R, d, H, act):
    moe = lib
    w = _experts(1, d, H, 3)
    x = torch.randn(R, d, generator=torch.Generator().manual_seed(R)).bfloat16()
    s = moe.MoeShape(T=R, d=d, E=1, k=1, H=H, act=act, wfmt=moe.WFMT_INT8)
    dv = {k_: v.to(DEV) for k_, v in w.items()}
    got = moe.moe_expert_ffn(s, x.to(DEV), dv["w13"], dv["w2"], s13=dv["s13"], s2=dv["s2"])[1]
    q, sc = O.quantize_rows_int8(np64(x))
    _check_rows(np64(got), q, sc, w, 0, act, "dense")


def test_slabs_overlong_groups_and_untouched_rows(lib):
    moe = lib
    # capacity slabs with rows behind the filled ones; groups out of order; the last one runs past the buffer
    _ffn_case(moe, 96, 64, 0, [10, 0, 40, 7], starts=[0, 40, 80, 120], R=160)
    _ffn_case(moe, 96, 64, 1, [10, 20, 30], starts=[50, 0, 20], R=64)
    w = _experts(2, 64, 32)
    dv = {k: v.to(DEV) for k, v in w.items()}
    s = moe.MoeShape(T=20, d=64, E=2, k=1, H=32, wfmt=moe.WFMT_INT8)
    x = torch.randn(20, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    xq, xs = moe.moe_quantize_int8(x)
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    full = moe.moe_expert_ffn_int8(s, xq, xs, **dv, group_start=t(0, 8), group_rows=t(8, 12))
    clip = moe.moe_expert_ffn_int8(s, xq, xs, **dv, group_start=t(0, 8), group_rows=t(8, 1000))
    assert torch.equal(full, clip)
    none = torch.full_like(full, 2.0)
    moe.moe_expert_ffn_int8(s, xq, xs, **dv, group_start=t(-5, 20), group_rows=t(8, 4), y=none)
    moe.moe_expert_ffn_int8(s, xq, xs, **dv, group_start=t(0, 0), group_rows=t(0, -3), y=none)
    assert (none == 2.0).all()


def test_largest_codes_and_zero_rows(lib):
    """All codes at their limits over a long reduction: sums of 127^2 K = 1.3e8, beyond 24 bits; and a zero row."""
    moe = lib
    d, H, n = 8192, 32, 3
    s = moe.MoeShape(T=n, d=d, E=1, k=1, H=H, wfmt=moe.WFMT_INT8)
    xq = torch.full((n, d), 127, dtype=torch.int8)
    xq[1], xq[2] = -127, 0
    xs = torch.tensor([2.0 ** -10, 2.0 ** -10, 0.0])
    w13 = torch.full((1, 2 * H, d), 127, dtype=torch.int8)
    w13[0, H:, ::2] = -128
    s13 = torch.full((1, 2 * H), 2.0 ** -16)
    w2 = torch.full((1, d, H), -128, dtype=torch.int8)
    s2 = torch.full((1, d), 2.0 ** -5)
    dv = [t.to(DEV) for t in (xq, xs, w13, s13, w2, s2)]
    got = np64(moe.moe_expert_ffn_int8(s, *dv))
    w = dict(w13=w13, s13=s13, w2=w2, s2=s2)
    want = _check_rows(got, np64(xq), np64(xs).astype(np.float32), w, 0, 0, "limits")
    assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want)).all() and (got[2] == 0).all() and (got[0] != 0).all()


def test_infinite_token_stays_in_its_row(lib):
    moe = lib
    w = {k: v.to(DEV) for k, v in _experts(1, 64, 128).items()}
    s = moe.MoeShape(T=200, d=64, E=1, k=1, H=128, wfmt=moe.WFMT_INT8)
    x = torch.randn(200, 64, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    good = moe.moe_expert_ffn(s, x, w["w13"], w["w2"], s13=w["s13"], s2=w["s2"])[1]
    x[50, 3], x[150, 9] = float("inf"), float("nan")
    bad = moe.moe_expert_ffn(s, x, w["w13"], w["w2"], s13=w["s13"], s2=w["s2"])[1]
    keep = torch.ones(200, dtype=torch.bool, device=DEV)
    keep[50] = keep[150] = False
    assert torch.equal(good[keep], bad[keep]) and not bad[50].isfinite().any() and not bad[150].isfinite().any()


def test_bf16_entry_quantises_and_runs_the_same(lib):
    moe = lib
    s, x, dv, starts, rows, y = _ffn_case(moe, 256, 64, 1, [33, 0, 200])
    t = lambda v: torch.from_numpy(np.asarray(v).astype(np.int32)).to(DEV)  # noqa: E731
    h, y2 = moe.moe_expert_ffn(s, x.to(DEV), dv["w13"], dv["w2"], s13=dv["s13"], s2=dv["s2"], group_start=t(starts),
                               group_rows=t(rows))
    assert h is None and torch.equal(y, y2)
    assert moe.moe_expert_ffn_int8(s, torch.empty(0, 256, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV),
                                   dv["w13"], dv["s13"], dv["w2"], dv["s2"], group_start=t([0, 0, 0]),
                                   group_rows=t([0, 0, 0])).shape == (0, 256)


def test_outputs_and_inputs_on_16_byte_boundaries(lib):
    moe = lib
    s, x, dv, starts, rows, y = _ffn_case(moe, 208, 64, 0, [33, 0, 200])
    t = lambda v: torch.from_numpy(np.asarray(v).astype(np.int32)).to(DEV)  # noqa: E731

    def shifted(a, n):   # the same values n elements behind a 256-byte boundary
        b = torch.empty(a.numel() + n, dtype=a.dtype, device=DEV)
        b[n:] = a.reshape(-1)
        return b[n:].view(a.shape)
    xq, xs = moe.moe_quantize_int8(shifted(x.to(DEV), 8))
    out = shifted(torch.zeros_like(y), 8)
    w = {k_: shifted(v, 16 // v.element_size()) for k_, v in dv.items()}
    got = moe.moe_expert_ffn_int8(s, shifted(xq, 16), shifted(xs, 4), w["w13"], w["s13"], w["w2"], w["s2"],
                                  group_start=t(starts), group_rows=t(rows), y=out)
    assert got.data_ptr() % 32 == 16 and torch.equal(got, y)


# ---------------------------------------------------------------- the layer


def _layer(moe, T, d, E, k, H, H_s=0, cap=0, act=0, seed=0):
    wl = synth.Workload("int8", T=T, d=d, E=E, k=k, H=H, H_s=H_s, act=act)
    inp = synth.make_inputs(wl, seed=seed, with_expert_weights=False)
    w = _experts(E, d, H, seed)
    sh = _experts(1, d, H_s, seed + 9) if H_s else {}
    s = moe.MoeShape(T=T, d=d, E=E, k=k, H=H, H_s=H_s, capacity=cap, act=act, wfmt=moe.WFMT_INT8)
    dv = dict(x=inp["x"].to(DEV), w_router=inp["w_router"].to(DEV), **{a: v.to(DEV) for a, v in w.items()},
              **{a + "_sh": v.to(DEV) for a, v in sh.items()})
    return s, inp, w, sh, dv


def _forward(moe, s, dv, **kw):
    ex = {a: dv[a] for a in ("s13", "s2", "w13_sh", "s13_sh", "w2_sh", "s2_sh") if a in dv}
    return moe.moe_forward(s, dv["x"], dv["w_router"], dv["w13"], dv["w2"], routing=True, **ex, **kw)


@pytest.mark.parametrize("T,d,E,k,H,H_s,cap,act", [(256, 64, 8, 2, 128, 64, 0, 0), (1, 512, 16, 4, 256, 0, 0, 0),
                                                   (500, 192, 24, 3, 80, 48, 70, 1), (700, 128, 4, 2, 256, 128, 0, 0),
                                                   (64, 1024, 48, 8, 512, 256, 0, 1),
                                                   (520, 1056, 16, 8, 64, 32, 300, 0)])
def test_layer_matches_the_oracle_and_its_steps(lib, T, d, E, k, H, H_s, cap, act):
    moe = lib
    s, inp, w, sh, dv = _layer(moe, T, d, E, k, H, H_s, cap, act, seed=T)
    r = _forward(moe, s, dv)
    idx, gates = npi(r["topk_idx"]), np64(r["topk_w"])
    # the layer from its own routing decision, in float64
    p = O.permute(idx, E, cap)
    q, sc = O.quantize_rows_int8(np64(inp["x"]))
    y = np.zeros((E * cap if cap else T * k, d))
    for e in range(E):
        rows = np.nonzero((p["slot_pos"] >= 0) & (idx == e))
        at = p["slot_pos"][rows]
        if at.size:
            y[at] = O.expert_ffn_int8(q[rows[0]], sc[rows[0]], np64(w["w13"][e]), np64(w["s13"][e]), np64(w["w2"][e]),
                                      np64(w["s2"][e]), act)[0]
    ysh = O.expert_ffn_int8(q, sc, np64(sh["w13"][0]), np64(sh["s13"][0]), np64(sh["w2"][0]), np64(sh["s2"][0]), act)[0] \
        if H_s else None
    assert_out_close(np64(r["out"]), O.combine(y, p["slot_pos"], gates, ysh), "int8 layer")
    assert (npi(r["drop_mask"]) == p["drop"]).all()
    # the same bits from the steps, and with the shared expert on a second stream
    g = moe.moe_permute_int8(s, dv["x"], r["topk_idx"])
    yp = moe.moe_expert_ffn_int8(s, g["xq_perm"], g["xs_perm"], dv["w13"], dv["s13"], dv["w2"], dv["s2"],
                                 group_start=g["offsets"], group_rows=g["kept"])
    yshd = None
    if H_s:
        xq, xs = moe.moe_quantize_int8(dv["x"])
        yshd = moe.moe_expert_ffn_int8(s, xq, xs, dv["w13_sh"], dv["s13_sh"], dv["w2_sh"], dv["s2_sh"], hidden=H_s)
    assert torch.equal(moe.moe_combine(s, yp, g["slot_pos"], r["topk_w"], yshd), r["out"])
    two = _forward(moe, s, dv, side_stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(two["out"], r["out"]) and moe.moe_get_status()[0] == 0


def test_layer_in_a_graph_and_on_another_stream(lib):
    moe = lib
    s, inp, w, sh, dv = _layer(moe, 300, 128, 12, 3, 256, 64, 90)
    ws = torch.empty(moe.moe_workspace_size(s), dtype=torch.uint8, device=DEV)
    want = _forward(moe, s, dv, ws=ws)["out"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _forward(moe, s, dv, ws=ws)["out"]
    ws.fill_(255)                                     # whatever the scratch held
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # with the shared expert on a second stream, captured too
    two, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(two):
        out2 = _forward(moe, s, dv, ws=ws, side_stream=side)["out"]
    ws.fill_(255)
    two.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, want)
    # the steps on a stream of their own, scratch and outputs allocated for it
    idx = _forward(moe, s, dv, ws=ws)["topk_idx"]
    a = moe.moe_permute_int8(s, dv["x"], idx, full=True)
    ya = moe.moe_expert_ffn_int8(s, a["xq_perm"], a["xs_perm"], dv["w13"], dv["s13"], dv["w2"], dv["s2"],
                                 group_start=a["offsets"], group_rows=a["kept"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = moe.moe_permute_int8(s, dv["x"], idx, stream=side)
    yb = moe.moe_expert_ffn_int8(s, b["xq_perm"], b["xs_perm"], dv["w13"], dv["s13"], dv["w2"], dv["s2"],
                                 group_start=b["offsets"], group_rows=b["kept"], stream=side)
    side.synchronize()
    f = (npi(a["row_src"]) >= 0)
    assert torch.equal(a["slot_pos"], b["slot_pos"]) and torch.equal(ya[torch.from_numpy(f)], yb[torch.from_numpy(f)])


def test_two_calls_at_once_with_their_own_scratch(lib):
    """Two layers on two streams at a time: each call of the steps has scratch of its own."""
    moe = lib
    a, b = _ffn_case(moe, 256, 256, 0, [200, 300, 0, 64], seed=1), _ffn_case(moe, 384, 512, 1, [64, 3, 500], seed=2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for _ in range(5):
        for (s, x, dv, st, ro, y), stream in ((a, sa), (b, sb)):
            i32 = lambda v: torch.from_numpy(v.astype(np.int32)).to(DEV)  # noqa: E731
            xd, st_, ro_ = x.to(DEV), i32(st), i32(ro)
            torch.cuda.current_stream().synchronize()
            outs.append((moe.moe_expert_ffn(s, xd, dv["w13"], dv["w2"], s13=dv["s13"], s2=dv["s2"], group_start=st_,
                                            group_rows=ro_, stream=stream)[1], y, (xd, st_, ro_)))
    torch.cuda.synchronize()
    assert all(torch.equal(got, want) for got, want, _ in outs)


def test_untouched_rows_of_the_codes(lib):
    """Through the C ABI: rows that no token fills keep what the caller's buffers held."""
    moe = lib
    L = moe.load()
    T, E, k, d, cap = 50, 6, 2, 64, 30
    s = moe.MoeShape(T=T, d=d, E=E, k=k, H=16, capacity=cap, wfmt=moe.WFMT_INT8)
    idx = synth.draw_topk_idx(T, E, k, seed=1).to(DEV)
    x = torch.randn(T, d, device=DEV).bfloat16()
    R = E * cap
    q = torch.full((R, d), 99, dtype=torch.int8, device=DEV)
    sc = torch.full((R,), 5.0, device=DEV)
    i32 = lambda *sh: torch.empty(*sh, dtype=torch.int32, device=DEV)  # noqa: E731
    slot, kept, offs = i32(T, k), i32(E), i32(E + 1)
    ws = torch.empty(moe.moe_workspace_size(s), dtype=torch.uint8, device=DEV)
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert L.moe_permute_int8(ctypes.byref(s), P(x), P(idx), P(slot), None, None, P(kept), P(offs), None, P(q), P(sc),
                              P(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    filled = torch.zeros(R, dtype=torch.bool)
    filled[slot.cpu()[slot.cpu() >= 0].long()] = True
    assert (q.cpu()[~filled] == 99).all() and (sc.cpu()[~filled] == 5.0).all() and (sc.cpu()[filled] != 5.0).all()


def test_expert_parallel_forward_of_int8_experts_on_one_rank(lib):
    """moe_forward_ep with one rank and 8-bit experts gives moe_forward's bits, with and without a capacity."""
    import socket
    import torch.distributed as dist
    from sparse_mixture_experts_expert_b200.ep import moe_forward_ep
    moe = lib
    with socket.socket() as so:
        so.bind(("127.0.0.1", 0))
        port = so.getsockname()[1]
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1)
    try:
        for cap in (0, 40):
            s, inp, w, sh, dv = _layer(moe, 150, 128, 8, 2, 128, 64, cap)
            out, _, _ = moe_forward_ep(s, dv["x"], dv["w_router"], dv["w13"], dv["w2"], s13_local=dv["s13"],
                                       s2_local=dv["s2"], w13_sh=dv["w13_sh"], s13_sh=dv["s13_sh"], w2_sh=dv["w2_sh"],
                                       s2_sh=dv["s2_sh"])
            assert torch.equal(out, _forward(moe, s, dv)["out"])
    finally:
        dist.destroy_process_group()
