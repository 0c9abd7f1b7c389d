"""Pins of the oracle's 8-bit rows, of its 8-bit experts, and of the gradients of the grouping and the combine."""

import numpy as np
import pytest

import oracle as O


def test_codes_of_a_worked_row():
    # m = 4: 127 x / m is 127, -63.5 (tie, to even), 31.75, 0, 0.49609375, -127
    x = np.array([[4.0, -2.0, 1.0, 0.0, 0.015625, -4.0]])
    q, s = O.quantize_rows_int8(x)
    assert q.tolist() == [[127.0, -64.0, 32.0, 0.0, 0.0, -127.0]]
    assert s.dtype == np.float32 and s[0] == np.float32(4.0) / np.float32(127.0)


def test_codes_stand_for_the_row_within_half_a_step():
    x = O.bf16_round(np.random.default_rng(0).normal(size=(50, 96))).astype(np.float64)
    q, s = O.quantize_rows_int8(x)
    assert np.abs(q).max() == 127 and (np.abs(q).max(axis=1) == 127).all()
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= s[:, None] * (0.5 + 1e-5)).all()


def test_empty_and_tiny_rows_have_no_scale():
    q, s = O.quantize_rows_int8(np.array([[0.0, -0.0], [2.0 ** -120, 0.0], [2.0 ** -119, 0.0]]))
    assert s[0] == 0 and s[1] == 0 and s[2] > 0 and q.tolist() == [[0, 0], [0, 0], [127, 0]]


@pytest.mark.parametrize("act", [0, 1])
def test_int8_expert_tends_to_the_float_expert(act):
    # with quantisation errors of half a step each, the 8-bit expert stays near the float one on the same values
    r = np.random.default_rng(1)
    x, w13, w2 = r.normal(size=(20, 64)), r.normal(size=(96, 64)) / 8, r.normal(size=(64, 48)) / 7
    xq, xs = O.quantize_rows_int8(x)
    q13, s13 = O.quantize_rows_int8(w13)
    q2, s2 = O.quantize_rows_int8(w2)
    y, h, hq, hs = O.expert_ffn_int8(xq, xs, q13, s13, q2, s2, act)
    assert (np.abs(hq * hs[:, None].astype(np.float64) - h) <= hs[:, None] * (0.5 + 1e-5)).all()
    want = O.expert_ffn(x, w13, w2, act)
    assert np.linalg.norm(y - want) <= 0.05 * np.linalg.norm(want)


@pytest.mark.parametrize("cap", [0, 3])
def test_sorting_gradients_against_differences(cap):
    # L = sum(G * combine(f(x_perm), w) + Gs * ysh) with f elementwise, through the oracle's grouping and combine
    r = np.random.default_rng(2)
    T, E, k, d = 7, 4, 2, 5
    idx = np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    p = O.permute(idx, E, cap)
    slot, R = p["slot_pos"], (E * cap if cap else T * k)
    x, w, G = r.normal(size=(T, d)), r.random((T, k)), r.normal(size=(T, d))

    def grouped(x):
        out = np.zeros((R, d))
        for t in range(T):
            for j in range(k):
                if slot[t, j] >= 0:
                    out[slot[t, j]] = x[t]
        return out

    def loss(x, w):
        return float((G * O.combine(np.sin(grouped(x)), slot, w)).sum())

    dy, dw = O.combine_backward(G, np.sin(grouped(x)), slot, w)
    dx = O.permute_backward(dy * np.cos(grouped(x)), slot)
    assert (slot < 0).any() == bool(cap)
    eps = 1e-6
    for grad, arr, pos in ((dx, x, 0), (dw, w, 1)):
        for at in np.ndindex(arr.shape):
            hi, lo = arr.copy(), arr.copy()
            hi[at] += eps
            lo[at] -= eps
            args = [(hi, w), (lo, w)] if pos == 0 else [(x, hi), (x, lo)]
            fd = (loss(*args[0]) - loss(*args[1])) / (2 * eps)
            assert abs(fd - grad[at]) <= 1e-7 * (1 + abs(fd)), (pos, at)
    assert (dw[slot < 0] == 0).all()
    assert np.abs(O.permute_backward(dy, slot, add=x) - O.permute_backward(dy, slot) - x).max() < 1e-14
