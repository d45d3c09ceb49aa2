"""Pins of the packed-attention oracle."""
import math

import numpy as np

import oracle.packed_oracle as A

T, Hq, Hk, DH = 13, 4, 2, 3
OFFS = [1, 1, 6, 7, 7, 12]  # empty sequences, one token, a row in front and one behind
SCALE = 0.7


def _case(seed=0):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal((T, H * DH)) for H in (Hq, Hk, Hk, Hq)]


def test_against_a_loop_over_elements():
    q, k, v, _ = _case()
    got = A.attn_fwd(q, k, v, OFFS, Hq, Hk, SCALE)
    seen = np.zeros(T, dtype=bool)
    for b, e in zip(OFFS, OFFS[1:]):
        for t in range(b, e):
            seen[t] = True
            for h in range(Hq):
                s = [SCALE * sum(q[t, h * DH + c] * k[j, h // 2 * DH + c] for c in range(DH)) for j in range(b, t + 1)]
                total = sum(math.exp(x) for x in s)
                assert abs(got["lse"][t, h] - math.log(total)) < 1e-12
                for c in range(DH):
                    want = sum(math.exp(x) / total * v[b + j, h // 2 * DH + c] for j, x in enumerate(s))
                    assert abs(got["o"][t, h * DH + c] - want) < 1e-12
    assert np.isnan(got["o"][~seen]).all() and np.isnan(got["lse"][~seen]).all() and (~seen).sum() == 2


def test_gradients_against_differences():
    q, k, v, g = _case(1)
    rows = np.arange(1, 12)

    def value():
        return (A.attn_fwd(q, k, v, OFFS, Hq, Hk, SCALE)["o"][rows] * g[rows]).sum()

    f = A.attn_fwd(q, k, v, OFFS, Hq, Hk, SCALE)
    got = A.attn_bwd(q, k, v, f["o"], f["lse"], g, OFFS, Hq, Hk, SCALE)
    h = 1e-6
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for t in rows:
            for c in range(x.shape[1]):
                keep = x[t, c]
                x[t, c] = keep + h
                up = value()
                x[t, c] = keep - h
                down = value()
                x[t, c] = keep
                assert abs((up - down) / (2 * h) - got[name][t, c]) < 1e-8


def test_sequences_do_not_see_each_other_nor_rows_of_none():
    q, k, v, g = _case(2)
    f = A.attn_fwd(q, k, v, OFFS, Hq, Hk, SCALE)
    for x in (q, k, v, g):
        x[[0, 12]] = np.nan
    again = A.attn_fwd(q, k, v, OFFS, Hq, Hk, SCALE)
    assert np.array_equal(f["o"][1:12], again["o"][1:12])
    part = A.attn_fwd(q[6:7], k[6:7], v[6:7], [0, 1], Hq, Hk, SCALE)
    assert np.allclose(part["o"], f["o"][6:7], rtol=0, atol=1e-15)
    assert np.allclose(part["o"].reshape(Hq, DH), np.repeat(v[6].reshape(Hk, DH), 2, 0))  # one key: its value


def test_rounding_bounds_hold_for_a_rounded_backward():
    q, k, v, g = _case(3)
    f = A.attn_fwd(q, k, v, OFFS, Hq, Hk, SCALE)
    want = A.attn_bwd(q, k, v, f["o"], f["lse"], g, OFFS, Hq, Hk, SCALE, rel_d=1e-3)
    got = A.attn_bwd(q, k, v, f["o"] * (1 + 1e-3 * np.sign(g) * np.sign(f["o"])), f["lse"], g, OFFS, Hq, Hk, SCALE)
    for n in ("dq", "dk"):
        off = np.abs(got[n] - want[n])[1:12]
        assert (off <= want["err_" + n][1:12] * (1 + 1e-9) + 1e-15).all() and off.max() > 1e-5
