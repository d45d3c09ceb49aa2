"""Pins of the fp64 oracle for the query/key norm and rotation and for gradient clipping (CPU)."""
import math

import numpy as np
import pytest

import oracle.qk_oracle as Q

CASES = [  # dh, rot, sections, layout, gain
    (8, 8, (4,), "half", True),
    (16, 8, (1, 3), "pairs", True),
    (24, 16, (3, 3, 2), "half", True),
    (16, 16, (2, 2, 2, 2), "pairs", False),
    (8, 0, (0,), "half", True),
]


def _case(dh, rot, sec, gain, T=3, H=2, seed=0):
    rng = np.random.default_rng(seed)
    x, dy = rng.standard_normal((T, H * dh)), rng.standard_normal((T, H * dh))
    g = 1 + 0.1 * rng.standard_normal(dh) if gain else None
    pos = rng.integers(-50, 1000, (len(sec), T))
    freq = [10.0 ** (-p / max(1, rot // 2)) for p in range(rot // 2)]
    return x, dy, g, Q.angles(pos, freq, sec)


def test_a_quarter_turn_by_hand():
    theta = np.array([[math.pi / 2]])
    half = Q.qk_fwd(np.array([[1.0, 2.0, 3.0]]), None, theta, 3, 2, "half", 0.0)
    assert np.allclose(half, [[-2.0, 1.0, 3.0]])
    two = np.array([[0.0, math.pi / 2]])
    adj = Q.qk_fwd(np.array([[1.0, 2.0, 3.0, 4.0]]), None, two, 4, 4, "pairs", 0.0)
    assert np.allclose(adj, [[1.0, 2.0, -4.0, 3.0]])
    half = Q.qk_fwd(np.array([[1.0, 2.0, 3.0, 4.0]]), None, two, 4, 4, "half", 0.0)
    assert np.allclose(half, [[1.0, -4.0, 3.0, 2.0]])


def test_angles_by_axis_and_far_positions():
    th = Q.angles(np.array([[2, 5], [7, -1]]), [0.25, 0.5, 0.125], (1, 2))
    want = np.array([[0.5, 3.5, 0.875], [1.25, -0.5, -0.125]]) % (2 * math.pi)
    assert np.allclose(th, want, atol=1e-14)
    big = (1 << 31) - 1
    assert Q.angles(np.array([[big]]), [1.0], (1,))[0, 0] == pytest.approx(math.fmod(big, 2 * math.pi), abs=1e-6)


def test_norm_has_unit_mean_square_and_inner_products_depend_on_distance():
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 1, 16))
    freq = [1.0 / (p + 1) for p in range(8)]
    n = Q.qk_fwd(x, np.ones(16), Q.angles(np.array([[9]]), freq, (8,)), 16, 16, "half", 0.0)
    assert np.mean(n ** 2) == pytest.approx(1.0, abs=1e-12)

    def score(a, b, layout):
        th = [Q.angles(np.array([[p]]), freq, (8,)) for p in (a, b)]
        return float(np.sum(Q.qk_fwd(x, None, th[0], 16, 16, layout, 0.0) * Q.qk_fwd(y, None, th[1], 16, 16, layout, 0.0)))

    for layout in ("half", "pairs"):
        assert score(3, 10, layout) == pytest.approx(score(1003, 1010, layout), abs=1e-9)
        assert abs(score(3, 10, layout) - score(3, 11, layout)) > 1e-3


@pytest.mark.parametrize("dh,rot,sec,layout,gain", CASES)
def test_gradients_match_finite_differences(dh, rot, sec, layout, gain):
    x, dy, g, th = _case(dh, rot, sec, gain)
    eps = 1e-3

    def loss(x_, g_):
        return float(np.sum(Q.qk_fwd(x_, g_, th, dh, rot, layout, eps) * dy))

    got = Q.qk_bwd(x, g, th, dy, dh, rot, layout, eps)
    h = 1e-6
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = h
        assert got["dx"][idx] == pytest.approx((loss(x + e, g) - loss(x - e, g)) / (2 * h), abs=2e-7)
    if gain:
        for c in range(dh):
            e = np.zeros(dh)
            e[c] = h
            assert got["dg"][c] == pytest.approx((loss(x, g + e) - loss(x, g - e)) / (2 * h), abs=2e-7)


def test_clip_by_hand():
    norm, scale, out = Q.clip([np.array([3.0]), np.zeros(0), np.array([0.0, 4.0])], 1.0)
    assert norm == pytest.approx(5.0) and scale == pytest.approx(1 / 5.000001)
    assert out[2][1] == pytest.approx(0.8, rel=1e-6)
    assert Q.clip([np.array([3.0, 4.0])], 7.0)[1] == 1.0
    assert Q.clip([np.full(4, 1e200)], 1.0)[0] == pytest.approx(2e200)


def test_block_gradients_match_finite_differences():
    """The block with norm and rotation of q and k: dx, both norms' gains and sampled weights by central differences."""
    rng = np.random.default_rng(3)
    b, s, H, dh, f, ra, rm = 1, 4, 2, 8, 12, 6, 5
    d, T, eps = H * dh, b * s, 1e-3
    W = {"g_attn": 1 + 0.1 * rng.standard_normal(d), "g_mlp": 1 + 0.1 * rng.standard_normal(d)}
    for n in "qkvo":
        W[f"A_{n}"], W[f"B_{n}"] = rng.standard_normal((ra, d)) / d ** 0.5, rng.standard_normal((d, ra)) / ra ** 0.5
    for n, i, o in (("gate", d, f), ("up", d, f), ("down", f, d)):
        W[f"A_{n}"], W[f"B_{n}"] = rng.standard_normal((rm, i)) / i ** 0.5, rng.standard_normal((o, rm)) / rm ** 0.5
    x, G = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    pos = np.stack([np.arange(T) % s, rng.integers(0, 9, T)])
    rot = dict(theta=Q.angles(pos, [1.0, 0.3, 0.1], (2, 1)), rot=6, layout="half",
               gq=1 + 0.1 * rng.standard_normal(dh), gk=1 + 0.1 * rng.standard_normal(dh))

    def loss():
        return float(np.sum(Q.block_fwd(x, W, rot, b, s, H, dh, eps)[0] * G))

    gr = Q.block_bwd(W, Q.block_fwd(x, W, rot, b, s, H, dh, eps)[1], rot, G, b, s, H, dh, eps)
    h = 1e-6
    places = {"dx": x, "dgq": rot["gq"], "dgk": rot["gk"], "dg_attn": W["g_attn"]}
    places.update({f"d{m}_{n}": W[f"{m}_{n}"] for m in "AB" for n in "qkv"})
    for name, arr in places.items():
        for i in rng.choice(arr.size, min(12, arr.size), replace=False):
            idx = np.unravel_index(i, arr.shape)
            keep = arr[idx]
            arr[idx] = keep + h
            up = loss()
            arr[idx] = keep - h
            down = loss()
            arr[idx] = keep
            assert gr[name][idx] == pytest.approx((up - down) / (2 * h), rel=2e-5, abs=2e-6), (name, idx)
