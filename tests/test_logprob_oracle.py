"""Pins of the log-probability oracle."""
import numpy as np
import pytest

import oracle.logprob_oracle as P


def _case(T=5, V=7, seed=0):
    rng = np.random.default_rng(seed)
    return 2 * rng.standard_normal((T, V)), np.array([0, 6, 3, -1, 7])


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_against_the_definition_and_differences(scale):
    z, target = _case()
    rng = np.random.default_rng(1)
    dl, de = rng.standard_normal(5), rng.standard_normal(5)
    f = P.fwd(z, target, scale)
    p = np.exp(scale * z) / np.exp(scale * z).sum(1, keepdims=True)
    assert np.allclose(f["lse"], np.log(np.exp(scale * z).sum(1)))
    assert np.allclose(f["entropy"], -(p * np.log(p)).sum(1))
    assert np.allclose(f["logp"][:3], np.log(p)[[0, 1, 2], [0, 6, 3]]) and (f["logp"][3:] == 0).all()
    got = P.bwd(z, target, f["lse"], f["entropy"], dl, de, scale)["dlogits"]

    def value():
        r = P.fwd(z, target, scale)
        return (dl * r["logp"] + de * r["entropy"]).sum()

    h = 1e-6
    for t in range(5):
        for j in range(7):
            keep = z[t, j]
            z[t, j] = keep + h
            up = value()
            z[t, j] = keep - h
            down = value()
            z[t, j] = keep
            assert abs((up - down) / (2 * h) - got[t, j]) < 1e-8
    assert np.allclose(got.sum(1), 0, atol=1e-12)


def test_masked_and_broken_rows():
    inf, nan = np.inf, np.nan
    z = np.array([[-inf] * 4, [-inf, 1.0, -inf, 1.0], [0.0, nan, 1.0, 2.0], [0.0, inf, 1.0, 2.0], [5.0] * 4])
    f = P.fwd(z, np.array([0, 1, 2, 3, 2]), 1.0)
    assert f["lse"][0] == -inf and f["logp"][0] == -inf and f["entropy"][0] == 0
    assert np.allclose([f["logp"][1], f["entropy"][1]], [-np.log(2), np.log(2)])
    assert np.isnan([f[n][t] for n in f for t in (2, 3)]).all()
    assert np.allclose([f["lse"][4], f["entropy"][4]], [5 + np.log(4), np.log(4)])
    d = P.bwd(z[:2], np.array([0, 1]), f["lse"], f["entropy"], np.ones(2), np.ones(2), 1.0)["dlogits"]
    assert (d[0] == 0).all() and np.isfinite(d[1]).all() and (d[1, [0, 2]] == 0).all()
    assert P.fwd(np.full((1, 3), -3.4e38), np.array([1]), 1.0)["entropy"][0] == pytest.approx(np.log(3))


def test_order_of_the_largest():
    z = np.array([[1.0, 3.0, 3.0, -0.0, 0.0, np.nan, -np.inf]])
    assert P.top(z, 7).tolist() == [[5, 1, 2, 0, 3, 4, 6]]
