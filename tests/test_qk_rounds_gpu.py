"""lr_qk_fwd / lr_qk_bwd where a lane group takes several rounds of items, the last ones in part: more vectors than
the blocks that run at once hold, in both types and pairings, with 4 to 32 lanes to a vector and 1 to 4 axes.

Every output and input gradient is compared with fp64 (bounds as in test_qk_gpu.py: 40 and 100 roundings u = 2^-24 of
the magnitude of its terms, and half a step of its type).  The gains' gradients are sums over all vectors, where such
a bound (256 u of the sum of magnitudes) would hide what a few vectors add.  So they are also taken of vectors of
+1 and -1 whose upstream gradients are +1 or -1 in one vector of every `m`, and 0 in the others, for each of the m
choices: the sum is r times a whole number, the bound is 256 u of N / m terms of magnitude 2 at most, and m is
chosen so that it is below 1/4.  A vector that is left out or taken twice changes every channel by r, nearly 1.
"""
import dataclasses

import pytest
import torch

from rank_bottleneck_block_gb300 import inputs as I

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def _shape(T, Hq, Hk, dh, rot, axes, layout):
    each = rot // 2 // axes
    return I.QkShape(T=T, Hq=Hq, Hk=Hk, dh=dh, rot=rot, sec=(rot // 2 - each * (axes - 1),) + (each,) * (axes - 1),
                     layout=layout)


SHAPES = [  # lanes to a vector in the backward, bf16 / fp32
    _shape(40000, 1, 0, 64, 64, 1, "half"),     # 8 / 8
    _shape(16001, 5, 3, 40, 24, 3, "pairs"),    # 5 / 5
    _shape(30011, 4, 1, 80, 48, 3, "half"),     # 5 / 10
    _shape(20011, 7, 1, 72, 40, 2, "half"),     # 10 / 10
    _shape(9973, 5, 2, 80, 56, 1, "pairs"),     # 10 / 10
    _shape(30011, 3, 1, 128, 96, 4, "pairs"),   # 8 / 16
    _shape(25013, 3, 2, 64, 64, 2, "half"),     # 4 / 8
    _shape(60013, 2, 1, 16, 16, 1, "pairs"),    # 4 / 8
    _shape(5003, 37, 3, 96, 96, 4, "half"),     # 8 / 16, a token's heads in several items
    _shape(4999, 18, 3, 256, 128, 1, "half"),   # 16 / 32, the same
    _shape(6007, 19, 2, 160, 160, 3, "half"),   # 10 / 32, the same
    _shape(3001, 23, 1, 512, 512, 2, "pairs"),  # 32 / 32, the same
    _shape(2503, 50, 2, 336, 320, 4, "pairs"),  # 32 / 32, lanes without channels
]


def _name(s):
    return f"T{s.T}-{s.Hq}-{s.Hk}-dh{s.dh}-rot{s.rot}-{len(s.sec)}-{s.layout}"


def _turn(v, c, s, shape):
    """[T, H, dh] with the pairs of its first rot channels turned, and the sums of their magnitudes."""
    rot = shape.rot
    i, j = ((slice(0, rot // 2), slice(rot // 2, rot)) if shape.layout == "half" else
            (slice(0, rot, 2), slice(1, rot, 2)))
    y, mag = v.clone(), v.abs()
    y[..., i], y[..., j] = v[..., i] * c - v[..., j] * s, v[..., i] * s + v[..., j] * c
    both = mag[..., i] + mag[..., j]
    mag[..., i], mag[..., j] = both, both
    return y, mag


def _angles(shape, case):
    """Cosines and sines [T, 1, pairs] in fp64: positions below 1000 lose 1e-13."""
    axis = torch.repeat_interleave(torch.arange(len(shape.sec)), torch.tensor(shape.sec)).cuda()
    theta = case["pos"].double()[axis].T * torch.tensor(case["freq"], dtype=torch.float64, device="cuda")
    return theta.cos()[:, None], theta.sin()[:, None]


def _close(got, want, mag, dtype, k, what):
    off = (got.double() - want).abs() / (HALF[dtype] * want.abs() + k * U * mag + 1e-37)
    assert torch.isfinite(got).all() and float(off.max()) <= 1.0, (what, float(off.max()), int(off.argmax()))


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=_name)
def test_every_vector_matches_fp64(shape, dtype, norm):
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = dataclasses.replace(shape, dtype=dtype)
    case = I.make_qk_case(shape, seed=shape.T, norm=norm, device="cuda")
    run = QkRotary(shape, case)
    run.step()
    c, s = _angles(shape, case)
    for n, H, y, dx, dg in (("q", shape.Hq, run.qo, run.dq, run.dgq), ("k", shape.Hk, run.ko, run.dk, run.dgk)):
        if not H:
            continue
        x, dy = (case[m].double().view(shape.T, H, shape.dh) for m in (n, f"d{n}o"))
        dn, mag = _turn(dy, c, -s, shape)
        if not norm:
            want, size = _turn(x, c, s, shape)
            _close(y.view_as(x), want, size, dtype, 40, n + "o")
            _close(dx.view_as(x), dn, mag, dtype, 100, "d" + n)
            continue
        g = case["g" + n].double()
        r = (x.square().mean(-1, keepdim=True) + shape.eps).rsqrt()
        want, size = _turn(x * r * g, c, s, shape)
        _close(y.view_as(x), want, size, dtype, 40, n + "o")
        w, mw = dn * g, mag * g.abs()
        want = r * (w - x * r * r * (w * x).mean(-1, keepdim=True))
        size = r * (mw + x.abs() * r * r * (mw * x.abs()).mean(-1, keepdim=True))
        _close(dx.view_as(x), want, size, dtype, 100, "d" + n)
        _close(dg, (dn * x * r).sum((0, 1)), (mag * x.abs() * r).sum((0, 1)), "f32", 256, "dg" + n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + [_shape(16384, 32, 32, 128, 128, 1, "half")], ids=_name)
def test_the_gains_gradients_count_every_vector_once(shape, dtype):
    from rank_bottleneck_block_gb300.runner import QkRotary

    T, dh = shape.T, shape.dh
    shape = dataclasses.replace(shape, dtype=dtype)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)

    def signs(H):
        return (torch.randint(0, 2, (T, H * dh), generator=gen, device="cuda") * 2 - 1).to(td)

    case = {"freq": I.rotary_freq(shape.rot), "pos": torch.zeros(len(shape.sec), T, dtype=torch.int32, device="cuda"),
            "gq": torch.ones(dh, dtype=td), "gk": torch.ones(dh, dtype=td)}
    for n, H in (("q", shape.Hq), ("k", shape.Hk)):
        case[n], case[f"d{n}o"] = signs(H), signs(H)
    run = QkRotary(shape, {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in case.items()})
    r = (1.0 + shape.eps) ** -0.5
    most = T * max(shape.Hq, shape.Hk)
    m = int(256 * U * 2 * most / 0.25) + 1
    assert 256 * U * 2 * (most / m + 1) < 0.25 + 1e-4
    for phase in range(m):
        sums = []
        for n, H, dy in (("q", shape.Hq, run.dqo), ("k", shape.Hk, run.dko)):
            at = torch.zeros(T * max(H, 1), 1, dtype=td, device="cuda")
            at[phase::m] = 1
            if H:
                dy.copy_((case[f"d{n}o"].view(T * H, dh) * at).view(T, H * dh))
                sums.append((dy.float() * case[n].float()).view(T * H, dh).sum(0))  # whole numbers below 2^24
        run.backward()
        for dg, want in zip((run.dgq, run.dgk), sums):
            assert float((dg.double() - r * want.double()).abs().max()) <= 0.2501, phase
