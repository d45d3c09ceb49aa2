"""lr_qk_fwd / lr_qk_bwd at the ends of the range of inputs that they are documented for: head vectors of a Euclidean
norm just below 1.8e19 (the sum of squares, 3.24e38, is still an fp32 number), and with eps 0 just above 4e-18.  There
the sum of squares is above 2^-116 and up to 512 squares or partial sums below 2^-126 are off by half of 2^-149 each:
2^-141 together, a 2^-25th of it, so the bounds of test_qk_gpu.py (40 and 100 roundings, of which 33 and 88 are
accounted for) hold with 34 and 92."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle.qk_oracle as Q
from oracle.compare import as64
from rank_bottleneck_block_gb300 import inputs as I

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,rot", [(8, 8), (72, 40), (128, 128), (256, 64), (336, 320), (512, 512)])
@pytest.mark.parametrize("norm,eps", [(1.79e19, 1e-6), (1.79e19, 0.0), (4.1e-18, 0.0), (4.1e-18, 1e-35)])
def test_head_vectors_of_the_largest_and_smallest_norm(dtype, dh, rot, norm, eps):
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = I.QkShape(T=9, Hq=3, Hk=2, dh=dh, rot=rot, sec=(rot // 2,), dtype=dtype, eps=eps)
    case = I.make_qk_case(shape, seed=dh)
    for n, H in (("q", 3), ("k", 2)):
        x = case[n].double().view(9, H, dh)
        x[1::3] = x[1::3].abs().clamp(0.5, 0.6)  # all channels alike
        x[2::3, :, 1:] *= 1e-4  # one channel carries the norm
        x *= 0.995 * norm / x.norm(dim=-1, keepdim=True) if norm > 1 else 1.01 * norm / x.norm(dim=-1, keepdim=True)
        case[n] = x.view(9, H * dh).to(case[n].dtype)
        size = case[n].double().view(9, H, dh).norm(dim=-1)
        assert (size < 1.8e19).all() and (size > 4e-18).all()
    run = QkRotary(shape, case)
    run.step()
    th = Q.angles(case["pos"].numpy(), case["freq"], shape.sec)
    args = (dh, rot, "half", eps)
    for n, y, dx, dg in (("q", run.qo, run.dq, run.dgq), ("k", run.ko, run.dk, run.dgk)):
        x, g, dy = as64(case[n]), as64(case["g" + n]), as64(case[f"d{n}o"])
        mag, back = Q.magnitudes(x, g, dy, *args), Q.qk_bwd(x, g, th, dy, *args)
        for got, want, m, k, t in ((y, Q.qk_fwd(x, g, th, *args), mag["y"], 40, dtype),
                                   (dx, back["dx"], mag["dx"], 100, dtype), (dg, back["dg"], mag["dg"], 256, "f32")):
            got = as64(got)
            assert np.isfinite(got).all()
            assert (np.abs(got - want) <= HALF[t] * np.abs(want) + k * U * m + 1e-37).all()
