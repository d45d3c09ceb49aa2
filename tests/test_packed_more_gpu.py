"""Packed attention on long sequences (a sample of rows and keys against fp64) and the gradients of large scores.  Bounds:
those of test_packed_gpu.py."""
import numpy as np
import pytest
import torch

import oracle.packed_oracle as A
from oracle.compare import as64
from rank_bottleneck_block_gb300 import inputs as I

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def _ok():
    from rank_bottleneck_block_gb300 import lowrank as L

    torch.cuda.synchronize()
    L.lr_check_device_error()


def _runner(shape, case):
    from rank_bottleneck_block_gb300.runner import PackedAttention

    return PackedAttention(shape, case)


def _within(got, want, bound, what):
    off = np.abs(got - want) / (bound + 1e-30)
    i = np.unravel_index(np.argmax(off), off.shape)
    assert np.isfinite(got).all() and off[i] <= 1.0, (what, i, got[i], want[i], off[i])


@pytest.mark.parametrize("scale,size", [(0.05, 1.0), (3.0, 1.0), (1.0, 12.0), (0.088, 40.0)])
def test_gradients_of_sharp_and_flat_scores(scale, size):
    """Scores of up to some thousands, maxima that keep rising along the keys."""
    lengths = [400, 150]
    shape = I.PackedShape(T=550, nseq=2, Hq=4, Hk=2, dh=64, scale=scale)
    case = I.make_packed_case(shape, lengths, seed=8)
    case["k"] = (case["k"].float() * torch.linspace(0.1, 1.0, shape.T)[:, None] * size).bfloat16()
    run = _runner(shape, case)
    run.step()
    _ok()
    x = {n: as64(case[n]) for n in ("q", "k", "v", "dout")}
    args = (case["offs"].numpy(), 4, 2, scale)
    f = A.attn_fwd(x["q"], x["k"], x["v"], *args)
    rel_s = 2 * (64 + 16) * 2 * U * f["mag_s"].max() + 2 * (400 + 64) * U
    o, lse = as64(run.o), as64(run.lse)
    b = A.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["dout"], *args, rel_p=HALF,
                   rel_s=rel_s + 4 * U * np.abs(lse).max(), abs_d=(64 + 16) * 2 * U)
    for n in ("dq", "dk", "dv"):
        _within(as64(getattr(run, n)), b[n], HALF * np.abs(b[n]) + (1 + HALF) * b["err_" + n], n)


@pytest.mark.parametrize("ramp", [None, "rising", "falling"])
@pytest.mark.parametrize("lengths,Hq,Hk,dh", [([16384], 8, 2, 128), ([16384], 12, 12, 128), ([9001, 7003], 20, 10, 64),
                                              ([12345, 1, 300], 6, 3, 96)])
def test_samples_of_long_sequences(lengths, Hq, Hk, dh, ramp):
    """Maxima that rise or fall over more than a hundred key blocks, more key heads than one group of them holds."""
    T = sum(lengths)
    shape = I.PackedShape(T=T, nseq=len(lengths), Hq=Hq, Hk=Hk, dh=dh)
    case = I.make_packed_case(shape, lengths, seed=dh, device="cuda")
    if ramp:
        size = torch.cat([torch.linspace(0.1, 8.0, n, device="cuda") for n in lengths])[:, None]
        case["k"] = (case["k"].float() * (size if ramp == "rising" else size.flip(0))).bfloat16()
    run = _runner(shape, case)
    run.step()
    _ok()
    G, scale = Hq // Hk, dh ** -0.5
    x = {n: as64(t).reshape(T, -1, dh) for n, t in [(n, case[n]) for n in ("q", "k", "v", "dout")] +
         [(n, getattr(run, n)) for n in ("o", "dq", "dk", "dv")]}
    lse, offs = as64(run.lse), case["offs"].cpu().numpy()
    rng = np.random.default_rng(dh)
    for b, e in zip(offs, offs[1:]):
        n = e - b
        rows = np.unique(np.clip(np.r_[0, 1, 127, 128, 129, n // 2, n - 130, n - 2, n - 1, rng.integers(0, n, 5)], 0, n - 1)) + b
        for h in {0, Hq - 1, int(rng.integers(0, Hq))}:
            q, k, v, o, g = x["q"][b:e, h], x["k"][b:e, h // G], x["v"][b:e, h // G], x["o"][b:e, h], x["dout"][b:e, h]
            for t in rows - b:
                S = scale * k[:t + 1] @ q[t]
                mag = scale * (np.abs(k[:t + 1]) @ np.abs(q[t])).max()
                err = (dh + 16) * 2 * U * mag
                rel = 2 * err + 2 * (t + 1 + 64) * U
                m = S.max()
                p = np.exp(S - m)
                total = p.sum()
                _within(lse[b + t:b + t + 1, h], np.array([m + np.log(total)]),
                        err + 2 * (t + 65) * U + 2 * U * abs(m + np.log(total)), ("lse", t, h))
                p /= total
                _within(o[t], p @ v[:t + 1], HALF * np.abs(p @ v[:t + 1]) + (HALF + rel) * (p @ np.abs(v[:t + 1])), ("o", t, h))
                p = np.exp(S - lse[b + t, h])
                rel += 4 * U * abs(lse[b + t, h])
                terms = np.abs(v[:t + 1]) @ np.abs(g[t]) + (np.abs(g[t]) * np.abs(o[t])).sum()
                dS = scale * p * (v[:t + 1] @ g[t] - g[t] @ o[t])
                err_S = (HALF + rel) * np.abs(dS) + scale * p * (dh + 16) * 2 * U * terms
                want = dS @ k[:t + 1]
                _within(x["dq"][b + t, h], want, HALF * np.abs(want) + (1 + HALF) * (err_S @ np.abs(k[:t + 1])), ("dq", t, h))
        for h in {0, Hk - 1}:
            k, v = x["k"][b:e, h], x["v"][b:e, h]
            for j in rows - b:
                dk, dv, err_k, err_v = (np.zeros(dh) for _ in range(4))
                for hq in range(h * G, h * G + G):
                    q, o, g = x["q"][b + j:e, hq], x["o"][b + j:e, hq], x["dout"][b + j:e, hq]
                    S, mag = scale * q @ k[j], scale * np.abs(q) @ np.abs(k[j])
                    p = np.exp(S - lse[b + j:e, hq])
                    rel = 4 * (dh + 16) * U * mag + 2 * (n + 64) * U + 4 * U * np.abs(lse[b + j:e, hq])
                    terms = np.abs(g) @ np.abs(v[j]) + (np.abs(g) * np.abs(o)).sum(1)
                    dS = scale * p * (g @ v[j] - (g * o).sum(1))
                    dk += dS @ q
                    dv += p @ g
                    err_k += ((HALF + rel) * np.abs(dS) + scale * p * (dh + 16) * 2 * U * terms) @ np.abs(q)
                    err_v += ((HALF + rel) * p) @ np.abs(g)
                # the products add (n - j) G terms in fp32
                adds = 2 * (n - j) * G * U
                _within(x["dk"][b + j, h], dk, HALF * np.abs(dk) + (1 + HALF + adds / HALF) * err_k, ("dk", j, h))
                _within(x["dv"][b + j, h], dv, HALF * np.abs(dv) + (1 + HALF + adds / HALF) * err_v, ("dv", j, h))
