"""lr_logprob_fwd / lr_logprob_bwd on the GPU against the fp64 oracle.

Bounds, with u = 2^-24, m the largest |scale x| of a row and V logits:
 * a difference x - max is exact or rounded once (u of it), its product with scale log2(e) twice more, the exponential
   adds 4 u (2^-22): a term is off by 4 u |d| + 4 u relative, d its difference in powers of e; terms of |d| > 30 weigh
   nothing, so every term is within 124 u, the sums too, and their additions (at most 1100 in a row: a thread's share of
   2^19 logits, 5 between lanes, 8 between warps, 64 parts) add 1180 u: s within 1310 u, and so log s;
 * logp = d - log s, entropy = log s - w/s: each within 1310 u of (1 + |d| + |log s|), the entropy's quotient (terms x d)
   of twice that; lse adds the rounding of its own size, u m and u |lse|;
 * dlogits: log p = scale x - lse, rounded to u of its operands (|scale x| + |lse|), p that relative to itself plus 4 u
   (|log p| times u in its product): within k = (m + |lse| + 2 |log p| + 8) 2 u of the terms, and rounded once.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle.logprob_oracle as P
from oracle.compare import as64
from rank_bottleneck_block_gb300 import inputs as I

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def _run(shape, case):
    from rank_bottleneck_block_gb300.runner import TokenLogProbs

    return TokenLogProbs(shape, case)


def _close(got, want, bound, what):
    got, want, bound = as64(got), np.asarray(want), np.broadcast_to(bound, np.shape(want))
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        off = np.where(same, 0.0, np.abs(got - want) / (bound + 1e-37))
    off = np.where(np.isnan(off), np.inf, off)
    i = np.unravel_index(np.argmax(off), off.shape)
    assert off[i] <= 1.0, (what, i, got[i], want[i], off[i])


def _check(shape, case, run, backward=True):
    torch.cuda.synchronize()
    z, target = as64(case["logits"]), case["target"].cpu().numpy()
    w = P.fwd(z, target, shape.scale)
    with np.errstate(invalid="ignore"):
        m = np.where(np.isfinite(z), np.abs(shape.scale * z), 0.0).max(1)
        log_s = np.log(shape.V) + 1.0
        logp = np.where(np.isfinite(w["logp"]), np.abs(w["logp"]), 0.0)
        lse = np.where(np.isfinite(w["lse"]), w["lse"], 0.0)
    k = 1310 * U
    _close(run.logp, w["logp"], k * (1 + logp + 2 * log_s), "logp")
    _close(run.entropy, w["entropy"], 4 * k * (1 + log_s), "entropy")
    _close(run.lse, w["lse"], k * (1 + log_s) + 4 * U * m + 2 * U * np.abs(lse), "lse")
    if shape.top:
        ids = P.top(z, shape.top)
        assert (run.top_ids.cpu().numpy() == ids).all()
        lp = np.stack([P.fwd(z, ids[:, i], shape.scale)["logp"] for i in range(shape.top)], 1)
        _close(run.top_logp, lp, k * (1 + np.where(np.isfinite(lp), np.abs(lp), 0.0) + 2 * log_s), "top_logp")
    if backward:
        _check_bwd(shape, case, run)


def _check_bwd(shape, case, run):
    z, target = as64(case["logits"]), case["target"].cpu().numpy()
    de = None if case["dentropy"] is None else as64(case["dentropy"])
    lse, entropy = as64(run.lse), as64(run.entropy)
    b = P.bwd(z, target, lse, entropy, as64(case["dlogp"]), de, shape.scale)
    with np.errstate(invalid="ignore"):
        lp = np.clip(np.abs(shape.scale * z - lse[:, None]), 0, 200)
        k = (np.abs(np.clip(shape.scale * z, -1e4, 1e4)) + np.abs(np.clip(lse, -1e4, 1e4))[:, None] + 2 * lp + 8) * 2 * U
    # log p + entropy cancels: its rounding is k u of |log p| + entropy, which the magnitude holds
    _close(run.dlogits, b["dlogits"], HALF[shape.dtype] * np.abs(b["dlogits"]) + 2 * k * b["mag"] + 1e-36, "dlogits")


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 7, 5), (2, 8, 8), (5, 31, 31), (4, 33, 20), (1, 255, 3), (3, 256, 32), (2, 257, 1),
          (7, 1000, 32), (3, 1023, 7), (2, 4096, 20), (1, 8192, 5), (5, 8193, 0), (2, 8191, 32), (37, 500, 0),
          (1, 32000, 20), (3, 50021, 32), (1, 131072, 20), (2, 131071, 1), (1, 262144, 32), (2, 262145, 32),
          (1, 1 << 19, 32), (1, (1 << 19) - 3, 32), (700, 300, 2), (1300, 129, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,top", SHAPES)
def test_forward_and_backward_match_the_oracle(T, V, top, dtype):
    shape = I.LogProbShape(T=T, V=V, top=top, dtype=dtype)
    case = I.make_logprob_case(shape, seed=V)
    run = _run(shape, case)
    run.step()
    _check(shape, case, run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.25, 1.7, 40.0])
def test_scale_and_a_gradient_of_logp_alone(scale, dtype):
    shape = I.LogProbShape(T=9, V=3001, top=3, scale=scale, dtype=dtype)
    case = I.make_logprob_case(shape, seed=2, entropy=False)
    run = _run(shape, case)
    run.step()
    _check(shape, case, run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [0, 1, 3, 8, 1000])
def test_rows_further_apart_on_any_alignment(extra, dtype):
    T, V = 6, 777
    shape = I.LogProbShape(T=T, V=V, top=6, dtype=dtype)
    case = I.make_logprob_case(shape, seed=3)
    td = case["logits"].dtype
    m = torch.full((T, V + extra), 100.0, dtype=td, device="cuda")  # larger than any logit, if it were read
    m[:, :V] = case["logits"]
    d = torch.full((T, V + 2 * extra + 5), 7.0, dtype=td, device="cuda")
    run = _run(shape, case)
    run.logits, run.dlogits = m[:, :V], d[:, :V]
    run.step()
    _check(shape, case, run)
    assert (m[:, V:] == 100).all() and (d[:, V:] == 7).all()
    run.dlogits = run.logits  # in place
    run.backward()
    torch.cuda.synchronize()
    assert torch.equal(m[:, :V], d[:, :V]) and (m[:, V:] == 100).all()


LOW = {"bf16": torch.finfo(torch.bfloat16).min, "f32": torch.finfo(torch.float32).min}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 9001])
def test_masked_and_broken_rows(V, dtype):
    shape = I.LogProbShape(T=9, V=V, top=4, dtype=dtype)
    case = I.make_logprob_case(shape, seed=4)
    z, inf = case["logits"], float("inf")
    case["target"] = torch.tensor([3, 3, V - 1, V - 1, 5, -1, 2, 0, V], dtype=torch.int32)
    z[0] = -inf                      # nothing left, with a target
    z[5] = -inf                      # nothing left, without one
    z[1, :V - 3] = -inf              # the target masked
    z[2, :V - 3] = -inf
    z[3, :V - 2] = LOW[dtype]        # masks of the type's lowest value
    z[4, V // 2] = float("nan")
    z[6, V // 2] = inf
    z[7] = LOW[dtype]                # nothing but those: a uniform distribution
    run = _run(shape, case)
    run.step()
    torch.cuda.synchronize()
    rows = [0, 1, 2, 3, 4, 5, 6, 8]
    part = dataclasses.replace(shape, T=len(rows))
    sub = {n: case[n][rows] for n in case}

    class Part:
        pass

    for n in ("logp", "entropy", "lse", "top_ids", "top_logp", "dlogits"):
        setattr(Part, n, getattr(run, n)[rows])
    _check(part, sub, Part, backward=False)
    d = as64(run.dlogits)
    assert (d[[0, 5]] == 0).all() and np.isnan(d[4]).all() and np.isnan(d[6]).all()
    fine = [1, 2, 3, 8]
    for n in ("logp", "entropy", "lse", "top_ids", "top_logp", "dlogits"):
        setattr(Part, n, getattr(run, n)[fine])
    _check_bwd(dataclasses.replace(shape, T=4), {n: case[n][fine] for n in case}, Part)
    assert abs(float(run.entropy[7]) - np.log(V)) < 1e-5 and abs(float(run.logp[7]) + np.log(V)) < 1e-5
    assert run.top_ids[7].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "two", "rising", "falling", "zeros", "nan", "negative"])
@pytest.mark.parametrize("V", [700, 20011, 300007])
def test_order_of_the_largest(V, kind, dtype):
    shape = I.LogProbShape(T=2, V=V, top=32, dtype=dtype)
    case = I.make_logprob_case(shape, seed=5, with_grad=False)
    z = case["logits"].float()
    if kind == "equal":
        z.fill_(1.5)
    elif kind == "two":
        z = (z > 0).float()
    elif kind in ("rising", "falling"):
        z = torch.arange(V).float().repeat(2, 1) * (1 if kind == "rising" else -1) / V * 50
    elif kind == "zeros":
        z = torch.where(z > 0, 0.0, -0.0)
    elif kind == "nan":
        z[:, V // 3::V // 9] = float("nan")
    else:
        z = -z.abs() - 1
    case["logits"] = z.to(case["logits"].dtype)
    run = _run(shape, case)
    run.forward()
    _check(shape, case, run, backward=False)


def test_rows_without_a_gradient_are_zero_whatever_they_hold():
    shape = I.LogProbShape(T=4, V=5000)
    case = I.make_logprob_case(shape, seed=6, entropy=False)
    case["target"] = torch.tensor([7, -1, 8, 5000], dtype=torch.int32)
    case["dlogp"][2] = 0.0
    case["logits"][1:] = float("nan")
    run = _run(shape, case)
    run.step()
    assert (run.dlogits[1:] == 0).all() and run.dlogits[0].abs().sum() > 0


def test_same_bits_every_time_and_in_a_graph():
    from rank_bottleneck_block_gb300.runner import GraphStep

    shape = I.LogProbShape(T=3, V=50021, top=8)
    case = I.make_logprob_case(shape, seed=7)
    run = _run(shape, case)
    run.step()
    names = ("logp", "entropy", "lse", "top_ids", "top_logp", "dlogits")
    keep = {n: getattr(run, n).clone() for n in names}
    graph = GraphStep(run.step)
    for _ in range(3):
        for n in names:
            getattr(run, n).zero_()
        graph()
        assert all(torch.equal(getattr(run, n), t) for n, t in keep.items())
    new = I.make_logprob_case(shape, seed=8)
    for n in ("logits", "target", "dlogp", "dentropy"):
        getattr(run, n).copy_(new[n])
    graph()
    _check(shape, new, run)


def test_two_calls_on_two_streams():
    runs = []
    for i, (T, V) in enumerate(((1, 131072), (300, 999))):
        shape = I.LogProbShape(T=T, V=V, top=5)
        case = I.make_logprob_case(shape, seed=40 + i)
        runs.append((shape, case, _run(shape, case), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for _, _, run, stream in runs:
            run.step(stream)
    for shape, case, run, _ in runs:
        _check(shape, case, run)


def test_rows_beyond_2_to_the_31_elements():
    T, V, ld = 2200, 300, 1 << 20
    shape = I.LogProbShape(T=T, V=V, top=2)
    case = I.make_logprob_case(shape, seed=9)
    run = _run(shape, case)
    m = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    m[:, :V] = case["logits"]
    run.logits, run.dlogits = m[:, :V], m[:, 1000:1000 + V]
    run.step()
    _check(shape, case, run)
