"""Gradients of log probabilities far from zero: rows whose logits share a large offset, of the type's lowest value alone,
or whose log-sum-exp leaves fp32's range.  The oracle takes the differences to each row's largest logit (gradients do not
depend on a common offset, and fp64 would lose log V beside one of 1e30), their fp64 log-sum-exp and entropy.

Bounds, u = 2^-24: p is off by (|log p| + 8 + a) 2 u of itself, a = V / 2048 + 40 additions and rescalings of a sum; a
log-sum-exp that is taken as given adds its rounding, at most u times the limit up to which it is taken (1024 for bf16,
64 for fp32).  The entropy is within (a + 40) 8 u (1 + log V).  The result is rounded once.  The exponential of a bf16
gradient gives 0 below 2^-126, so p is off by that besides, and the result by 2^-126 times p's factor, scale (|dlogp| +
|dentropy| (|log p| + entropy)).
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
LIMIT = {"f32": 64.0, "bf16": 1024.0}
LOW = {"bf16": torch.finfo(torch.bfloat16).min, "f32": torch.finfo(torch.float32).min}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def _check_gradient(shape, case, got, rows=None):
    rows = np.arange(shape.T) if rows is None else np.asarray(rows)
    z, target = as64(case["logits"][rows]), case["target"].cpu().numpy()[rows]
    z = z - z.max(1, keepdims=True)
    w = P.fwd(z, target, shape.scale)
    de = None if case["dentropy"] is None else as64(case["dentropy"])[rows]
    b = P.bwd(z, target, w["lse"], w["entropy"], as64(case["dlogp"])[rows], de, shape.scale)
    a = shape.V / 2048 + 40
    lp = np.clip(np.abs(shape.scale * z - w["lse"][:, None]), 0, 200)
    k = ((lp + 8 + a) * 2 + LIMIT[shape.dtype]) * U
    bound = HALF[shape.dtype] * np.abs(b["dlogits"]) + 2 * k * b["mag"]
    bound += 2.0 ** -126 * shape.scale * (1 + np.abs(as64(case["dlogp"])[rows])[:, None])
    if de is not None:
        bound += 2.0 ** -126 * shape.scale * np.abs(de)[:, None] * (lp + w["entropy"][:, None])
        p = np.exp(shape.scale * z - w["lse"][:, None])
        bound += np.abs(de)[:, None] * shape.scale * p * (a + 40) * 8 * U * (1 + np.log(shape.V))
    got = as64(got)
    assert np.isfinite(got).all()
    off = np.abs(got - b["dlogits"]) / bound
    i = np.unravel_index(np.argmax(off), off.shape)
    assert off[i] <= 1.0, (i, got[i], b["dlogits"][i], off[i])


OFFSETS = [0.0, 60.0, 100.0, -100.0, 900.0, -1100.0, 3e3, 1e5, -1e5, 1e7, 3e30]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 9001, 131071])
@pytest.mark.parametrize("entropy", [True, False])
def test_rows_with_a_common_offset(V, entropy, dtype):
    """Logits a few of their type's steps around an offset; a batch of such rows beside ordinary ones."""
    shape = I.LogProbShape(T=len(OFFSETS), V=V, dtype=dtype)
    case = I.make_logprob_case(shape, seed=V, entropy=entropy)
    case["logits"] = (case["logits"].float() + torch.tensor(OFFSETS)[:, None]).to(case["logits"].dtype)
    case["target"] = torch.arange(shape.T, dtype=torch.int32) * 3
    from rank_bottleneck_block_gb300.runner import TokenLogProbs

    run = TokenLogProbs(shape, case)
    run.step()
    torch.cuda.synchronize()
    _check_gradient(shape, case, run.dlogits)
    apart = run.dlogits.clone()
    run.dlogits = run.logits  # in place
    run.backward()
    torch.cuda.synchronize()
    assert torch.equal(run.logits, apart)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.3, 7.0])
@pytest.mark.parametrize("V", [40, 9001, 50021])
def test_rows_of_the_largest_and_lowest_values(V, scale, dtype):
    """Every logit the type's lowest value, or its largest: a uniform distribution, whether or not the log-sum-exp of the
    scaled logits is a number of fp32.  A row of -inf alone has no gradient, one with a NaN has NaN."""
    shape = I.LogProbShape(T=6, V=V, scale=scale, dtype=dtype)
    case = I.make_logprob_case(shape, seed=1)
    case["target"] = torch.tensor([3, -1, V - 1, 7, 5, 6], dtype=torch.int32)
    z = case["logits"]
    z[0] = z[1] = LOW[dtype]
    z[2] = -LOW[dtype]
    z[3] = -float("inf")
    z[4, V // 2] = float("nan")
    from rank_bottleneck_block_gb300.runner import TokenLogProbs

    run = TokenLogProbs(shape, case)
    run.step()
    torch.cuda.synchronize()
    rows = [0, 1, 2, 5]
    _check_gradient(dataclasses.replace(shape, T=4), {n: t[rows] for n, t in case.items()}, run.dlogits[rows])
    assert (run.dlogits[3] == 0).all() and torch.isnan(run.dlogits[4]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_batch_with_some_rows_far_from_zero(dtype):
    """Blocks of several rounds; every third row has a large offset, and a row of 100 apart from it."""
    shape = I.LogProbShape(T=1300, V=33001, dtype=dtype)
    case = I.make_logprob_case(shape, seed=2, device="cuda")
    case["logits"][::3] += 2e3
    case["logits"][1::300] += 100
    from rank_bottleneck_block_gb300.runner import TokenLogProbs

    run = TokenLogProbs(shape, case)
    run.step()
    torch.cuda.synchronize()
    rows = [0, 1, 2, 3, 299, 300, 301, 650, 1299]
    _check_gradient(shape, case, run.dlogits[rows], rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("extra", [(3, 0), (0, 5), (1, 1), (8, 16), (1001, 2)])
def test_far_rows_that_lie_apart_and_in_a_graph(extra, dtype):
    """Rows of logits and of the gradient on any alignment, the two different; nothing beside them changes."""
    from rank_bottleneck_block_gb300.runner import GraphStep, TokenLogProbs

    T, V = 7, 20003
    shape = I.LogProbShape(T=T, V=V, dtype=dtype)
    case = I.make_logprob_case(shape, seed=3, device="cuda")
    case["logits"][::2] += 5e3
    case["logits"][3] = LOW[dtype]
    td = case["logits"].dtype
    m = torch.full((T, V + extra[0]), LOW[dtype] * -1, dtype=td, device="cuda")  # larger than any logit, if it were read
    m[:, :V] = case["logits"]
    d = torch.full((T, V + extra[1]), 7.0, dtype=td, device="cuda")
    run = TokenLogProbs(shape, case)
    run.logits, run.dlogits = m[:, :V], d[:, :V]
    run.step()
    torch.cuda.synchronize()
    _check_gradient(shape, case, run.dlogits)
    keep = d.clone()
    graph = GraphStep(run.step)
    d[:, :V] = 0
    graph()
    torch.cuda.synchronize()
    assert torch.equal(d, keep) and (d[:, V:] == 7).all() and (m[:, V:] == LOW[dtype] * -1).all()
