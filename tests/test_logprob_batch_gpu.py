"""Log probabilities where the kernels do the most work a block: rows kept in one block over many rounds of its loop, rows
cut over many blocks, blocks of the gradient that take several rounds; and no logit lost or taken twice anywhere.

Bounds, u = 2^-24: a term 2^d is within (3 |d| + 4) u of itself, |d| <= 30 for any that weighs (94 u, as for sums of them); a
thread adds r groups of 8 logits (5 additions in one, and one for it), rescales each round (8 u) and joins 13 times (8 u):
s is within rel_s = (94 + 6 r + 2 r + 104) u, r = V / 2048 + 8 at most (a cut row has fewer).  lse is off by that, the
logarithm (4 u of itself) and its own rounding; logp and entropy as the terms that they are sums of.
"""
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


def _runner(shape, case):
    from rank_bottleneck_block_gb300.runner import TokenLogProbs

    return TokenLogProbs(shape, case)


def _within(got, want, bound, what):
    off = np.abs(as64(got) - want) / bound
    i = np.unravel_index(np.argmax(off), off.shape)
    assert off[i] <= 1.0, (what, i, as64(got)[i], want[i], off[i])


def _check(shape, case, run, rows):
    torch.cuda.synchronize()
    V, scale = shape.V, shape.scale
    z, target = as64(case["logits"][rows]), case["target"].cpu().numpy()[rows]
    w = P.fwd(z, target, scale)
    rel_s = (200 + 8 * (V / 2048 + 8)) * U
    log_s = w["lse"] - scale * z.max(1)
    _within(run.lse[rows], w["lse"], rel_s + 4 * U * (log_s + np.abs(w["lse"])), "lse")
    _within(run.logp[rows], w["logp"], rel_s + 4 * U * (log_s + 2 * np.abs(w["logp"]) + 1), "logp")
    # entropy = log s - w / s: w is a sum of terms x d, within rel_s of their magnitude log s + entropy at most
    _within(run.entropy[rows], w["entropy"], 2 * rel_s * (1 + 2 * log_s + w["entropy"]), "entropy")
    if shape.top:
        ids = P.top(z, shape.top)
        assert (run.top_ids[rows].cpu().numpy() == ids).all()
        lp = np.stack([P.fwd(z, ids[:, i], scale)["logp"] for i in range(shape.top)], 1)
        _within(run.top_logp[rows], lp, rel_s + 4 * U * (log_s[:, None] + 2 * np.abs(lp) + 1), "top_logp")
    if run.dlogits is None:
        return
    de = None if case["dentropy"] is None else as64(case["dentropy"][rows])
    b = P.bwd(z, target, w["lse"], w["entropy"], as64(case["dlogp"][rows]), de, scale)
    lp = np.clip(np.abs(scale * z - w["lse"][:, None]), 0, 200)
    k = rel_s + 2 * U * (lp + 8 + 4 * np.abs(w["lse"][:, None]))
    bound = HALF[shape.dtype] * np.abs(b["dlogits"]) + 2 * k * b["mag"] + 1e-36
    if de is not None:  # the entropy's own error
        p = np.exp(scale * z - w["lse"][:, None])
        bound += np.abs(de)[:, None] * scale * p * 2 * rel_s * (1 + 2 * log_s + w["entropy"])[:, None]
    _within(run.dlogits[rows], b["dlogits"], bound, "dlogits")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,top,extra,rising", [
    (1300, 20011, 0, 0, False), (1300, 20011, 5, 3, True), (2500, 33001, 0, 7, True), (2500, 33001, 3, 0, False),
    (1217, 131072, 0, 0, True), (1216, 131071, 20, 1, False), (400, 70001, 0, 2, True), (40, 262147, 7, 0, True),
    (5000, 9000, 0, 0, True),
])
def test_training_batches(T, V, top, extra, rising, dtype):
    """Rising: the running maximum grows from round to round of every second row, and falls in the others."""
    shape = I.LogProbShape(T=T, V=V, top=top, dtype=dtype)
    case = I.make_logprob_case(shape, seed=T + V, device="cuda")
    if rising:
        ramp = torch.linspace(0, 20, V, device="cuda")
        sign = torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.0)
        case["logits"] = (case["logits"].float() + sign[:, None] * ramp).to(case["logits"].dtype)
    if extra:
        m = torch.empty(T, V + extra, dtype=case["logits"].dtype, device="cuda")
        m[:, :V] = case["logits"]
        case["logits"] = m[:, :V]
    run = _runner(shape, case)
    run.step()
    rows = np.unique(np.r_[0, 1, 2, 3, T // 2, T - 2, T - 1, np.random.default_rng(V).integers(0, T, 12)])
    _check(shape, case, run, torch.from_numpy(rows))
    # and every row, by a plain softmax in fp64 on the device
    for r in range(0, T, 200):
        z = case["logits"][r:r + 200].double()
        lse = torch.logsumexp(z, -1)
        bound = (200 + 8 * (V / 2048 + 8)) * U + 8 * U * (lse.abs() + np.log(V))
        assert ((run.lse[r:r + 200] - lse).abs() <= bound).all()




@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,extra", [(1, 5000, 0), (2, 50021, 0), (3, 131071, 1), (1, 262145, 0), (4, (1 << 19) - 3, 0),
                                       (1, 1 << 19, 0), (64, 32768, 5), (1280, 20011, 3), (1280, 8193, 0)])
def test_every_logit_counts_once(T, V, extra, dtype):
    """lse and entropy of a row are the logarithm of the number of its finite logits, and each of them has its gradient."""
    shape = I.LogProbShape(T=T, V=V, dtype=dtype)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    places = torch.arange(V, device="cuda") % 64
    m = torch.empty(T, V + extra, dtype=td, device="cuda")
    case = {"logits": m[:, :V], "target": torch.full((T,), -1, dtype=torch.int32, device="cuda"),
            "dlogp": torch.ones(T, device="cuda"), "dentropy": None}
    run = _runner(shape, case)
    for first in range(0, 64, T):
        which = (first + torch.arange(T, device="cuda")) % 64
        here = places[None, :] == which[:, None]
        m.fill_(9.0)  # larger than any logit, if it were read beside a row
        case["logits"].copy_(torch.where(here, 0.0, -float("inf")))
        target = which.int()  # a place of the row
        run.target.copy_(target)
        run.step()
        n = here.sum(1).double()
        bound = 4 * U * (n.log() + 1)  # the sum of n ones is exact
        assert ((run.lse - n.log()).abs() <= bound).all()
        assert ((run.entropy - n.log()).abs() <= bound).all()
        assert ((run.logp + n.log()).abs() <= bound).all()
        want = torch.where(here, (-1 / n)[:, None], 0.0).double()
        want[torch.arange(T, device="cuda"), which] += 1.0
        off = (run.dlogits.double() - want).abs()
        assert (off <= HALF[dtype] * want.abs() + (16 * U * (1 + n.log()) / n)[:, None] * here).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 131072), (3, 50021), (1, (1 << 19) - 3), (1300, 33001)])
def test_equal_logits(T, V, dtype):
    shape = I.LogProbShape(T=T, V=V, top=32, dtype=dtype)
    case = I.make_logprob_case(shape, seed=1, device="cuda")
    case["logits"].fill_(0.5)
    run = _runner(shape, case)
    run.step()
    bound = 4 * U * (np.log(V) + 1)
    assert ((run.lse.double() - 0.5 - np.log(V)).abs() <= bound).all()
    assert ((run.entropy.double() - np.log(V)).abs() <= bound).all()
    assert (run.top_ids == torch.arange(32, device="cuda")).all()
    assert ((run.top_logp.double() + np.log(V)).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,extra", [(2, 131071, 1), (1300, 33001, 2)])
def test_large_logits_at_the_borders(T, V, extra, dtype):
    """Two large logits on both sides of a border (of 8, 256, 1024, 2048, 4096, 8192 logits, counted from the row's start and
    from the aligned place before it) and at a row's ends: found, weighed and ranked."""
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    shape = I.LogProbShape(T=T, V=V, top=4, dtype=dtype)
    m = torch.full((T, V + extra), 50.0, dtype=td, device="cuda")
    z = m[:, :V]
    z.fill_(-20.0)
    step = 16 // z.element_size()
    borders = [b + s for b in (8, 256, 1024, 2048, 4096, 8192, 16384, 32768) for s in range(1 - step, 1) if b + s > 0]
    case = {"logits": z, "target": torch.zeros(T, dtype=torch.int32, device="cuda")}
    run = _runner(shape, case)
    for lo in range(0, len(borders), T):
        some = [borders[(lo + t) % len(borders)] for t in range(T)]
        at = torch.tensor(some, device="cuda")
        rows = torch.arange(T, device="cuda")
        z.fill_(-20.0)
        z[rows, at - 1], z[rows, at] = 4.0, 5.0
        z[:, 0], z[:, V - 1] = 3.0, 2.0
        run.forward()
        first = (at == 1)  # the place before the border is the row's first
        x = z.double()
        lse = torch.logsumexp(x, -1)
        assert ((run.lse - lse).abs() <= 300 * U).all()
        ids = run.top_ids.long()
        assert (ids[:, 0] == at).all() and torch.equal(x.gather(1, ids), x.topk(4, -1).values)
        assert (ids[~first][:, 1] == at[~first] - 1).all() and (ids[~first][:, 2] == 0).all()
        assert (ids[~first][:, 3] == V - 1).all()
