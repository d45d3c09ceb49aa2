"""The transformer block with norm and rotation of its queries and keys, and its training step with clipping: parity
with the fp64 oracle (the bounds of oracle.compare, as for the block without them), bitwise agreement where nothing is
turned, graph capture."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle.compare as C
import oracle.qk_oracle as Q
from rank_bottleneck_block_gb300 import inputs as I

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def _case(shape, qk, seed, norm=True, pos=True):
    case = I.make_block_case(shape, seed)
    more = I.make_qk_case(qk, seed, norm=norm, with_grad=False)
    case.update({k: more[k] for k in ("gq", "gk", "pos", "freq")})
    if not pos:
        case["pos"] = None
    return case


def _qk(shape, rot, sec, layout="half"):
    return I.QkShape(T=shape.T, Hq=shape.H, Hk=shape.H, dh=shape.dh, rot=rot, sec=sec, layout=layout)


@pytest.mark.parametrize("dims,rot,sec,layout,norm,pos", [
    ((2, 256, 2, 128, 344, 32, 48), 128, (64,), "half", True, False),
    ((1, 512, 3, 128, 264, 24, 40), 128, (16, 24, 24), "half", True, True),
    ((1, 256, 2, 256, 264, 32, 40), 96, (48,), "pairs", True, False),
    ((2, 256, 2, 128, 344, 32, 48), 64, (16, 16), "half", False, True),
])
def test_block_matches_oracle(dims, rot, sec, layout, norm, pos):
    from rank_bottleneck_block_gb300 import lowrank as L
    from rank_bottleneck_block_gb300.runner import TransformerBlock

    shape = I.BlockShape(*dims)
    qk = _qk(shape, rot, sec, layout)
    case = _case(shape, qk, sum(dims), norm, pos)
    blk = TransformerBlock(shape, case, qk=qk)
    blk.step()
    torch.cuda.synchronize()
    L.lr_check_device_error()
    W = {k: v.double().numpy() for k, v in case.items() if k[:2] in ("A_", "B_", "g_")}
    where = case["pos"].numpy() if pos else np.tile(np.arange(shape.T) % shape.s, (len(sec), 1))
    turn = dict(theta=Q.angles(where, case["freq"], sec), rot=rot, layout=layout,
                **{g: None if case[g] is None else case[g].double().numpy() for g in ("gq", "gk")})
    args = (shape.b, shape.s, shape.H, shape.dh, shape.eps)
    out, saved = Q.block_fwd(case["x"].double().numpy(), W, turn, *args)
    gr = Q.block_bwd(W, saved, turn, case["G"].double().numpy(), *args)
    errs = {"out": C.metrics(blk.out, out), "dx": C.metrics(blk.dx, gr["dx"]),
            "dg_attn": C.metrics(blk.dg_attn, gr["dg_attn"]), "dg_mlp": C.metrics(blk.dg_mlp, gr["dg_mlp"])}
    for n in ("dgq", "dgk"):
        assert (getattr(blk, n) is None) == (not norm)
        if norm:
            errs[n] = C.metrics(getattr(blk, n), gr[n])
    for n in ("q", "k", "v", "o", "gate", "up", "down"):
        for m in ("A", "B"):
            errs[f"d{m}_{n}"] = C.weight(blk.grads[f"d{m}_{n}"], gr[f"d{m}_{n}"])
    C.assert_close(errs, "bf16", f"block {dims}")


def test_without_gains_and_turns_it_is_the_plain_block():
    """rot 0 and no gains: the copies of q and k equal q and k, so every result is the plain block's bit for bit."""
    from rank_bottleneck_block_gb300.runner import TransformerBlock

    shape = I.BlockShape(2, 256, 2, 128, 344, 32, 48)
    case = I.make_block_case(shape, 4)
    plain = TransformerBlock(shape, case)
    plain.step()
    same = TransformerBlock(shape, dict(case, freq=[]), qk=_qk(shape, 0, (0,)))
    same.step()
    assert torch.equal(plain.out, same.out) and torch.equal(plain.dx, same.dx)
    assert all(torch.equal(plain.grads[k], same.grads[k]) for k in plain.grads)


def test_a_training_step_with_clipping_repeats_and_replays():
    """Step and clipping, three times in a row and as a captured graph: the same bits each time."""
    from rank_bottleneck_block_gb300 import lowrank as L
    from rank_bottleneck_block_gb300.runner import GraphStep, TransformerBlock

    shape = I.BlockShape(2, 256, 2, 128, 344, 32, 48)
    qk = _qk(shape, 128, (24, 20, 20))
    blk = TransformerBlock(shape, _case(shape, qk, 6), qk=qk)
    blk.step()
    before = [t.clone() for t in blk.grad_tensors()]
    assert len(before) == 4 + 14
    norm = float(blk.clip_grads(1.0))
    want = float(torch.stack([t.double().square().sum() for t in before]).sum().sqrt())
    assert norm == pytest.approx(want, rel=1e-5) and norm > 1.0
    ref = [blk.out.clone(), blk.dx.clone()] + [t.clone() for t in blk.grad_tensors()]
    total = float(torch.stack([t.double().square().sum() for t in blk.grad_tensors()]).sum().sqrt())
    assert total == pytest.approx(1.0, rel=1e-5)

    def step():
        blk.step()
        blk.clip_grads(1.0)

    for _ in range(3):
        step()
    graph = GraphStep(step)
    for run in (lambda: None, graph, graph):
        run()
        torch.cuda.synchronize()
        L.lr_check_device_error()
        now = [blk.out, blk.dx] + blk.grad_tensors()
        assert all(torch.equal(a, b) for a, b in zip(ref, now))
        for t in now:
            t.zero_()


def test_the_pieces_one_after_another_are_the_block():
    """Projection group, norm and rotation, attention through their own entry points give the block's attention output."""
    from rank_bottleneck_block_gb300 import lowrank as L
    from rank_bottleneck_block_gb300.runner import Attention, QkRotary, TransformerBlock

    shape = I.BlockShape(2, 256, 2, 128, 344, 32, 48)
    qk = _qk(shape, 128, (64,))
    case = _case(shape, qk, 7, pos=False)
    blk = TransformerBlock(shape, case, qk=qk)
    blk.forward()
    T, d = shape.T, shape.d
    t = blk.t
    outs = [torch.empty(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    saved = torch.empty(L.lr_proj_saved_bytes(L.LR_BF16, T, d, d, shape.ra, 3, 1), dtype=torch.uint8, device="cuda")
    ws = torch.empty(L.lr_proj_fwd_workspace_bytes(L.LR_BF16, T, d, d, shape.ra, 3, 1), dtype=torch.uint8, device="cuda")
    L.lr_proj_fwd(L.LR_BF16, T, d, d, shape.ra, [L.pair(t[f"A_{n}"], t[f"B_{n}"]) for n in "qkv"], t["g_attn"], shape.eps,
                  t["x"], outs, saved, ws)
    rotary = QkRotary(dataclasses.replace(qk, seq=shape.s),
                      dict(q=outs[0], k=outs[1], gq=case["gq"], gk=case["gk"], pos=None, freq=case["freq"]))
    qo, ko = rotary.forward()
    att = Attention(shape.b, shape.s, shape.H, shape.dh, qo, ko, outs[2])
    att.forward()
    # o, the o-projection with its residual and the MLP, as the block runs them
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    so = torch.empty(L.lr_proj_saved_bytes(L.LR_BF16, T, d, d, shape.ra, 1, 0), dtype=torch.uint8, device="cuda")
    wo = torch.empty(L.lr_proj_fwd_workspace_bytes(L.LR_BF16, T, d, d, shape.ra, 1, 0), dtype=torch.uint8, device="cuda")
    L.lr_proj_fwd(L.LR_BF16, T, d, d, shape.ra, [L.pair(t["A_o"], t["B_o"])], None, shape.eps, att.o, [y], so, wo)
    x1 = (t["x"].float() + y.float())
    ms = torch.empty(L.lr_mlp_saved_bytes(L.LR_BF16, 1, T, d, shape.f, shape.rm), dtype=torch.uint8, device="cuda")
    mw = torch.empty(L.lr_mlp_fwd_workspace_bytes(L.LR_BF16, 1, T, d, shape.f, shape.rm), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(y)
    L.lr_mlp_fwd(L.LR_BF16, 1, T, d, shape.f, shape.rm, shape.eps, x1.bfloat16(), t["g_mlp"],
                 *(L.pair(t[f"A_{n}"], t[f"B_{n}"]) for n in ("gate", "up", "down")), out, ms, mw)
    # y is rounded to bf16 before the residual here (2^-8 of |y|, which is below the output's scale), and the
    # block adds it to x in fp32: the outputs agree to a few bf16 roundings
    assert C.metrics(out, blk.out.float().cpu().numpy())["maxrel"] < 2e-2


def test_the_readme_example_runs():
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    code = re.search(r"and clipping:\n\n((?:    .*\n|\n)+)", text).group(1)
    names = {}
    exec("\n".join(line[4:] for line in code.splitlines()), names)
    assert torch.isfinite(names["norm"]).all() and torch.isfinite(names["blk"].dx.float()).all()
