"""A padded batch of packed sequences through the operators as they are used together.  Bounds: those of test_packed_gpu.py
and test_logprob_gpu.py, and of oracle/compare.py for the output layer."""
import numpy as np
import pytest
import torch

import oracle.compare as C
import oracle.logprob_oracle as P
import oracle.lowrank_oracle as O
import oracle.packed_oracle as A
import oracle.qk_oracle as Q
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


def test_padded_batch_through_an_output_layer_and_back():
    """Norm and rotation, packed attention, the framework's output layer, log probabilities, and back through all of them to
    every gradient, with rows before and behind the sequences: they have no target and add nothing
    to any gradient, whatever the memory of the attention's outputs held before."""
    from rank_bottleneck_block_gb300.runner import GradClip, PackedAttention, ProjGroup, QkRotary, TokenLogProbs

    lengths, front, Hq, Hk, dh, V = [61, 128, 0, 19], 3, 4, 2, 64, 1000
    used = sum(lengths)
    T = front + used + 40
    shape = I.PackedShape(T=T, nseq=len(lengths), Hq=Hq, Hk=Hk, dh=dh)
    case = I.make_packed_case(shape, lengths, seed=30, first=front, packed=True, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32)
    pos[front:front + used] = torch.cat([torch.arange(n) for n in lengths])
    qk_shape = I.QkShape(T=T, Hq=Hq, Hk=Hk, dh=dh, rot=dh, sec=(dh // 2,))
    qk = I.make_qk_case(qk_shape, seed=31)
    qk.update(q=case["q"], k=case["k"], pos=pos[None])
    target = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(5)).int()
    target[:front] = target[front + used:] = -1
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)  # new memory holds NaN
    try:
        rot = QkRotary(qk_shape, qk)
        attn = PackedAttention(shape, dict(case, q=rot.qo, k=rot.ko))
    finally:
        torch.use_deterministic_algorithms(was)
    out_shape = I.ProjShape(T=T, d_in=Hq * dh, d_out=V, r=64, group=1, norm=True)
    out_case = I.make_proj_case(out_shape, seed=32)
    head = ProjGroup(out_shape, out_case)
    lp = TokenLogProbs(I.LogProbShape(T=T, V=V, top=4), dict(logits=head.outs[0], target=target,
                                                          dlogp=torch.full((T,), -1.0 / used)))
    head.x, head.G = attn.o, [lp.dlogits]
    attn.dout, rot.dqo, rot.dko = head.dx, attn.dq, attn.dk
    grads = [rot.dgq, rot.dgk, head.dg, *head.dA, *head.dB]
    clip = GradClip(grads, 1e-3)
    rot.forward()
    attn.forward()
    head.forward()
    lp.step()
    head.backward()
    attn.backward()
    rot.backward()
    before = [as64(t) for t in grads]
    norm = clip.clip()
    _ok()
    assert all(np.isfinite(x).all() for x in before)
    for n in ("dq", "dk", "dv"):
        assert (getattr(attn, n)[:front] == 0).all() and (getattr(attn, n)[front + used:] == 0).all()
    # every step against the oracle, on what the step before has left
    rows = slice(front, front + used)
    args = (case["offs"].cpu().numpy(), Hq, Hk, dh ** -0.5)
    f = A.attn_fwd(as64(rot.qo), as64(rot.ko), as64(case["v"]), *args)
    assert (np.abs(as64(attn.o) - f["o"]) <= HALF * np.abs(f["o"]) + 1.01 * HALF * f["mag_o"])[rows].all()
    outs, saved = O.proj_group_fwd(attn.o.cpu(), out_case["g"], out_case["A"], out_case["B"], out_shape.eps)
    gr = O.proj_group_bwd(out_case["g"], out_case["A"], out_case["B"], saved, [lp.dlogits.cpu()])
    C.assert_close({"logits": C.metrics(head.outs[0], outs[0], "bf16"),
                    "dx": C.metrics(head.dx, gr["dx"], "bf16"),
                    "dg": C.metrics(before[2], gr["dg"], "bf16", scale=C.dg_scale(gr["dA"], out_case["A"], out_case["g"])),
                    "dA": C.weight(before[3], gr["dA"][0], "bf16", T),
                    "dB": C.weight(before[4], gr["dB"][0], "bf16", T)}, "bf16", "output layer")
    z = as64(head.outs[0])
    w = P.fwd(z, target.numpy(), 1.0)
    assert np.abs(as64(lp.logp) - w["logp"]).max() <= 1e-5 and (lp.logp[:front] == 0).all()
    assert (lp.top_ids.cpu().numpy() == P.top(z, 4)).all()
    d = P.bwd(z, target.numpy(), w["lse"], w["entropy"], np.full(T, -1.0 / used), None, 1.0)
    assert (np.abs(as64(lp.dlogits) - d["dlogits"]) <= HALF * np.abs(d["dlogits"]) + 1e-5 * d["mag"]).all()
    b = A.attn_bwd(as64(rot.qo), as64(rot.ko), as64(case["v"]), as64(attn.o), as64(attn.lse), as64(head.dx), *args,
                   rel_p=HALF, rel_s=1e-3, abs_d=80 * 2 * U)
    for n in ("dq", "dk", "dv"):
        assert (np.abs(as64(getattr(attn, n)) - b[n]) <= HALF * np.abs(b[n]) + 1.01 * b["err_" + n])[rows].all(), n
    th = Q.angles(pos[None].numpy(), qk["freq"], qk_shape.sec)
    for n, got in zip("qk", before):
        want = Q.qk_bwd(as64(case[n]), as64(qk["g" + n]), th, as64(getattr(attn, "d" + n)), dh, dh, "half", 1e-6)
        assert np.abs(got - want["dg"]).max() <= 1e-4 * np.abs(want["dg"]).max()
    total = np.sqrt(sum((x ** 2).sum() for x in before))
    assert abs(float(norm) - total) <= 1e-5 * total


def test_a_first_call_on_another_stream():
    """The outputs' first zeros are written by then, however much work the constructor's stream had before it."""
    from rank_bottleneck_block_gb300.runner import PackedAttention

    lengths = [200, 77]
    shape = I.PackedShape(T=300, nseq=2, Hq=4, Hk=2, dh=64)
    case = I.make_packed_case(shape, lengths, seed=1, first=3, device="cuda")
    want = PackedAttention(shape, case)
    want.step()
    m = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        m @ m
    run = PackedAttention(shape, case)
    run.step(side)
    _ok()
    for n in ("o", "lse", "dq", "dk", "dv"):
        assert torch.equal(getattr(run, n), getattr(want, n)), n
