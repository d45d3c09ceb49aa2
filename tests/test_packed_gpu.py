"""lr_packed_attn_fwd / lr_packed_attn_bwd on the GPU against the fp64 oracle.

Bounds, with u = 2^-24, half = 2^-8 (half a step of bf16), n keys and the magnitudes of the oracle:
 * products are of bf16 numbers, exact in fp32; a sum of dh of them on the tensor cores loses at most 2 u of its terms'
   magnitude for each addition, and the scale, the difference to the maximum and the exponential some 16 u more: a score
   is off by at most (dh + 16) 2 u mag_s, its exponential by that relative to itself (doubled here), and sums over n
   keys by 2 (n + 64) u of theirs: together rel_s;
 * P is rounded to bf16 for its product, o for its output: |o - o*| <= half |o*| + (half + rel_s) mag_o;
 * lse is off by the scores' error and the sum's;
 * backward: P and dS are rounded to bf16 (half of each term), P is off by rel_s, lse is given; dout.v and D are sums of
   dh products, off by (dh + 16) 2 u of their terms' magnitude; results are rounded once, half of themselves.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle.packed_oracle as A
from oracle.compare import as64
from rank_bottleneck_block_gb300 import inputs as I

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8
ROWS = ("o", "dq", "dk", "dv")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


def _shape(lengths, Hq, Hk, dh, spare=0, **kw):
    return I.PackedShape(T=max(1, sum(lengths) + spare), nseq=len(lengths), Hq=Hq, Hk=Hk, dh=dh, **kw)


def _ok():
    from rank_bottleneck_block_gb300 import lowrank as L

    torch.cuda.synchronize()
    L.lr_check_device_error()


def _make(shape, case):
    """A runner whose outputs hold 7 everywhere."""
    from rank_bottleneck_block_gb300.runner import PackedAttention

    run = PackedAttention(shape, case)
    for n in ROWS + ("lse",):
        getattr(run, n).fill_(7.0)
    return run


def _within(got, want, bound, rows, what):
    got = as64(got)
    assert (got[~rows] == 7.0).all(), f"{what}: a row of no sequence was written"
    got, want, bound = got[rows], want[rows], bound[rows] + 1e-30
    if not got.size:
        return
    assert np.isfinite(got).all(), what
    off = np.abs(got - want) / bound
    i = np.unravel_index(np.argmax(off), off.shape)
    assert off[i] <= 1.0, (what, i, got[i], want[i], off[i])


def _check(shape, case, run, backward=True):
    _ok()
    offs = case["offs"].cpu().numpy()
    rows = np.zeros(shape.T, dtype=bool)
    rows[offs[0]:offs[-1]] = True
    scale = shape.dh ** -0.5 if shape.scale is None else shape.scale
    args = (offs, shape.Hq, shape.Hk, scale)
    x = {n: as64(case[n]) for n in "qkv"}
    f = A.attn_fwd(x["q"], x["k"], x["v"], *args)
    n = max([e - b for b, e in zip(offs, offs[1:])] + [0])
    score = (shape.dh + 16) * 2 * U * np.nanmax(np.append(f["mag_s"], 0.0))
    rel_s = 2 * score + 2 * (n + 64) * U
    _within(run.o, f["o"], HALF * np.abs(f["o"]) + (HALF + rel_s) * f["mag_o"], rows, "o")
    _within(run.lse, f["lse"], score + 2 * (n + 64) * U + 2 * U * np.abs(f["lse"]), rows, "lse")
    if not backward:
        return
    o, lse = as64(run.o), as64(run.lse)
    b = A.attn_bwd(x["q"], x["k"], x["v"], o, lse, as64(case["dout"]), *args, rel_p=HALF,
                   rel_s=rel_s + 4 * U * np.abs(lse[rows]).max(initial=0.0), abs_d=(shape.dh + 16) * 2 * U)
    for name in ROWS[1:]:
        _within(getattr(run, name), b[name], HALF * np.abs(b[name]) + (1 + HALF) * b["err_" + name], rows, name)


CASES = [  # lengths, Hq, Hk, dh, rows in front, rows behind
    ([1], 1, 1, 8, 0, 0),
    ([1], 32, 8, 128, 0, 0),
    ([17], 32, 8, 128, 0, 0),
    ([128], 2, 2, 128, 0, 0),
    ([129], 4, 1, 128, 0, 0),
    ([300, 1, 0, 77, 128, 2], 4, 2, 128, 0, 0),
    ([0, 0, 5, 0], 3, 1, 64, 0, 0),
    ([0], 2, 1, 64, 0, 3),                      # no token at all
    ([33, 250], 6, 2, 64, 5, 9),
    ([513], 1, 1, 64, 1, 0),
    ([700], 2, 1, 128, 0, 130),
    ([40, 140, 3], 5, 1, 72, 2, 1),             # five heads to a key head, an odd width
    ([90, 90], 7, 1, 40, 0, 7),
    ([200, 61], 14, 2, 96, 3, 200),
    ([65, 3, 130], 6, 2, 80, 0, 0),
    ([31] * 9, 8, 8, 16, 0, 1),
    ([1] * 40, 8, 2, 128, 0, 0),                # single tokens
    ([260], 16, 1, 56, 0, 0),
    ([45, 70], 64, 1, 128, 0, 0),
    ([9, 20], 128, 1, 24, 1, 1),                # as many heads to a key head as there can be
    ([50, 20], 100, 1, 120, 0, 0),
    ([1100], 3, 3, 104, 0, 0),
    ([257, 255], 2, 2, 88, 0, 0),
    ([64, 192, 320], 12, 4, 48, 0, 64),
    ([385], 4, 4, 32, 0, 0),
    ([1024], 8, 2, 128, 0, 0),                  # few key blocks with many queries each: dK and dV in parts
    ([600, 20, 0, 410], 4, 1, 64, 3, 5),
    ([777], 5, 1, 72, 0, 0),
    ([1500, 4], 16, 1, 40, 0, 2),
]


@pytest.mark.parametrize("lengths,Hq,Hk,dh,front,behind", CASES)
def test_forward_and_backward_match_the_oracle(lengths, Hq, Hk, dh, front, behind):
    shape = _shape(lengths, Hq, Hk, dh, front + behind)
    case = I.make_packed_case(shape, lengths, seed=dh + Hq, first=front)
    run = _make(shape, case)
    run.step()
    _check(shape, case, run)


@pytest.mark.parametrize("lengths,Hq,Hk,dh", [([70, 0, 141], 6, 2, 128), ([60, 5], 3, 3, 40), ([1], 4, 1, 64)])
def test_columns_of_wider_matrices(lengths, Hq, Hk, dh):
    """q, k, v inside one matrix, every other tensor with rows of its own distance: nothing beside them changes."""
    shape = _shape(lengths, Hq, Hk, dh, 3)
    case = I.make_packed_case(shape, lengths, seed=3, first=1, packed=True, device="cuda")
    run = _make(shape, case)
    wide = {}
    for i, n in enumerate(ROWS + ("dout",)):
        t = getattr(run, n)
        m = torch.full((shape.T, t.shape[1] + 16 + 8 * i), 7.0, dtype=t.dtype, device="cuda")
        m[:, 8:8 + t.shape[1]] = t
        wide[n] = m
        setattr(run, n, m[:, 8:8 + t.shape[1]])
    assert run.q.stride(0) == (Hq + 2 * Hk) * dh
    run.step()
    _check(shape, case, run)
    for n in ROWS:
        w = getattr(run, n).shape[1]
        assert (wide[n][:, :8] == 7).all() and (wide[n][:, 8 + w:] == 7).all(), n


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3.3e38])
def test_rows_of_no_sequence_and_other_sequences_do_not_matter(value):
    lengths, front, behind = [130, 40, 200], 7, 90
    shape = _shape(lengths, 4, 2, 128, front + behind)
    case = I.make_packed_case(shape, lengths, seed=5, first=front)
    run = _make(shape, case)
    run.step()
    _check(shape, case, run)
    keep = {n: getattr(run, n).clone() for n in ROWS + ("lse",)}
    other = slice(front + 130, front + 170)  # the middle sequence
    for n in ("q", "k", "v", "dout"):
        t = getattr(run, n)
        t[:front] = t[front + 370:] = value
        t[other] = value
    run.step()
    _ok()
    rest = torch.ones(shape.T, dtype=torch.bool, device="cuda")
    rest[other] = False
    for n, t in keep.items():
        assert torch.equal(getattr(run, n)[rest], t[rest]), n


@pytest.mark.parametrize("scale,size", [(0.05, 1.0), (3.0, 1.0), (1.0, 12.0), (0.088, 40.0)])
def test_sharp_and_flat_scores(scale, size):
    """Scores of up to some thousands: all of a row's weight on one key, and maxima that keep rising along the keys."""
    lengths = [400, 150]
    shape = _shape(lengths, 4, 2, 64, scale=scale)
    case = I.make_packed_case(shape, lengths, seed=8)
    ramp = torch.linspace(0.1, 1.0, shape.T)[:, None] * size
    case["k"] = (case["k"].float() * ramp).bfloat16()
    run = _make(shape, case)
    run.step()
    _check(shape, case, run, backward=size <= 1.0)
    if size > 1.0:
        assert all(torch.isfinite(getattr(run, n)).all() for n in ROWS)


def test_scores_far_below_and_above_zero():
    """Every score of a row at -5000 or at +5000 (bf16 channels hold these sums exactly): a softmax of equal scores."""
    shape = _shape([200], 2, 1, 64, scale=1.0)
    case = I.make_packed_case(shape, [200], seed=9)
    for sign in (-1.0, 1.0):
        case["q"], case["k"] = torch.full_like(case["q"], sign * 8.0), torch.full_like(case["k"], 10.0)
        run = _make(shape, case)
        run.step()
        _check(shape, case, run)


def test_whole_chain_matches_differentiation():
    """Gradients of the whole forward, o not given but computed: its rounding adds half of |o| to D."""
    lengths = [100, 37, 150]
    shape = _shape(lengths, 4, 2, 64)
    case = I.make_packed_case(shape, lengths, seed=11)
    run = _make(shape, case)
    run.step()
    x = {n: as64(case[n]) for n in "qkv"}
    args = (case["offs"].numpy(), 4, 2, 0.125)
    f = A.attn_fwd(x["q"], x["k"], x["v"], *args)
    rel_s = 4 * (64 + 16) * 2 * U * f["mag_s"].max() + 4 * (150 + 64) * U
    b = A.attn_bwd(x["q"], x["k"], x["v"], f["o"], f["lse"], as64(case["dout"]), *args, rel_p=HALF, rel_s=rel_s,
                   abs_d=80 * 2 * U, rel_d=0.0)
    # o is off by half |o| + half mag_o at most (the oracle's bound takes one factor of |o|: the larger magnitude)
    d = A.attn_bwd(x["q"], x["k"], x["v"], f["o"] + 2 * f["mag_o"] * np.sign(f["o"]), f["lse"], as64(case["dout"]), *args,
                   rel_d=HALF)
    rows = np.ones(shape.T, dtype=bool)
    for n in ROWS[1:]:
        bound = HALF * np.abs(b[n]) + (1 + HALF) * b["err_" + n] + (d["err_" + n] if n != "dv" else 0.0)
        _within(getattr(run, n), b[n], bound, rows, n)


def test_same_bits_every_time_and_in_a_graph():
    from rank_bottleneck_block_gb300.runner import GraphStep

    lengths = [400, 3, 129, 260]
    shape = _shape(lengths, 8, 2, 128, 20)
    case = I.make_packed_case(shape, lengths, seed=12)
    run = _make(shape, case)
    run.step()
    _ok()
    keep = {n: getattr(run, n).clone() for n in ROWS + ("lse",)}
    graph = GraphStep(run.step)
    for _ in range(3):
        for n in ROWS + ("lse",):
            getattr(run, n).fill_(7.0)
        graph()
        _ok()
        for n, t in keep.items():
            assert torch.equal(getattr(run, n), t), n
    # new offsets and values in the captured buffers
    other = [1, 700, 0, 91]
    new = I.make_packed_case(shape, other, seed=13, first=2)
    for n in ("q", "k", "v", "dout", "offs"):
        getattr(run, n).copy_(new[n])
    for n in ROWS + ("lse",):
        getattr(run, n).fill_(7.0)
    graph()
    _check(shape, new, run)


def test_many_calls_give_the_same_bits():
    """Blocks that wait for slow loads beside others that do not: every call ends, and with the same gradients."""
    shape = _shape([2048], 32, 8, 128)
    case = I.make_packed_case(shape, [2048], seed=14, device="cuda")
    run = _make(shape, case)
    run.step()
    _ok()
    keep = {n: getattr(run, n).clone() for n in ROWS + ("lse",)}
    for i in range(3000):
        run.step()
        if i % 300 == 0:
            _ok()
            assert all(torch.equal(getattr(run, n), t) for n, t in keep.items())
    _ok()
    assert all(torch.equal(getattr(run, n), t) for n, t in keep.items())


def test_other_offsets_in_a_graph_that_makes_a_list():
    """More items than SMs: the captured calls cut the sequences that they find."""
    from rank_bottleneck_block_gb300.runner import GraphStep

    lengths = [300] * 10
    shape = _shape(lengths, 8, 8, 64)
    case = I.make_packed_case(shape, lengths, seed=17)
    run = _make(shape, case)
    graph = GraphStep(run.step)
    graph()
    _check(shape, case, run)
    for other in ([3000] + [0] * 9, [0, 1, 700, 0, 0, 1500, 31, 2, 128, 129], [0] * 10):
        new = I.make_packed_case(shape, other, seed=18, first=3 if sum(other) < 2990 else 0)
        for n in ("q", "k", "v", "dout", "offs"):
            getattr(run, n).copy_(new[n])
        for n in ROWS + ("lse",):
            getattr(run, n).fill_(7.0)
        graph()
        _check(shape, new, run)


@pytest.mark.parametrize("lengths,Hq,Hk,front,back", [([40], 4, 1, 1, 2), ([1024], 8, 2, 1, 3), ([300] * 60, 8, 8, 2, 2),
                                                      ([1] * 40 + [0] * 300, 2, 1, 2, 2)])
def test_launches_are_counted(lengths, Hq, Hk, front, back):
    """The list (of a forward: where not every item has an SM) and the attention; the sums of dK and dV where their key
    blocks are cut in parts."""
    from rank_bottleneck_block_gb300 import lowrank as L

    shape = _shape(lengths, Hq, Hk, 64)
    run = _make(shape, I.make_packed_case(shape, lengths, seed=15))
    for call, want in ((run.forward, front), (run.backward, back)):
        before = L.lr_launch_count()
        call()
        assert L.lr_launch_count() - before == want
    _ok()


def test_two_graphs_with_one_workspace():
    """Captured calls whose workspaces are the same memory, replayed one after another in any order."""
    from rank_bottleneck_block_gb300.runner import GraphStep

    runs = []
    for i, lengths in enumerate(([300, 211, 0, 514], [1, 64, 900, 60])):
        shape = _shape(lengths, 4, 2, 128)
        case = I.make_packed_case(shape, lengths, seed=40 + i)
        runs.append((shape, case, _make(shape, case)))
    first, second = runs[0][2], runs[1][2]
    second.ws, second.ws_b = first.ws, first.ws_b
    graphs = [GraphStep(run.step) for _, _, run in runs]
    for order in ((0, 1), (1, 0), (0, 0, 1, 1, 0)):
        for _, _, run in runs:
            for n in ROWS + ("lse",):
                getattr(run, n).fill_(7.0)
        for i in order:
            graphs[i]()
        for shape, case, run in runs:
            _check(shape, case, run)


@pytest.mark.parametrize("Hq,Hk,dh", [(2, 1, 64), (12, 4, 128)])
def test_thousands_of_sequences(Hq, Hk, dh):
    """More sequences than the list's kernel has threads, most of them empty or of one token."""
    rng = np.random.default_rng(3)
    lengths = rng.choice([0, 0, 0, 1, 1, 2, 5], size=5000).tolist()
    lengths[4321] = 333
    shape = _shape(lengths, Hq, Hk, dh, 4)
    case = I.make_packed_case(shape, lengths, seed=16, first=1)
    run = _make(shape, case)
    run.step()
    _check(shape, case, run)


def test_two_calls_on_two_streams():
    cases = []
    for i, lengths in enumerate(([300, 211], [64] * 7)):
        shape = _shape(lengths, 4, 2, 128, 5)
        case = I.make_packed_case(shape, lengths, seed=20 + i)
        cases.append((shape, case, _make(shape, case), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for _, _, run, stream in cases:
            run.step(stream)
    for shape, case, run, _ in cases:
        _check(shape, case, run)


@pytest.mark.parametrize("offs", [[0, 50, 40, 100], [-1, 10, 20, 30], [0, 10, 20, 101], [0, 200, 20, 100],
                                  [0, -2 ** 31, 20, 100], [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], [90, 80, 70, 60]])
def test_offsets_out_of_order_write_nothing(offs):
    _refuses_offsets(I.PackedShape(T=100, nseq=3, Hq=4, Hk=2, dh=64), [20, 30, 50], offs)


@pytest.mark.parametrize("nseq,bad", [(n, i) for n in (60, 256, 257, 300) for i in (0, 1, 31, 32, 33, 255, 256, 257, 299)
                                      if i < n])
def test_one_offset_out_of_order_among_many(nseq, bad):
    """Whether a list is made or every block finds its own item."""
    lengths = [0] * nseq
    lengths[nseq // 2] = 40
    offs = np.concatenate([[0], np.cumsum(lengths)])
    offs[bad] = offs[bad + 1] + 1
    _refuses_offsets(I.PackedShape(T=50, nseq=nseq, Hq=2, Hk=1, dh=64), lengths, offs.tolist())


def _refuses_offsets(shape, lengths, offs):
    from rank_bottleneck_block_gb300 import lowrank as L

    case = I.make_packed_case(shape, lengths, seed=1)
    run = _make(shape, case)
    good = run.offs
    run.offs = torch.tensor(offs, dtype=torch.int32, device="cuda")
    for call in (run.forward, run.backward):
        call()
        torch.cuda.synchronize()
        with pytest.raises(L.LowRankError) as e:
            L.lr_check_device_error()
        assert e.value.status == 2 and "offsets" in str(e.value)
        assert all((getattr(run, n) == 7).all() for n in ROWS + ("lse",))
    run.offs = good  # and the next call is none the worse
    run.step()
    _check(shape, case, run)


def test_rows_beyond_2_to_the_31_elements():
    """A packed matrix of 2.3e9 elements: offsets within it do not fit 32 bits."""
    T, Hq, Hk, dh = 4500, 2, 1, 64
    lengths = [30, 4000, 300]
    shape = _shape(lengths, Hq, Hk, dh, T - sum(lengths))
    case = I.make_packed_case(shape, lengths, seed=4, first=100)
    run = _make(shape, case)
    m = torch.zeros(T, 512 * 1000, dtype=torch.bfloat16, device="cuda")
    at = 0
    for n in ("q", "k", "v", "dout") + ROWS:
        t = getattr(run, n)
        m[:, at:at + t.shape[1]] = t
        setattr(run, n, m[:, at:at + t.shape[1]])
        at += t.shape[1]
    run.step()
    _check(shape, case, run)


def test_against_the_attention_of_equal_sequences():
    """b sequences of one length, a key head to each query head: what lr_attn_* computes, within both roundings."""
    from rank_bottleneck_block_gb300.runner import Attention

    b, s, H, dh = 2, 512, 2, 128
    shape = _shape([s] * b, H, H, dh)
    case = I.make_packed_case(shape, [s] * b, seed=6)
    run = _make(shape, case)
    run.step()
    ref = Attention(b, s, H, dh, case["q"], case["k"], case["v"])
    ref.forward()
    ref.backward(case["dout"].cuda())
    _ok()
    for n in ROWS:
        got, want = as64(getattr(run, n)), as64(getattr(ref, n))
        # each is within half a step and its terms' roundings of the same value; 0.02 is the suite's bf16 tolerance
        assert np.abs(got - want).max() <= 2e-2 * np.abs(want).max(), n


def test_results_are_those_of_the_assigned_tensors():
    lengths = [90, 41]
    shape = _shape(lengths, 4, 2, 64)
    first, second = (I.make_packed_case(shape, lengths, seed=s) for s in (1, 2))
    run = _make(shape, first)
    run.step()
    case = dict(first)
    for n in ("q", "k", "v", "dout"):
        case[n] = second[n]
        setattr(run, n, second[n].cuda())
        run.step()
        _check(shape, case, run)


def test_prompt_to_loss_and_back():
    """The operators as they are used together: norm and rotation of packed, shared heads, attention over the packed
    sequences, log probabilities of the next tokens, their gradient back to q, k, v, and clipping."""
    import oracle.logprob_oracle as P
    import oracle.qk_oracle as Q
    from rank_bottleneck_block_gb300.runner import GradClip, PackedAttention, QkRotary, TokenLogProbs

    lengths, Hq, Hk, dh = [61, 128, 19], 4, 2, 64
    T = sum(lengths)
    shape = _shape(lengths, Hq, Hk, dh)
    case = I.make_packed_case(shape, lengths, seed=30, packed=True, device="cuda")
    pos = torch.cat([torch.arange(n) for n in lengths]).int()[None]
    qk_shape = I.QkShape(T=T, Hq=Hq, Hk=Hk, dh=dh, rot=dh, sec=(dh // 2,))
    qk = I.make_qk_case(qk_shape, seed=31)
    qk.update(q=case["q"], k=case["k"], pos=pos)
    rot = QkRotary(qk_shape, qk)
    attn = PackedAttention(shape, dict(case, q=rot.qo, k=rot.ko))
    V = Hq * dh  # the attention's output stands for the logits
    lp = TokenLogProbs(I.LogProbShape(T=T, V=V, top=4), dict(logits=attn.o, target=torch.randint(0, V, (T,)).int(),
                                                          dlogp=torch.full((T,), -1.0 / T)))
    attn.dout, rot.dqo, rot.dko = lp.dlogits, attn.dq, attn.dk
    clip = GradClip([rot.dgq, rot.dgk], 1e-3)
    rot.forward()
    attn.forward()
    lp.forward()
    lp.backward()
    attn.backward()
    rot.backward()
    before = {n: as64(getattr(rot, n)) for n in ("dgq", "dgk")}
    norm = clip.clip()
    _ok()
    # every step against the oracle, on what the step before has left
    th = Q.angles(pos.numpy(), qk["freq"], qk_shape.sec)
    for n in "qk":
        want = Q.qk_fwd(as64(case[n]), as64(qk["g" + n]), th, dh, dh, "half", 1e-6)
        assert np.abs(as64(getattr(rot, n + "o")) - want).max() <= 2 * HALF * np.abs(want).max()
    args = (case["offs"].cpu().numpy(), Hq, Hk, dh ** -0.5)
    f = A.attn_fwd(as64(rot.qo), as64(rot.ko), as64(case["v"]), *args)
    assert (np.abs(as64(attn.o) - f["o"]) <= HALF * np.abs(f["o"]) + 1.01 * HALF * f["mag_o"]).all()
    w = P.fwd(as64(attn.o), lp.target.cpu().numpy(), 1.0)
    assert np.abs(as64(lp.logp) - w["logp"]).max() <= 1e-5
    assert (lp.top_ids.cpu().numpy() == P.top(as64(attn.o), 4)).all()
    d = P.bwd(as64(attn.o), lp.target.cpu().numpy(), w["lse"], w["entropy"], np.full(T, -1.0 / T), None, 1.0)
    assert (np.abs(as64(lp.dlogits) - d["dlogits"]) <= HALF * np.abs(d["dlogits"]) + 1e-5 * d["mag"]).all()
    b = A.attn_bwd(as64(rot.qo), as64(rot.ko), as64(case["v"]), as64(attn.o), as64(attn.lse), as64(lp.dlogits), *args,
                   rel_p=HALF, rel_s=1e-3, abs_d=80 * 2 * U)
    for n in ("dq", "dk", "dv"):
        assert (np.abs(as64(getattr(attn, n)) - b[n]) <= HALF * np.abs(b[n]) + 1.01 * b["err_" + n]).all(), n
    for n in "qk":
        want = Q.qk_bwd(as64(case[n]), as64(qk["g" + n]), th, as64(getattr(attn, "d" + n)), dh, dh, "half", 1e-6)
        assert np.abs(as64(getattr(rot, "d" + n)) - want["dx"]).max() <= 2 * HALF * np.abs(want["dx"]).max()
        assert np.abs(before["dg" + n] - want["dg"]).max() <= 1e-4 * np.abs(want["dg"]).max()
    total = np.sqrt(sum((x ** 2).sum() for x in before.values()))
    assert abs(float(norm) - total) <= 1e-5 * total
