"""lr_qk_fwd / lr_qk_bwd on the GPU against the fp64 oracle.

Bounds, with u = 2^-24 and M the magnitude of the terms of a channel (oracle.magnitudes): the output is rounded
once, half a step of its type (eps/2 relative: fp32 u, bf16 2^-8 at most); before that
 * the mean square of dh <= 512 values is a sum of at most 16 terms per lane and 5 between lanes, all positive:
   21 u, half of it in r, and 4 u more for the division, eps, the root and the reciprocal: r within 15 u;
 * n = x r g adds 2 u; cos and sin are off by 14 u at most (bf16: the hardware functions' 2^-21.19, and the angle,
   rounded twice to 24 bits at up to pi, 2 * 2^-22.35); the turn itself adds 2 u: 33 u of |n_i| + |n_j| in all,
   bounded by 40 u here;
 * backward: dn within 16 u of its pair, w = dn g 17 u, mean(w x) adds 21 u, r^2 30 u, and the last products and
   the difference 4 u: 88 u of the terms, bounded by 100 u;
 * dg: each term within 35 u, and a sum over N terms cut over lanes, warps and blocks, at most 200 additions in
   a row: bounded by 256 u of the sum of magnitudes.
"""
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


def _shape(T, Hq, Hk, dh, rot=None, axes=1, **kw):
    rot = dh if rot is None else rot
    each = rot // 2 // axes
    return I.QkShape(T=T, Hq=Hq, Hk=Hk, dh=dh, rot=rot, sec=(rot // 2 - each * (axes - 1),) + (each,) * (axes - 1), **kw)


def _close(got, want, mag, dtype, k, what):
    got, bound = as64(got), HALF[dtype] * np.abs(want) + k * U * mag + 1e-37
    assert got.shape == want.shape, what
    off = np.abs(got - want) / bound
    i = np.unravel_index(np.argmax(off), off.shape)
    assert np.isfinite(got).all() and off[i] <= 1.0, (what, i, got[i], want[i], off[i])


def _check_fwd(shape, case, qo, ko, pos=None):
    th = Q.angles(case["pos"].cpu().numpy() if pos is None else pos, case["freq"], shape.sec)
    for n, H, out in (("q", shape.Hq, qo), ("k", shape.Hk, ko)):
        if not H:
            continue
        x, g = as64(case[n]), None if case["g" + n] is None else as64(case["g" + n])
        want = Q.qk_fwd(x, g, th, shape.dh, shape.rot, shape.layout, shape.eps)
        mag = Q.magnitudes(x, g, None, shape.dh, shape.rot, shape.layout, shape.eps)["y"]
        _close(out, want, mag, shape.dtype, 40, n)


def _check_bwd(shape, case, run, pos=None):
    th = Q.angles(case["pos"].cpu().numpy() if pos is None else pos, case["freq"], shape.sec)
    for n, H, dx, dg in (("q", shape.Hq, run.dq, run.dgq), ("k", shape.Hk, run.dk, run.dgk)):
        if not H:
            continue
        g = None if case["g" + n] is None else as64(case["g" + n])
        x, dy = as64(case[n]), as64(case[f"d{n}o"])
        args = (shape.dh, shape.rot, shape.layout, shape.eps)
        want, mag = Q.qk_bwd(x, g, th, dy, *args), Q.magnitudes(x, g, dy, *args)
        _close(dx, want["dx"], mag["dx"], shape.dtype, 100, "d" + n)
        if g is not None:
            _close(dg, want["dg"], mag["dg"], "f32", 256, "dg" + n)


SHAPES = [
    _shape(1, 32, 8, 128),                                  # one token
    _shape(1, 1, 1, 8),                                     # the smallest vectors
    _shape(3, 5, 1, 80, 56, layout="pairs"),                # odd head count, part of an odd width turned
    _shape(37, 7, 2, 72, 40, 2),
    _shape(65, 4, 4, 64, 64, 3),
    _shape(130, 32, 8, 128, 128, 4, layout="pairs"),
    _shape(33, 3, 3, 256, 256, 3),
    _shape(17, 2, 1, 512, 256, 2),                          # the widest
    _shape(9, 2, 2, 496, 496, layout="pairs"),
    _shape(50, 6, 2, 96, 0),                                # norm alone
    _shape(20, 2, 0, 128),                                  # queries alone
    _shape(20, 0, 3, 128, 64),                              # keys alone
    _shape(700, 1, 1, 24, 8),
    _shape(5, 100, 1, 16),
    _shape(1000, 16, 4, 128),
    _shape(7, 3, 2, 248, 8, layout="pairs"),
    _shape(31, 7, 3, 40),                                   # 5, 9 and 10 lanes to a vector
    _shape(29, 5, 2, 80, 80, 2),
    _shape(45, 3, 1, 144, 96, 3, layout="pairs"),
    _shape(23, 4, 2, 160),
    _shape(21, 3, 1, 16, 16, 4),                            # more than two axes in one lane
    _shape(21, 3, 1, 64, 24, 4, layout="pairs"),
    _shape(11, 2, 2, 336, 320, 4, layout="pairs"),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"T{s.T}-{s.Hq}-{s.Hk}-dh{s.dh}-rot{s.rot}-{len(s.sec)}-{s.layout}")
def test_forward_and_backward_match_the_oracle(shape, dtype, norm):
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = dataclasses.replace(shape, dtype=dtype)
    case = I.make_qk_case(shape, seed=shape.T + shape.dh, norm=norm)
    run = QkRotary(shape, case)
    run.step()
    torch.cuda.synchronize()
    _check_fwd(shape, case, run.qo, run.ko)
    _check_bwd(shape, case, run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1000, -(1 << 31), -500])
def test_far_and_negative_positions(dtype, far):
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = _shape(11, 2, 1, 64, 64, 2, dtype=dtype)
    case = I.make_qk_case(shape, seed=2, far=far)
    run = QkRotary(shape, case)
    run.step()
    _check_fwd(shape, case, run.qo, run.ko)
    _check_bwd(shape, case, run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(19, 5, 2, 128, 128, 3), (1, 4, 2, 64, 32, 1), (40, 3, 1, 72, 40, 2)])
def test_columns_of_a_packed_matrix_in_place(dtype, dims):
    """q and k are columns of one [T, (Hq + 2 Hk) dh + 8] matrix with rows further apart than that; outputs replace
    them; nothing else of the matrix changes."""
    from rank_bottleneck_block_gb300 import lowrank as L

    shape = _shape(*dims, dtype=dtype)
    case = I.make_qk_case(shape, seed=5)
    T, nq, nk = shape.T, shape.Hq * shape.dh, shape.Hk * shape.dh
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    dt = L.dtype_code(case["q"])
    ld = nq + 2 * nk + 16
    turns = L.lr_rot_turns(case["freq"])
    turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device="cuda")
    pos, gq, gk = (case[n].cuda() for n in ("pos", "gq", "gk"))
    sh = L.qk_shape(shape.Hq, shape.Hk, shape.dh, shape.rot, shape.sec)

    def packed(a, b):
        m = torch.full((T + 2, ld), 7.0, dtype=td)
        m[1:T + 1, :nq], m[1:T + 1, nq:nq + nk] = a, b
        return m.cuda()

    def untouched(m):
        rest = m.clone()
        rest[1:T + 1, :nq + nk] = 7.0
        assert (rest == 7.0).all()
        return m[1:T + 1, :nq], m[1:T + 1, nq:nq + nk]

    x = packed(case["q"], case["k"])
    q, k = x[1:T + 1, :nq], x[1:T + 1, nq:nq + nk]
    d = packed(case["dqo"], case["dko"])
    dq, dk = d[1:T + 1, :nq], d[1:T + 1, nq:nq + nk]
    dgq, dgk = torch.empty(shape.dh, device="cuda"), torch.empty(shape.dh, device="cuda")
    ws = torch.empty(L.lr_qk_bwd_workspace_bytes(dt, T, sh), dtype=torch.uint8, device="cuda")
    L.lr_qk_bwd(dt, T, sh, shape.eps, turns, pos, gq, gk, q, ld, k, ld, dq, ld, dk, ld, dq, ld, dk, ld, dgq, dgk, ws)
    L.lr_qk_fwd(dt, T, sh, shape.eps, turns, pos, gq, gk, q, ld, k, ld, q, ld, k, ld)
    torch.cuda.synchronize()

    class Got:
        pass

    qo, ko = untouched(x)
    _check_fwd(shape, case, qo, ko)
    Got.dq, Got.dk = untouched(d)
    Got.dgq, Got.dgk = dgq, dgk
    _check_bwd(shape, case, Got)


def test_without_positions_tokens_count_from_each_sequence_start():
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = _shape(50, 3, 2, 64, 48, 2, seq=16)
    case = I.make_qk_case(shape, seed=8)
    case["pos"] = None
    run = QkRotary(shape, case)
    run.step()
    pos = np.tile(np.arange(50) % 16, (2, 1))
    _check_fwd(shape, case, run.qo, run.ko, pos)
    _check_bwd(shape, case, run, pos)


@pytest.mark.parametrize("which", ["gq", "gk"])
def test_the_norm_of_one_tensor_alone(which):
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = _shape(29, 4, 2, 128)
    case = I.make_qk_case(shape, seed=9)
    case[which] = None
    run = QkRotary(shape, case)
    run.step()
    assert (run.dgq is None) == (which == "gq") and (run.dgk is None) == (which == "gk")
    _check_fwd(shape, case, run.qo, run.ko)
    _check_bwd(shape, case, run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_vectors_of_zeros_and_of_extreme_scale(dtype):
    """A zero vector gives zero (r = eps^-1/2), and its gradient is r w; scales from 1e-6 to 1e6 beside it."""
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = _shape(12, 2, 2, 64, dtype=dtype)
    case = I.make_qk_case(shape, seed=10)
    for n in ("q", "k"):
        for t, s in enumerate([0.0, 1e-6, 1e-3, 1e3, 1e6]):
            case[n][t] = (case[n][t].float() * s).to(case[n].dtype)
    run = QkRotary(shape, case)
    run.step()
    assert (run.qo[0] == 0).all() and (run.ko[0] == 0).all()
    _check_fwd(shape, case, run.qo, run.ko)
    _check_bwd(shape, case, run)


def test_what_is_not_finite_stays_in_its_vector():
    """A NaN or an infinity reaches its own head vector only (without the norm: its own pair only)."""
    from rank_bottleneck_block_gb300.runner import QkRotary

    for norm in (True, False):
        shape = _shape(6, 4, 2, 64, 32, dtype="f32")
        case = I.make_qk_case(shape, seed=11, norm=norm)
        clean = QkRotary(shape, case)
        clean.step()
        bad = dict(case, q=case["q"].clone(), dqo=case["dqo"].clone())
        for m in (bad["q"], bad["dqo"]):
            m[2, 64 + 3] = float("nan")    # head 1, pair (3, 19)
            m[3, 2 * 64 + 40] = float("inf")  # head 2, a channel that is not turned
        run = QkRotary(shape, bad)
        run.step()
        for got, want in ((run.qo, clean.qo), (run.dq, clean.dq)):
            hit = torch.zeros_like(got, dtype=torch.bool)
            if norm:
                hit[2, 64:128] = hit[3, 128:192] = True
            else:
                hit[2, 64 + 3] = hit[2, 64 + 19] = hit[3, 128 + 40] = True
            assert torch.equal(got[~hit], want[~hit])
            assert not torch.isfinite(got[2, 64 + 3]) and not torch.isfinite(got[3, 128 + 40])
        assert torch.equal(run.ko, clean.ko) and torch.equal(run.dk, clean.dk)


def test_repeats_bitwise_and_in_a_graph_and_on_another_stream():
    from rank_bottleneck_block_gb300.runner import GraphStep, QkRotary

    shape = _shape(777, 12, 4, 128, 128, 3)
    case = I.make_qk_case(shape, seed=12)
    run = QkRotary(shape, case)

    def outs():
        return [t.clone() for t in (run.qo, run.ko, run.dq, run.dk, run.dgq, run.dgk)]

    def wipe():
        for t in (run.qo, run.ko, run.dq, run.dk, run.dgq, run.dgk):
            t.zero_()

    run.step()
    ref = outs()
    for _ in range(3):
        run.step()
    assert all(torch.equal(a, b) for a, b in zip(ref, outs()))
    graph = GraphStep(run.step)
    for _ in range(2):
        wipe()
        graph()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs()))
    side = torch.cuda.Stream()
    wipe()
    side.wait_stream(torch.cuda.current_stream())
    run.step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, outs()))


def test_sections_of_no_pairs():
    """An axis may own no pairs: the others' positions alone count."""
    from rank_bottleneck_block_gb300.runner import QkRotary

    for sec in ((0, 32), (32, 0), (0, 0, 32), (5, 0, 20, 7)):
        shape = dataclasses.replace(_shape(19, 2, 1, 64, dtype="f32"), sec=sec)
        case = I.make_qk_case(shape, seed=14)
        run = QkRotary(shape, case)
        run.step()
        _check_fwd(shape, case, run.qo, run.ko)
        _check_bwd(shape, case, run)


def test_tensors_elsewhere_are_refused():
    """Buffers that are not on the current GPU are refused before anything is launched."""
    from rank_bottleneck_block_gb300 import lowrank as L
    from rank_bottleneck_block_gb300.runner import GradClip, QkRotary

    shape = _shape(5, 2, 1, 64)
    case = I.make_qk_case(shape, seed=18)
    run = QkRotary(shape, case, device="cpu")
    before = L.lr_launch_count()
    with pytest.raises(ValueError, match="current device"):
        run.forward()
    with pytest.raises(ValueError, match="current device"):
        GradClip([torch.zeros(64)]).clip()
    assert L.lr_launch_count() == before
    with pytest.raises(ValueError, match="one device"):
        L.Prepared("lr_grad_norm", L.LR_F32, 0, None, None, torch.zeros(4, device="cuda"), torch.zeros(4), 16)


def test_launches_are_counted():
    from rank_bottleneck_block_gb300 import lowrank as L
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = _shape(40, 4, 2, 64)
    for norm, want in ((True, 3), (False, 2)):
        run = QkRotary(shape, I.make_qk_case(shape, seed=15, norm=norm))
        before = L.lr_launch_count()
        run.step()
        assert L.lr_launch_count() - before == want
    L.lr_profile_start()
    run.step()
    assert {"qk_fwd", "qk_bwd"} <= set(L.lr_profile_stop())


def test_rows_past_2_to_the_31_elements():
    """Rows so far apart that the last ones start past element 2^31 of their tensor."""
    from rank_bottleneck_block_gb300 import lowrank as L

    T, dh, ld = 40000, 64, 65536
    shape = _shape(T, 1, 0, dh, seq=T)
    case = I.make_qk_case(shape, seed=16)
    wide = [torch.empty(T, ld, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for m, n in zip(wide, ("q", "dqo")):
        m[:, :dh] = case[n].cuda()
    sh = L.qk_shape(1, 0, dh, dh, (dh // 2,), seq=T)
    turns, g = L.turns_tensor(case["freq"], "cuda"), case["gq"].cuda()
    dg = torch.empty(dh, device="cuda")
    ws = torch.empty(L.lr_qk_bwd_workspace_bytes(L.LR_BF16, T, sh), dtype=torch.uint8, device="cuda")
    x, d = wide
    L.lr_qk_bwd(L.LR_BF16, T, sh, shape.eps, turns, None, g, None, x, ld, None, 0, d, ld, None, 0, d, ld, None, 0, dg, None,
                ws)
    L.lr_qk_fwd(L.LR_BF16, T, sh, shape.eps, turns, None, g, None, x, ld, None, 0, x, ld, None, 0)
    rows = I.sample_rows(T, 64)
    part = dataclasses.replace(shape, T=len(rows))
    sub = {n: case[n][rows] for n in ("q", "dqo")}
    sub.update(gq=case["gq"], freq=case["freq"])
    pos = rows.numpy()[None]
    _check_fwd(part, sub, x[:, :dh][rows.cuda()], None, pos)
    th = Q.angles(pos, case["freq"], shape.sec)
    args = (dh, dh, "half", shape.eps)
    want = Q.qk_bwd(as64(sub["q"]), as64(case["gq"]), th, as64(sub["dqo"]), *args)
    mag = Q.magnitudes(as64(sub["q"]), as64(case["gq"]), as64(sub["dqo"]), *args)
    _close(d[:, :dh][rows.cuda()], want["dx"], mag["dx"], "bf16", 100, "dq")


def test_graphs_that_share_a_workspace():
    """Two captured backward passes with one workspace, replayed one after the other on one stream."""
    from rank_bottleneck_block_gb300 import lowrank as L
    from rank_bottleneck_block_gb300.runner import GraphStep, QkRotary

    runs = [QkRotary(s, I.make_qk_case(s, seed=17)) for s in (_shape(500, 6, 2, 128), _shape(90, 3, 3, 64, 48, 2))]
    ref = []
    for r in runs:
        r.backward()
        ref.append([t.clone() for t in (r.dq, r.dk, r.dgq, r.dgk)])
    ws = max((r.ws for r in runs), key=lambda t: t.numel())

    def call(r):
        rows = [v for t in (r.dqo, r.dko, r.dq, r.dk) for v in (t, t.stride(0))]
        s = r.s
        return lambda: L.lr_qk_bwd(r.dt, s.T, r.sh, s.eps, r.turns, r.pos, r.gq, r.gk, r.q, r.q.stride(0), r.k,
                                   r.k.stride(0), *rows, r.dgq, r.dgk, ws)

    graphs = [GraphStep(call(r)) for r in runs]
    for _ in range(3):
        for r in runs:
            for t in (r.dq, r.dk, r.dgq, r.dgk):
                t.zero_()
        for g in graphs:
            g()
        for r, want in zip(runs, ref):
            assert all(torch.equal(a, b) for a, b in zip(want, (r.dq, r.dk, r.dgq, r.dgk)))


def test_two_runs_at_once_on_two_streams():
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = _shape(3000, 8, 8, 128)
    runs = [QkRotary(shape, I.make_qk_case(shape, seed=s)) for s in (1, 2)]
    ref = []
    for r in runs:
        r.step()
        torch.cuda.synchronize()
        ref.append([t.clone() for t in (r.qo, r.ko, r.dq, r.dk, r.dgq, r.dgk)])
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for r, st in zip(runs, streams):
            r.step(st)
    torch.cuda.synchronize()
    for r, want in zip(runs, ref):
        assert all(torch.equal(a, b) for a, b in zip(want, (r.qo, r.ko, r.dq, r.dk, r.dgq, r.dgk)))


def test_the_training_batch_on_sampled_tokens():
    """4 x 4096 tokens, 32 heads of 128: sampled tokens' outputs and input gradients against the oracle, dg against
    fp64 sums on the GPU."""
    from rank_bottleneck_block_gb300.runner import QkRotary

    shape = _shape(16384, 32, 32, 128, seq=4096)
    case = I.make_qk_case(shape, seed=3, device="cuda")
    case["pos"] = None
    run = QkRotary(shape, case)
    run.step()
    rows = I.sample_rows(shape.T, 64)
    part = dataclasses.replace(shape, T=len(rows))
    sub = {n: v[rows.cuda()].cpu() if n in ("q", "k", "dqo", "dko") else v for n, v in case.items()}
    pos = rows.numpy()[None] % 4096
    _check_fwd(part, sub, run.qo[rows.cuda()], run.ko[rows.cuda()], pos)

    th = Q.angles(pos, case["freq"], shape.sec)
    for n, dx in (("q", run.dq[rows.cuda()]), ("k", run.dk[rows.cuda()])):
        args = (shape.dh, shape.rot, shape.layout, shape.eps)
        x, g, dy = as64(sub[n]), as64(case["g" + n]), as64(sub[f"d{n}o"])
        want, mag = Q.qk_bwd(x, g, th, dy, *args), Q.magnitudes(x, g, dy, *args)
        _close(dx, want["dx"], mag["dx"], "bf16", 100, "d" + n)
    # dg = sum dn x r in fp64, the angles from the turns of positions below 4096 (exact in fp64 to 1e-12)
    theta = (torch.arange(16384, device="cuda") % 4096).double()[:, None] * \
        torch.tensor(case["freq"], dtype=torch.float64, device="cuda")
    c, s = theta.cos()[:, None], theta.sin()[:, None]
    for n, dg in (("q", run.dgq), ("k", run.dgk)):
        dy = case[f"d{n}o"].double().view(16384, 32, 128)
        dn = torch.cat([dy[..., :64] * c + dy[..., 64:] * s, dy[..., 64:] * c - dy[..., :64] * s], -1)
        x = case[n].double().view(16384, 32, 128)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + shape.eps)
        term = dn * x
        mag = (dy[..., :64].abs() + dy[..., 64:].abs()).repeat(1, 1, 2) * x.abs()
        # at most 1500 additions in a row: 2^19 vectors over the blocks' warps, then the partial sums
        _close(dg, term.sum((0, 1)).cpu().numpy(), mag.sum((0, 1)).cpu().numpy(), "f32", 1500, "dg" + n)
