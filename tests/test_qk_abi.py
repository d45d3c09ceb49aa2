"""lr_rot_turns, lr_qk_* and lr_grad_* without a GPU: the host arithmetic, size queries and refusals."""
import ctypes
from fractions import Fraction

import pytest

import oracle.qk_oracle as Q

P = 0x10000  # a 16-byte aligned fake address: what reaches validation never launches


@pytest.fixture(scope="module")
def L():
    from rank_bottleneck_block_gb300 import build

    build.build()
    from rank_bottleneck_block_gb300 import lowrank

    lowrank.lib()
    return lowrank


def test_turns_are_the_frequencies_modulo_a_turn(L):
    freq = [10000.0 ** (-p / 64) for p in range(64)] + [0.0, 1e-300, 1.0, 6.283185307179586, 3.5, 65536.0, 12345.678,
                                                        5e-20, 2.0 ** -60]
    freq += [-f for f in freq]
    for f, got in zip(freq, L.lr_rot_turns(freq)):
        want = Fraction(f) / Q.TWO_PI % 1 * 2 ** 64
        off = abs(got - want)
        off = min(off, 2 ** 64 - off)
        # the last bit of the result, and the 2^-100 (of the frequency) that two doubles of 1/(2 pi) leave out
        assert off <= 2, (f, got, float(want))


def test_turns_refusals(L):
    assert L.lr_rot_turns([]) == []
    for bad in (float("nan"), float("inf"), 65537.0, -1e9):
        with pytest.raises(L.LowRankError) as e:
            L.lr_rot_turns([1.0, bad])
        assert e.value.status == 2 and "freq[1]" in str(e.value)
    lib = L.lib()
    assert lib.lr_rot_turns(1, None, None) == 1
    assert lib.lr_rot_turns(-1, None, None) == 2


def _shape(L, **over):
    a = dict(Hq=4, Hk=2, dh=64, rot=64, sec=(32,), layout=0, seq=0)
    a.update(over)
    return L.qk_shape(**a)


def _fwd(L, dt=1, T=16, sh=None, eps=1e-6, turns=P, pos=P, gq=P, gk=P, q=P, ldq=256, k=P, ldk=128, qo=P, ldqo=256, ko=P,
         ldko=128):
    return L.lib().lr_qk_fwd(dt, T, ctypes.byref(sh or _shape(L)), eps, turns, pos, gq, gk, q, ldq, k, ldk, qo, ldqo, ko,
                             ldko, None)


def _bwd(L, dt=1, T=16, sh=None, eps=1e-6, turns=P, pos=P, gq=P, gk=P, q=P, ldq=256, k=P, ldk=128, dqo=P, lddqo=256,
         dko=P, lddko=128, dq=P, lddq=256, dk=P, lddk=128, dgq=P, dgk=P, ws=P, ws_bytes=1 << 30):
    return L.lib().lr_qk_bwd(dt, T, ctypes.byref(sh or _shape(L)), eps, turns, pos, gq, gk, q, ldq, k, ldk, dqo, lddqo,
                             dko, lddko, dq, lddq, dk, lddk, dgq, dgk, ws, ws_bytes, None)


SHAPE_REFUSALS = [  # (overrides of the shape, status)
    (dict(dh=60, rot=56, sec=(28,)), 2),  # dh not a multiple of 8
    (dict(rot=60, sec=(30,)), 2),
    (dict(rot=72, sec=(36,)), 2),  # rot > dh
    (dict(rot=-8, sec=(-4,)), 2),
    (dict(dh=264, rot=8, sec=(4,)), 2),  # above 256 both must be multiples of 16
    (dict(dh=272, rot=8, sec=(4,)), 2),
    (dict(dh=528, rot=16, sec=(8,)), 2),
    (dict(dh=0, rot=0, sec=(0,)), 2),
    (dict(Hq=0, Hk=0), 2),
    (dict(Hq=-1), 2),
    (dict(Hk=1 << 19), 2),  # Hk*dh = 2^25 channels
    (dict(layout=2), 4),
    (dict(sec=(31,)), 2),  # sections do not hold every pair
    (dict(sec=(16, 17)), 2),
    (dict(sec=(40, -8)), 2),
]


@pytest.mark.parametrize("over,status", SHAPE_REFUSALS)
def test_shapes_are_refused(L, over, status):
    sh = _shape(L, **over)
    assert _fwd(L, sh=sh) == status
    assert L.lr_last_error()
    assert _bwd(L, sh=sh) == status
    assert L.lr_qk_bwd_workspace_bytes(1, 16, sh) == 0


def test_too_many_vectors_are_refused(L):
    sh = _shape(L, Hq=64, Hk=1)  # 2^24 tokens of 64 heads: 2^30 vectors are the most
    assert L.lr_qk_bwd_workspace_bytes(1, 1 << 24, sh) > 0
    sh.Hq = 65
    assert L.lr_qk_bwd_workspace_bytes(1, 1 << 24, sh) == 0


def test_axes_are_refused(L):
    sh = _shape(L)
    for axes in (0, 5, -1):
        sh.axes = axes
        assert _fwd(L, sh=sh) == 2
    for sec in ((), (8,) * 5):
        with pytest.raises(ValueError):
            _shape(L, sec=sec)


FWD_REFUSALS = [
    (dict(dt=2), 4), (dict(T=0), 2), (dict(T=(1 << 24) + 1), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(eps=float("inf")), 2),
    (dict(turns=None), 1), (dict(turns=P + 8), 3), (dict(pos=P + 4), 3), (dict(pos=None), 2),  # no positions, no seq
    (dict(gq=P + 2), 3), (dict(gk=P + 2), 3), (dict(q=None), 1), (dict(q=P + 8), 3), (dict(ldq=255), 2),
    (dict(ldq=248), 2), (dict(ldq=260), 2), (dict(ldq=1 << 32), 2), (dict(k=None), 1), (dict(ldk=120), 2), (dict(qo=None), 1),
    (dict(ldqo=0), 2), (dict(ko=None), 1), (dict(ldko=-128), 2),
]


@pytest.mark.parametrize("over,status", FWD_REFUSALS)
def test_forward_refusals(L, over, status):
    assert _fwd(L, **over) == status


BWD_REFUSALS = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(dqo=None), 1), (dict(lddqo=128), 2), (dict(dko=None), 1),
    (dict(lddko=64), 2), (dict(dq=None), 1), (dict(lddq=250), 2), (dict(dk=P + 4), 3), (dict(lddk=0), 2),
    (dict(dgq=None), 1), (dict(dgk=None), 1), (dict(ws=None), 1), (dict(ws_bytes=16), 5), (dict(pos=None), 2),
]


@pytest.mark.parametrize("over,status", BWD_REFUSALS)
def test_backward_refusals(L, over, status):
    assert _bwd(L, **over) == status


def test_unused_arguments_are_not_asked_for(L):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a device is present: these calls would launch")
    ok = 8  # validated, but no device
    assert _fwd(L) == ok and _bwd(L) == ok
    assert _fwd(L, sh=_shape(L, Hk=0), k=None, ko=None, gk=None, ldk=0, ldko=0) == ok
    assert _fwd(L, sh=_shape(L, Hq=0), q=None, qo=None, gq=None, ldq=0, ldqo=0) == ok
    assert _fwd(L, gq=None, gk=None) == ok
    assert _bwd(L, gq=None, gk=None, q=None, k=None, dgq=None, dgk=None) == ok
    assert _bwd(L, gk=None, k=None, dgk=None) == ok
    assert _fwd(L, pos=None, sh=_shape(L, seq=4)) == ok
    assert _fwd(L, turns=None, pos=None, sh=_shape(L, rot=0, sec=(0,))) == ok  # nothing is turned
    wide = dict(ldq=512, ldk=512, ldqo=512, ldko=512)
    assert _fwd(L, sh=_shape(L, dh=512, rot=512, sec=(128, 128, 0, 0), Hq=1, Hk=1), **wide) == ok
    assert _fwd(L, sh=_shape(L, dh=512, rot=512, sec=(128, 127), Hq=1, Hk=1), **wide) == 2  # 256 pairs needed


def _arr(L, numel, ptr=P):
    n = len(numel)
    return (ctypes.c_void_p * max(n, 1))(*[ptr] * n), (ctypes.c_longlong * max(n, 1))(*numel)


def _clip(L, numel=(8, 9), dt=0, max_norm=1.0, stat=P, ws=P, ws_bytes=1 << 20, ptr=P, n=None, outs=True):
    g, m = _arr(L, numel, ptr)
    n = len(numel) if n is None else n
    return L.lib().lr_grad_clip(dt, n, g, m, max_norm, g if outs else None, stat, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(dt=3), 4), (dict(n=-1), 2), (dict(n=65537), 2), (dict(numel=(8, -1)), 2), (dict(numel=(1 << 40,)), 2),
    (dict(ptr=None), 1), (dict(ptr=P + 4), 3), (dict(max_norm=-1.0), 2), (dict(max_norm=float("nan")), 2),
    (dict(max_norm=float("inf")), 2), (dict(stat=None), 1), (dict(stat=P + 4), 3), (dict(ws=None), 1),
    (dict(ws_bytes=8), 5), (dict(outs=False), 1),
])
def test_clip_refusals(L, over, status):
    assert _clip(L, **over) == status


def test_grad_size_queries_and_unused_pointers(L):
    import torch

    one = L.lr_grad_workspace_bytes(1)
    assert one > 0 and L.lr_grad_workspace_bytes(0) > 0 and L.lr_grad_workspace_bytes(65536) > one
    assert L.lr_grad_workspace_bytes(-1) == 0 and L.lr_grad_workspace_bytes(65537) == 0
    if torch.cuda.is_available():
        pytest.skip("a device is present: the rest would launch")
    assert _clip(L) == 8
    assert _clip(L, numel=(0, 0), ptr=None) == 8
    assert _clip(L, numel=()) == 8
    assert L.lib().lr_grad_norm(0, 0, None, None, P, P, 1 << 20, None) == 8


def test_clip_runner_refuses_what_it_cannot_scale():
    import torch

    from rank_bottleneck_block_gb300.runner import GradClip

    a, b = torch.zeros(64), torch.zeros(64)
    for grads, outs in [([], None), ([a, b.bfloat16()], None), ([a], [a, b]), ([a], [b[:32]]),
                        ([torch.zeros(8, 8).T], None), ([a, a], None), ([a, a[16:32]], None), ([a, b], [b, b]),
                        ([a, b], [b, a]), ([a[:32], a[32:]], [a[32:], b[:32]]), ([a.double()], None)]:
        with pytest.raises((ValueError, TypeError)):
            GradClip(grads, 1.0, outs)
    GradClip([a, b], 1.0)
    GradClip([a[:32], a[32:]], 1.0)
    GradClip([a, a], 1.0, [b, torch.zeros(64)])  # read twice, written apart


def test_rotary_runner_refuses_mismatched_inputs():
    import dataclasses

    from rank_bottleneck_block_gb300 import inputs as I
    from rank_bottleneck_block_gb300.runner import QkRotary

    sh = I.QkShape(T=4, Hq=2, Hk=1, dh=16, rot=16, sec=(8,), dtype="f32")
    case = I.make_qk_case(sh)
    QkRotary(sh, case, device="cpu")
    for name, bad in [("q", case["q"][:, :16]), ("q", case["q"].bfloat16()), ("gq", case["gq"][:8]),
                      ("pos", case["pos"].long()), ("pos", case["pos"][:, :3]), ("freq", case["freq"][:4]),
                      ("dko", case["dko"].T)]:
        with pytest.raises(ValueError):
            QkRotary(sh, dict(case, **{name: bad}), device="cpu")
    with pytest.raises(KeyError):
        QkRotary(dataclasses.replace(sh, layout="other"), case, device="cpu")


def test_block_with_rotation_shape_rules_and_refusals(L):
    dims = (1, 256, 2, 128, 344, 32, 48)
    act = 256 * 256 * 2
    assert L.lr_block_qk_saved_bytes(*dims) >= L.lr_block_saved_bytes(*dims) + 2 * act  # q' and k' too
    assert L.lr_block_qk_workspace_bytes(*dims) >= L.lr_block_workspace_bytes(*dims)
    assert L.lr_block_qk_saved_bytes(1, 200, 2, 128, 344, 32, 48) == 0  # s not a multiple of 256
    assert L.lr_block_qk_workspace_bytes(1, 256, 2, 640, 344, 32, 48) == 0  # dh above 512
    lib = L.lib()
    w, g = L.lr_block_weights(), L.lr_block_grads()

    def qk(H=2, dh=128, rot=64, sec=(32,), turns=P, pos=None, gq=P, gk=P):
        return L.lr_block_qk(L.qk_shape(H, H, dh, rot, sec), turns, pos, gq, gk)

    def fwd(q, dt=L.LR_BF16, eps=1e-6):
        return lib.lr_block_qk_fwd(dt, *dims, eps, P, ctypes.byref(w), ctypes.byref(q) if q else None, P, P, 1 << 30, P,
                                   1 << 30, None)

    def bwd(q, dgq=P, dgk=P):
        return lib.lr_block_qk_bwd(L.LR_BF16, *dims, 1e-6, P, ctypes.byref(w), ctypes.byref(q), P, 1 << 30, P, P,
                                   ctypes.byref(g), dgq, dgk, P, 1 << 30, None)

    assert fwd(qk(), dt=L.LR_F32) == 8
    assert fwd(None) == 1
    assert fwd(qk(H=1)) == 2 and "the block has" in L.lr_last_error()
    assert fwd(qk(dh=64)) == 2
    assert fwd(qk(rot=60, sec=(30,))) == 2
    assert fwd(qk(turns=None)) == 1
    assert fwd(qk(pos=P + 4)) == 3
    assert fwd(qk(gq=P + 2)) == 3
    assert fwd(qk(), eps=float("nan")) == 2
    assert fwd(qk()) == 1 and "weight" in L.lr_last_error()  # the rotation is accepted, the weights are missing
    assert bwd(qk(), dgq=None) == 1 and "dgq" in L.lr_last_error()
    assert bwd(qk(), dgk=P + 4) == 3
    assert bwd(qk(gq=None, gk=None), dgq=None, dgk=None) == 1 and "weight" in L.lr_last_error()


def test_block_runner_refuses_a_rotation_of_other_sizes():
    import dataclasses

    from rank_bottleneck_block_gb300 import inputs as I
    from rank_bottleneck_block_gb300.runner import TransformerBlock

    shape = I.BlockShape(1, 256, 2, 128, 344, 32, 48)
    case = dict(I.make_block_case(shape), freq=I.rotary_freq(128))
    qk = I.QkShape(T=256, Hq=2, Hk=2, dh=128, rot=128, sec=(64,))
    TransformerBlock(shape, case, device="cpu", qk=qk)
    for bad in (dict(T=512), dict(Hk=1), dict(dh=64), dict(dtype="f32"), dict(rot=64, sec=(32,))):
        with pytest.raises(ValueError):
            TransformerBlock(shape, case, device="cpu", qk=dataclasses.replace(qk, **bad))
    import torch

    for bad in (dict(pos=torch.zeros(1, 256)), dict(gq=torch.ones(128)), dict(gk=torch.ones(64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            TransformerBlock(shape, dict(case, **bad), device="cpu", qk=qk)
