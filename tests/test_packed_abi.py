"""lr_packed_attn_* and lr_logprob_* without a GPU: size queries and refusals, of the entry points and of the runners."""
import ctypes

import pytest
import torch

from rank_bottleneck_block_gb300 import inputs as I
from rank_bottleneck_block_gb300 import runner as R

P = 0x10000  # a 16-byte aligned fake address: what reaches validation never launches


@pytest.fixture(scope="module")
def L():
    from rank_bottleneck_block_gb300 import build

    build.build()
    from rank_bottleneck_block_gb300 import lowrank

    lowrank.lib()
    return lowrank


def _sh(L, T=16, nseq=2, Hq=4, Hk=2, dh=64):
    return L.lr_packed_shape(T, nseq, Hq, Hk, dh)


def _fwd(L, sh=None, dt=1, scale=0.1, offs=P, q=P, ldq=256, k=P, ldk=128, v=P, ldv=128, o=P, ldo=256, lse=P, ws=P,
         ws_bytes=1 << 30):
    sh = _sh(L) if sh is None else sh
    return L.lib().lr_packed_attn_fwd(dt, ctypes.byref(sh) if sh else None, scale, offs, q, ldq, k, ldk, v, ldv, o, ldo,
                                      lse, ws, ws_bytes, None)


def _bwd(L, sh=None, dt=1, scale=0.1, offs=P, q=P, ldq=256, k=P, ldk=128, v=P, ldv=128, o=P, ldo=256, lse=P, dout=P,
         lddout=256, dq=P, lddq=256, dk=P, lddk=128, dv=P, lddv=128, ws=P, ws_bytes=1 << 30):
    sh = _sh(L) if sh is None else sh
    return L.lib().lr_packed_attn_bwd(dt, ctypes.byref(sh) if sh else None, scale, offs, q, ldq, k, ldk, v, ldv, o, ldo,
                                      lse, dout, lddout, dq, lddq, dk, lddk, dv, lddv, ws, ws_bytes, None)


@pytest.mark.parametrize("over", [
    dict(T=0), dict(T=-5), dict(nseq=0), dict(nseq=(1 << 24) + 1), dict(Hq=0), dict(Hk=0), dict(Hq=-4), dict(Hk=3),
    dict(Hq=129, Hk=1), dict(dh=0), dict(dh=60), dict(dh=136), dict(dh=-8), dict(T=(1 << 28) + 1), dict(T=2 ** 31 - 1),
])
def test_packed_shapes_are_refused(L, over):
    sh = _sh(L, **over)
    wide = dict(ldq=1 << 20, ldk=1 << 20, ldv=1 << 20, ldo=1 << 20)
    assert _fwd(L, sh, **wide) == 2 and L.lr_last_error()
    assert _bwd(L, sh, **wide) == 2
    assert L.lr_packed_attn_fwd_workspace_bytes(sh) == 0 and L.lr_packed_attn_bwd_workspace_bytes(sh) == 0


@pytest.mark.parametrize("over,status", [
    (dict(dt=0), 8), (dict(dt=2), 4), (dict(sh=False), 1), (dict(scale=0.0), 2), (dict(scale=-1.0), 2),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(offs=None), 1), (dict(offs=P + 4), 3),
    (dict(q=None), 1), (dict(q=P + 8), 3), (dict(ldq=248), 2), (dict(ldq=260), 2), (dict(ldq=1 << 32), 2),
    (dict(k=None), 1), (dict(ldk=120), 2), (dict(v=None), 1), (dict(v=P + 2), 3), (dict(ldv=0), 2), (dict(o=None), 1),
    (dict(ldo=-256), 2), (dict(lse=None), 1), (dict(lse=P + 4), 3), (dict(ws=None), 1), (dict(ws=P + 8), 3),
    (dict(ws_bytes=16), 5),
])
def test_packed_refusals(L, over, status):
    assert _fwd(L, **over) == status
    assert _bwd(L, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dout=None), 1), (dict(lddout=100), 2), (dict(dq=None), 1), (dict(dq=P + 4), 3), (dict(lddq=264 + 4), 2),
    (dict(dk=None), 1), (dict(lddk=64), 2), (dict(dv=None), 1), (dict(lddv=64), 2),
])
def test_packed_backward_refusals(L, over, status):
    assert _bwd(L, **over) == status


def test_packed_workspace_grows_with_what_it_holds(L):
    size = L.lr_packed_attn_fwd_workspace_bytes
    assert 0 < size(_sh(L)) <= size(_sh(L, T=1 << 20)) and size(_sh(L, nseq=1 << 20)) >= size(_sh(L))
    assert L.lr_packed_attn_bwd_workspace_bytes(_sh(L)) > 0
    if torch.cuda.is_available():
        pytest.skip("a device is present: the rest would launch")
    assert _fwd(L) == 8 and _bwd(L) == 8  # validated, but no device
    assert _fwd(L, ldq=512, ldk=512, ldv=512, ldo=1024) == 8
    assert _fwd(L, _sh(L, Hq=128, Hk=1, dh=8), ldq=1024, ldo=1024) == 8


def _lfwd(L, dt=1, T=4, V=100, scale=1.0, top=2, logits=P, ld=100, target=P, logp=P, entropy=P, lse=P, top_ids=P,
          top_logp=P, ws=P, ws_bytes=1 << 30):
    return L.lib().lr_logprob_fwd(dt, T, V, scale, top, logits, ld, target, logp, entropy, lse, top_ids, top_logp, ws,
                                  ws_bytes, None)


def _lbwd(L, dt=1, T=4, V=100, scale=1.0, logits=P, ld=100, target=P, lse=P, entropy=P, dlogp=P, dentropy=P, dlogits=P,
          ldd=100):
    return L.lib().lr_logprob_bwd(dt, T, V, scale, logits, ld, target, lse, entropy, dlogp, dentropy, dlogits, ldd, None)


@pytest.mark.parametrize("over,status", [
    (dict(dt=2), 4), (dict(T=0), 2), (dict(T=(1 << 24) + 1), 2), (dict(V=0), 2), (dict(V=(1 << 19) + 1, ld=1 << 21), 2),
    (dict(scale=0.0), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(logits=None), 1),
    (dict(logits=P + 2), 3), (dict(ld=99), 2), (dict(ld=1 << 32), 2), (dict(target=None), 1), (dict(target=P + 4), 3),
    (dict(lse=None), 1),
])
def test_logprob_refusals(L, over, status):
    assert _lfwd(L, **over) == status
    assert _lbwd(L, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(top=-1), 2), (dict(top=33), 2), (dict(V=1, top=2), 2), (dict(logp=None), 1), (dict(entropy=None), 1),
    (dict(top_ids=None), 1), (dict(top_logp=P + 4), 3), (dict(ws=None), 1), (dict(ws_bytes=0), 5),
])
def test_logprob_forward_refusals(L, over, status):
    assert _lfwd(L, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dlogp=None), 1), (dict(entropy=None), 1), (dict(dentropy=P + 4), 3), (dict(dlogits=None), 1),
    (dict(dlogits=P + 8), 3), (dict(ldd=99), 2),
])
def test_logprob_backward_refusals(L, over, status):
    assert _lbwd(L, **over) == status


def test_logprob_sizes_and_unused_arguments(L):
    assert L.lr_logprob_workspace_bytes(1, 1, 1, 0) > 0
    assert L.lr_logprob_workspace_bytes(1, 4096, 131072, 20) > L.lr_logprob_workspace_bytes(1, 4096, 131072, 0)
    assert L.lr_logprob_workspace_bytes(1, 0, 1, 0) == 0 and L.lr_logprob_workspace_bytes(1, 1, 1, 2) == 0
    if torch.cuda.is_available():
        pytest.skip("a device is present: these calls would launch")
    assert _lfwd(L, top=0, top_ids=None, top_logp=None) == 8
    assert _lbwd(L, dentropy=None, entropy=None) == 8
    assert _lfwd(L, ld=101) == 8 and _lbwd(L, ldd=1000) == 8


PACKED = I.PackedShape(T=12, nseq=3, Hq=4, Hk=2, dh=16)
LOGP = I.LogProbShape(T=6, V=33, top=3, dtype="f32")


def _packed_run(**over):
    return R.PackedAttention(PACKED, dict(I.make_packed_case(PACKED, [5, 0, 7]), **over), device="cpu")


def _logp_run(**over):
    return R.TokenLogProbs(LOGP, dict(I.make_logprob_case(LOGP), **over), device="cpu")


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Prepared:
        def __init__(self, name, *args):
            self.got = (name, [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args])

        def __call__(self, stream=None):
            made.append(self.got)

    monkeypatch.setattr(R.L, "Prepared", Prepared)
    return made


@pytest.mark.parametrize("make,names", [
    (_packed_run, ("offs", "q", "k", "v", "dout", "o", "lse", "dq", "dk", "dv", "ws", "ws_b")),
    (_logp_run, ("logits", "target", "logp", "entropy", "lse", "top_ids", "top_logp", "dlogp", "dentropy", "dlogits", "ws")),
])
def test_an_assigned_tensor_is_the_one_that_is_used(L, calls, make, names):
    run = make()
    run.step()
    for n in names:
        new = torch.empty_like(getattr(run, n))
        setattr(run, n, new)
        calls.clear()
        run.step()
        assert any(new.data_ptr() in args for _, args in calls), n
        if new.dim() == 2 and n not in run._WHOLE:
            wide = torch.empty(new.shape[0], new.shape[1] + 24, dtype=new.dtype)[:, 8:8 + new.shape[1]]
            setattr(run, n, wide)
            calls.clear()
            run.step()
            at = [args.index(wide.data_ptr()) for _, args in calls if wide.data_ptr() in args]
            args = [a for _, a in calls if wide.data_ptr() in a]
            assert at and all(a[i + 1] == new.shape[1] + 24 for a, i in zip(args, at)), n


@pytest.mark.parametrize("make,name,bad", [
    (_packed_run, "q", lambda t: t[:, :32]), (_packed_run, "q", lambda t: t.float()), (_packed_run, "k", lambda t: t[:5]),
    (_packed_run, "offs", lambda t: t.long()), (_packed_run, "offs", lambda t: t[:2]), (_packed_run, "dout", lambda t: t.T),
    (_packed_run, "lse", lambda t: t.T.contiguous().T), (_packed_run, "o", lambda t: t[:, ::2]),
    (_packed_run, "dq", lambda t: t.double()), (_packed_run, "ws", lambda t: t.float()),
    (_packed_run, "v", lambda t: t.to("meta")),
    (_logp_run, "logits", lambda t: t.bfloat16()), (_logp_run, "logits", lambda t: t[:, :30]),
    (_logp_run, "target", lambda t: t.long()), (_logp_run, "dlogp", lambda t: t[:3]),
    (_logp_run, "top_ids", lambda t: t[:, :2]), (_logp_run, "lse", lambda t: t.double()),
    (_logp_run, "dlogits", lambda t: t.T),
])
def test_a_tensor_that_does_not_fit_is_refused(L, calls, make, name, bad):
    run = make()
    old = getattr(run, name)
    with pytest.raises(ValueError):
        setattr(run, name, bad(old))
    assert getattr(run, name) is old


def test_outputs_that_overlap_are_refused(L, calls):
    run = _packed_run()
    for name, other in (("o", "q"), ("dq", "dk"), ("dv", "dk"), ("dq", "dout"), ("dk", "k"), ("dq", "q")):
        run = _packed_run()
        t, target = getattr(run, name), getattr(run, other)
        m = torch.zeros(12, 200, dtype=torch.bfloat16)
        setattr(run, other, m[:, :target.shape[1]])
        setattr(run, name, m[:, 8:8 + t.shape[1]])
        with pytest.raises(ValueError, match="overlaps"):
            run.step()
    run = _logp_run()
    run.dlogits = run.logits  # in place
    run.step()
    m = torch.zeros(6, 80)
    run.logits, run.dlogits = m[:, :33], m[:, 8:41]
    with pytest.raises(ValueError, match="overlaps"):
        run.backward()
    run = _logp_run()
    run.entropy = run.lse
    with pytest.raises(ValueError, match="overlaps"):
        run.forward()


def test_shapes_that_do_not_fit_and_missing_gradients(L, calls):
    for shape in (I.PackedShape(12, 3, 4, 3, 16), I.PackedShape(12, 3, 4, 2, 20), I.PackedShape(0, 3, 4, 2, 16),
                  I.PackedShape(12, 3, 4, 2, 256)):
        with pytest.raises(ValueError):
            R.PackedAttention(shape, I.make_packed_case(PACKED, [5, 0, 7]), device="cpu")
    for shape in (I.LogProbShape(6, 33, 40, dtype="f32"), I.LogProbShape(0, 33, dtype="f32")):
        with pytest.raises(ValueError):
            R.TokenLogProbs(shape, I.make_logprob_case(LOGP), device="cpu")
    with pytest.raises(ValueError):
        I.make_packed_case(PACKED, [5, 7])
    for run in (_packed_run(dout=None), _logp_run(dlogp=None)):
        run.forward()
        with pytest.raises(ValueError, match="upstream"):
            run.backward()
    for run, name in ((_packed_run(), "scale"), (_packed_run(), "sh"), (_logp_run(), "s"), (_logp_run(), "dt")):
        with pytest.raises(AttributeError):
            setattr(run, name, 1)
