"""QkRotary and TransformerBlock when a caller replaces the tensors that they hold."""
import dataclasses

import pytest
import torch

from rank_bottleneck_block_gb300 import inputs as I
from rank_bottleneck_block_gb300 import runner as R


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


SHAPE = I.QkShape(T=6, Hq=3, Hk=2, dh=32, rot=16, sec=(4, 4))
INPUTS = ("q", "k", "gq", "gk", "pos", "dqo", "dko")
OUTPUTS = ("qo", "ko", "dq", "dk", "dgq", "dgk")


def _at(*names):
    """Places of the tensors' pointers among the arguments of lr_qk_fwd and lr_qk_bwd."""
    fwd = ["turns", "pos", "gq", "gk", "q", "ldq", "k", "ldk", "qo", "ldqo", "ko", "ldko"]
    bwd = fwd[:8] + ["dqo", "lddqo", "dko", "lddko", "dq", "lddq", "dk", "lddk", "dgq", "dgk", "ws"]
    return {"lr_qk_fwd": {n: 4 + i for i, n in enumerate(fwd)}, "lr_qk_bwd": {n: 4 + i for i, n in enumerate(bwd)}}


@pytest.fixture
def calls(monkeypatch):
    """Prepared calls that only note what they would be called with: {entry point: {argument: value}}."""
    made = {}

    class Prepared:
        def __init__(self, name, *args):
            self.name, self.args = name, [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]

        def __call__(self, stream=None):
            made[self.name] = {n: self.args[i] for n, i in _at()[self.name].items()}

    monkeypatch.setattr(R.L, "Prepared", Prepared)
    return made


def _wide(t):
    """The same values as columns of a wider matrix."""
    m = torch.zeros(t.shape[0], t.shape[1] + 24, dtype=t.dtype, device=t.device)
    m[:, 8:8 + t.shape[1]] = t
    return m[:, 8:8 + t.shape[1]]


@pytest.mark.parametrize("name", INPUTS + OUTPUTS + ("turns", "ws"))
def test_an_assigned_tensor_is_the_one_that_is_used(calls, name):
    run = R.QkRotary(SHAPE, I.make_qk_case(SHAPE), device="cpu")
    run.step()
    new = torch.empty_like(getattr(run, name))
    setattr(run, name, new)
    run.step()
    used = [c[name] for c in calls.values() if name in c]
    assert used and all(p == new.data_ptr() for p in used)
    if "ld" + name in calls["lr_qk_fwd"] or "ld" + name in calls["lr_qk_bwd"]:
        new = _wide(new)
        setattr(run, name, new)
        run.step()
        for c in calls.values():
            if name in c:
                assert (c[name], c["ld" + name]) == (new.data_ptr(), new.shape[1] + 24)


def test_what_may_be_left_out_may_be_taken_out(calls):
    run = R.QkRotary(dataclasses.replace(SHAPE, seq=2), I.make_qk_case(SHAPE), device="cpu")
    run.pos = run.gq = None
    run.step()
    for c in calls.values():
        assert c["pos"] is None and c["gq"] is None and c["gk"] == run.gk.data_ptr()


@pytest.mark.parametrize("name,bad", [
    ("q", lambda t: t[:, :32]), ("q", lambda t: t.float()), ("k", lambda t: t[:5]), ("dqo", lambda t: t.T),
    ("gq", lambda t: t[:16]), ("gk", lambda t: t.float()), ("pos", lambda t: t.long()), ("pos", lambda t: t[:1]),
    ("pos", lambda t: t.T.contiguous().T), ("qo", lambda t: t[:, ::2]), ("dk", lambda t: t.double()),
    ("dgq", lambda t: t.bfloat16()), ("turns", lambda t: t[:4]), ("turns", lambda t: t.int()),
    ("q", lambda t: t.to("meta")), ("ws", lambda t: t.float()),
])
def test_a_tensor_that_does_not_fit_is_refused_and_the_old_one_stays(calls, name, bad):
    run = R.QkRotary(SHAPE, I.make_qk_case(SHAPE), device="cpu")
    old = getattr(run, name)
    with pytest.raises(ValueError):
        setattr(run, name, bad(old))
    assert getattr(run, name) is old
    run.step()
    assert all(c[name] == old.data_ptr() for c in calls.values() if name in c)


def test_the_shape_is_fixed():
    run = R.QkRotary(SHAPE, I.make_qk_case(SHAPE), device="cpu")
    for name, value in (("s", SHAPE), ("sh", run.sh), ("dt", 0)):
        with pytest.raises(AttributeError):
            setattr(run, name, value)


def test_without_upstream_gradients_there_is_no_backward(calls):
    run = R.QkRotary(SHAPE, I.make_qk_case(SHAPE, with_grad=False), device="cpu")
    with pytest.raises(ValueError, match="upstream"):
        run.backward()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_results_are_those_of_the_assigned_tensors(dtype):
    shape = dataclasses.replace(SHAPE, T=70, dtype=dtype)
    first, second = I.make_qk_case(shape, seed=1), I.make_qk_case(shape, seed=2)
    run = R.QkRotary(shape, first)
    run.step()
    case = dict(first)
    for name in INPUTS:  # one after the other
        new = second[name].cuda()
        setattr(run, name, _wide(new) if name in ("q", "k", "dqo", "dko") else new)
        case[name] = second[name]
        fresh = R.QkRotary(shape, case)
        run.step()
        fresh.step()
        assert all(torch.equal(getattr(run, n), getattr(fresh, n)) for n in OUTPUTS), name
    old = {n: getattr(run, n) for n in OUTPUTS}
    want = {n: t.clone() for n, t in old.items()}
    for n, t in old.items():
        t.zero_()
        setattr(run, n, torch.empty_like(t))
    run.ws = torch.empty_like(run.ws)
    run.step()
    assert all(torch.equal(getattr(run, n), want[n]) and not old[n].any() for n in OUTPUTS)


@pytest.mark.gpu
def test_in_place_by_assignment():
    case = I.make_qk_case(SHAPE, seed=4)
    want = R.QkRotary(SHAPE, case)
    want.step()
    run = R.QkRotary(SHAPE, {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in case.items()})
    run.dq, run.dk = run.dqo, run.dko
    run.backward()
    run.qo, run.ko = run.q, run.k
    run.forward()
    assert all(torch.equal(getattr(run, n), getattr(want, n)) for n in OUTPUTS)


BLOCK = I.BlockShape(1, 256, 2, 128, 344, 32, 48)
BLOCK_QK = I.QkShape(T=256, Hq=2, Hk=2, dh=128, rot=128, sec=(40, 24))
PAIRS = [f"{m}_{n}" for n in ("q", "k", "v", "o", "gate", "up", "down") for m in "AB"]


def _block_case(seed=0):
    case, qk = I.make_block_case(BLOCK, seed), I.make_qk_case(BLOCK_QK, seed, with_grad=False)
    return dict(case, **{n: qk[n] for n in ("gq", "gk", "pos", "freq")})


def _pointers(struct):
    """The pointers of a struct of pairs, in order."""
    out = []
    for name, _ in struct._fields_:
        v = getattr(struct, name)
        out += _pointers(v) if hasattr(v, "_fields_") else [v]
    return out


@pytest.fixture
def block_calls(monkeypatch):
    made = {}
    for name in ("lr_block_qk_fwd", "lr_block_qk_bwd"):
        monkeypatch.setattr(R.L, name, lambda *args, _name=name: made.__setitem__(_name, args))
    return made


@pytest.mark.parametrize("name", ["x", "pos", "gq", "gk", "g_attn", "g_mlp", "A_q", "B_o", "A_gate", "B_down"])
def test_the_block_reads_the_tensors_of_the_moment(block_calls, name):
    blk = R.TransformerBlock(BLOCK, _block_case(), device="cpu", qk=BLOCK_QK)
    blk.step()
    t = blk.t[name] = blk.t[name].clone()
    for renew in (False, True):
        if renew:
            t.data = t.data.clone()
        block_calls.clear()
        blk.step()
        for args in block_calls.values():
            x, w, qk = args[9], args[10], args[11]
            assert x is blk.t["x"]
            assert (qk.turns, qk.pos, qk.gq, qk.gk) == (blk.turns.data_ptr(), *(blk.t[n].data_ptr() for n in
                                                                               ("pos", "gq", "gk")))
            order = ["g_attn", *PAIRS[:8], "g_mlp", *PAIRS[8:]]
            assert _pointers(w) == [blk.t[n].data_ptr() for n in order]


def test_the_block_writes_the_gradients_of_the_moment(block_calls):
    blk = R.TransformerBlock(BLOCK, _block_case(), device="cpu", qk=BLOCK_QK)
    blk.step()
    for n in list(blk.grads):
        blk.grads[n] = torch.empty_like(blk.grads[n])
    blk.dg_attn, blk.dgq = torch.empty_like(blk.dg_attn), torch.empty_like(blk.dgq)
    blk.grads["dA_v"].data = torch.empty_like(blk.grads["dA_v"])
    blk.step()
    g, dgq = block_calls["lr_block_qk_bwd"][15], block_calls["lr_block_qk_bwd"][16]
    order = [blk.dg_attn, *(blk.grads["d" + n] for n in PAIRS[:8]), blk.dg_mlp, *(blk.grads["d" + n] for n in PAIRS[8:])]
    assert _pointers(g) == [t.data_ptr() for t in order] and dgq is blk.dgq


@pytest.mark.parametrize("name,bad", [
    ("pos", lambda t: t.long()), ("pos", lambda t: t[:1]), ("gq", lambda t: t[:64]), ("gk", lambda t: t.float()),
    ("A_q", lambda t: t[:8]), ("B_up", lambda t: t.float()), ("A_o", lambda t: t.repeat(1, 2)[:, ::2]),
    ("g_mlp", lambda t: t.to("meta")),
])
def test_the_block_refuses_what_does_not_fit(block_calls, name, bad):
    blk = R.TransformerBlock(BLOCK, _block_case(), device="cpu", qk=BLOCK_QK)
    old = blk.t[name]
    blk.step()
    block_calls.clear()
    blk.t[name] = bad(old)
    for call in (blk.forward, blk.backward):
        with pytest.raises(ValueError, match=name):
            call()
    assert not block_calls
    blk.t[name] = old
    blk.step()
    blk.grads["dA_k"] = blk.grads["dA_k"].bfloat16()
    with pytest.raises(ValueError, match="dA_k"):
        blk.backward()
    blk.grads["dA_k"] = blk.grads["dA_k"].float()
    blk.dgk = blk.dgk[:64]
    with pytest.raises(ValueError, match="dgk"):
        blk.backward()


@pytest.mark.gpu
def test_the_block_follows_new_positions_gains_weights_and_gradients():
    first, second = _block_case(1), _block_case(2)
    blk = R.TransformerBlock(BLOCK, first, qk=BLOCK_QK)
    blk.step()
    for n, v in second.items():
        if isinstance(v, torch.Tensor):
            blk.t[n] = v.cuda()
    blk.grads = {n: torch.zeros_like(g) for n, g in blk.grads.items()}
    blk.step()
    fresh = R.TransformerBlock(BLOCK, second, qk=BLOCK_QK)
    fresh.step()
    assert torch.equal(blk.out, fresh.out) and torch.equal(blk.dx, fresh.dx)
    assert all(torch.equal(a, b) for a, b in zip(blk.grad_tensors(), fresh.grad_tensors()))
    assert torch.equal(blk.clip_grads(0.5), fresh.clip_grads(0.5))
    assert all(torch.equal(a, b) for a, b in zip(blk.grad_tensors(), fresh.grad_tensors()))


def _packed(T, width, dtype=torch.bfloat16):
    m = torch.zeros(T, width, dtype=dtype)
    return lambda a, b: m[:, a:b]


@pytest.mark.parametrize("change", [
    lambda r: setattr(r, "qo", r.k.new_zeros(6, 96)) or setattr(r, "ko", r.qo[:, :64]),        # two outputs
    lambda r: setattr(r, "qo", r.dqo) or setattr(r, "dq", r.dqo) or setattr(r, "q", r.dqo),     # dq in q's place
    lambda r: setattr(r, "dgk", r.dgq),
    lambda r: setattr(r, "q", r.q[:1].expand(6, 96).clone()) or setattr(r, "ko", r.q[:, 8:72]),  # k's output in q
    lambda r: setattr(r, "ws", r.dq.view(torch.uint8).view(-1)),
    lambda r: setattr(r, "qo", torch.zeros(9, 96, dtype=torch.bfloat16)[3:]) or setattr(r, "q", r.qo._base[:6]),
    lambda r: (lambda at: setattr(r, "qo", at(0, 96)) or setattr(r, "ko", at(88, 152)))(_packed(6, 200)),
])
def test_outputs_that_overlap_are_refused(calls, change):
    run = R.QkRotary(SHAPE, I.make_qk_case(SHAPE), device="cpu")
    change(run)
    with pytest.raises(ValueError, match="overlap"):
        run.step()
    assert "lr_qk_bwd" not in calls


def test_outputs_beside_one_another_and_in_place_are_not(calls):
    run = R.QkRotary(SHAPE, I.make_qk_case(SHAPE), device="cpu")
    at, back = _packed(6, 200), _packed(6, 160)
    run.q, run.k, run.qo, run.ko = at(0, 96), at(96, 160), at(0, 96), at(96, 160)  # columns of one matrix, in place
    run.dqo, run.dko = back(64, 160), back(0, 64)
    run.dq, run.dk = run.dqo, run.dko
    run.step()
    run.k = run.q[:, :64]  # inputs may share memory ...
    run.ko = torch.zeros(6, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlap"):
        run.step()  # ... but not with an output
    run.qo = torch.zeros(6, 96, dtype=torch.bfloat16)
    run.step()
    run.k = torch.zeros(6, 64, dtype=torch.bfloat16)  # apart from q again
    run.gq = None
    run.dq = run.q  # not read by a backward without the norm
    run.backward()
    one = dataclasses.replace(SHAPE, T=1)
    run = R.QkRotary(one, I.make_qk_case(one), device="cpu")
    row = torch.zeros(1, 160, dtype=torch.bfloat16)
    run.q, run.qo, run.ko = row[:, :96], row[:, :96], row[:, 96:]
    run.step()
