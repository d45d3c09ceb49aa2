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
