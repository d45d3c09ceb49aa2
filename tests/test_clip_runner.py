"""clip_grads of the runners: the buffers it makes inside a call, on whatever stream the call names."""
import contextlib
import gc
import weakref

import numpy as np
import pytest
import torch

from rank_bottleneck_block_gb300 import runner as R


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_bottleneck_block_gb300 import build

    build.build()


class Holder(R._Clipped):
    def __init__(self, grads):
        self.tensors = list(grads)

    def grad_tensors(self):
        return list(self.tensors)


class Stream:
    """Stands in for a stream where there is no GPU."""

    cuda_stream = 1234


@pytest.fixture
def calls(monkeypatch):
    """Prepared calls that only note their name, arguments and stream."""
    made = []

    class Prepared:
        def __init__(self, *args):
            self.args = args

        def __call__(self, stream=None):
            made.append((self.args, stream))

    monkeypatch.setattr(R.L, "Prepared", Prepared)
    return made


def test_buffers_are_made_on_the_stream_of_the_call(monkeypatch, calls):
    """Memory that torch hands out, and anything it fills, is ordered after the work of torch's current stream; the
    kernels run on the stream of the call.  So that one has to be current while the buffers are made."""
    made, current = [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("empty", "zeros", "full", "ones"):
        def make(*args, _real=getattr(torch, name), **kw):
            made.append(current[-1] if current else None)
            return _real(*args, **kw)

        monkeypatch.setattr(torch, name, make)
    side, first, second = Stream(), torch.randn(64), torch.randn(32)
    h = Holder([first])
    h.clip_grads(1.0, stream=side)
    assert made and all(s is side for s in made)
    h.tensors = [second] + [torch.randn(8) for _ in range(1100)]  # another list, and a longer workspace
    made.clear()
    h.clip_grads(1.0, stream=side)
    assert all(s is side for s in made)
    assert [s for _, s in calls] == [side, side]
    made.clear()
    Holder([first]).clip_grads(1.0)
    assert made and all(s is None for s in made)


@pytest.mark.parametrize("handle,want", [(1234, ("external", 1234)), (0, "default")])
def test_a_handle_of_a_stream_serves_too(monkeypatch, calls, handle, want):
    """0 is the default stream: torch would make a new stream of it."""
    seen = []

    @contextlib.contextmanager
    def stream(s):
        seen.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    Holder([torch.randn(64)]).clip_grads(1.0, stream=handle)
    assert seen == [want] and calls[0][1] == handle


def test_buffers_stay_when_gradients_are_replaced(calls):
    """A graph that was captured before, or a stream that still runs, goes on writing where it did."""
    h = Holder([torch.randn(64), torch.randn(8)])
    norm = h.clip_grads(1.0)
    ws = h._clip.ws
    h.tensors[0] = torch.randn(64)
    assert h.clip_grads(1.0).data_ptr() == norm.data_ptr() and h._clip.ws.data_ptr() == ws.data_ptr()
    kept = weakref.ref(ws)
    del ws
    h.tensors = [torch.randn(8) for _ in range(1100)]
    assert h.clip_grads(1.0).data_ptr() == norm.data_ptr()
    calls.clear()
    assert kept() is not None and h._clip.ws.numel() > kept().numel()


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_the_first_clip_on_a_side_stream_beside_a_busy_one(handle):
    """The current stream is busy for some 20 ms when the first clip runs on another stream, and when a replaced
    gradient makes it look its list up again.  More than 512 partial sums: three launches, which leave the scale in
    memory between the last two."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in (2100 * 8192, 77)]
    h, side = Holder(grads), torch.cuda.Stream()
    a = torch.randn(8192, 8192, generator=gen, device="cuda").bfloat16()
    b = torch.empty_like(a)
    for again in (False, True):
        if again:
            h.tensors[1] = torch.randn(99, generator=gen, device="cuda")
        keep = [g.clone() for g in h.tensors]
        norm = float(torch.stack([g.double().square().sum() for g in keep]).sum().sqrt())
        torch.cuda.synchronize()
        for _ in range(30):
            torch.matmul(a, a, out=b)
        got = h.clip_grads(1.0, side.cuda_stream if handle else side)
        for wait in (side.synchronize, torch.cuda.synchronize):  # before and after the busy stream has ended
            wait()
            with torch.cuda.stream(side):
                # 34 roundings in the norm, 38 in the scale, one in the product (as for the kernels' own tests)
                assert abs(float(got) - norm) <= 34 * 2.0 ** -24 * norm
                assert abs(float(h._clip.scale) * (norm + 1e-6) - 1.0) <= 38 * 2.0 ** -24
                for g, k in zip(h.tensors, keep):
                    want = k.double() / (norm + 1e-6)
                    assert ((g.double() - want).abs() <= 41 * 2.0 ** -24 * want.abs() + 1e-40).all()


def _last(calls):
    """(pointers of the gradients, of the outputs, element counts) of the newest prepared clip."""
    name, _, n, grads, counts, _, outs = calls[-1][0][:7]
    assert name == "lr_grad_clip" and len(grads) == len(outs) == len(counts) == n
    return list(grads), list(outs), list(counts)


def _as_list(tensors):
    return [t.data_ptr() for t in tensors], [t.data_ptr() for t in tensors], [t.numel() for t in tensors]


def _like(ts, n):
    return torch.randn(n, device=ts[0].device)


CHANGES = {
    "added": lambda ts: ts.append(_like(ts, 24)),
    "lost": lambda ts: ts.pop(),
    "inserted": lambda ts: ts.insert(0, _like(ts, 4)),
    "replaced": lambda ts: ts.__setitem__(1, _like(ts, 40)),
    "reordered": lambda ts: ts.reverse(),
    "new memory": lambda ts: setattr(ts[0], "data", _like(ts, 64)),
    "other size": lambda ts: setattr(ts[0], "data", _like(ts, 48)),
    "shorter, same memory": lambda ts: setattr(ts[0], "data", ts[0].data[:32]),
    "set": lambda ts: ts[2].set_(_like(ts, 16)),
}


@pytest.mark.parametrize("change", CHANGES)
def test_clipping_takes_the_gradients_of_the_moment(calls, change):
    h = Holder([torch.randn(n) for n in (64, 40, 16)])
    h.clip_grads(1.0)
    assert _last(calls) == _as_list(h.tensors)
    CHANGES[change](h.tensors)
    h.clip_grads(1.0)
    assert _last(calls) == _as_list(h.tensors)


@pytest.mark.parametrize("bad", [torch.randn(64).bfloat16(), torch.randn(8, 8).T, torch.randn(128)[::2]])
def test_a_gradient_that_cannot_be_clipped_any_more_is_refused(calls, bad):
    h = Holder([torch.randn(64), torch.randn(8)])
    h.clip_grads(1.0)
    h.tensors[0].data = bad
    for _ in range(2):
        with pytest.raises(ValueError):
            h.clip_grads(1.0)
    h.tensors[0].data = torch.randn(64)
    h.clip_grads(1.0)
    assert _last(calls) == _as_list(h.tensors)


def test_a_list_is_fixed_and_its_memory_stays(calls):
    """A GradClip of the caller's own works on the memory that it was given, which lives as long as it does."""
    memory = np.zeros(64, dtype=np.float32)
    kept = weakref.ref(memory)
    grads = [torch.from_numpy(memory), torch.randn(8)]
    del memory
    clip = R.GradClip(grads, outs=[torch.empty(64), torch.empty(8)])
    before = clip.grads[0].data_ptr()
    grads[0].data = torch.randn(64)
    grads.append(torch.randn(4))
    gc.collect()
    assert kept() is not None and len(clip.grads) == 2
    clip.clip()
    assert _last(calls)[0][0] == before
    for name in ("grads", "outs", "stat", "norm", "scale"):
        with pytest.raises(AttributeError):
            setattr(clip, name, getattr(clip, name))
    for change in (lambda ts: ts.__setitem__(0, grads[0]), lambda ts: ts.append(grads[0]), lambda ts: ts.pop(),
                   lambda ts: ts.clear(), lambda ts: ts.__delitem__(0), lambda ts: ts.reverse()):
        for ts in (clip.grads, clip.outs):
            with pytest.raises(TypeError):
                change(ts)
    del clip, calls[:]
    gc.collect()
    assert kept() is None


def test_buffers_of_a_prepared_call_stay(monkeypatch):
    """A call that has been prepared keeps the memory whose addresses it holds."""
    memory = np.zeros(64, dtype=np.float32)
    kept = weakref.ref(memory)
    ws = torch.from_numpy(memory)
    del memory
    call = R.L.Prepared("lr_grad_norm", R.L.LR_F32, 0, None, None, torch.zeros(4), ws, 256)
    ws.data = torch.zeros(64)
    gc.collect()
    assert kept() is not None
    del call
    gc.collect()
    assert kept() is None


@pytest.mark.gpu
@pytest.mark.parametrize("change", CHANGES)
def test_what_changed_is_clipped_on_the_gpu(change):
    h = Holder([torch.randn(n).cuda() for n in (64, 40, 16)])
    h.clip_grads(1.0)
    CHANGES[change](h.tensors)
    for i, t in enumerate(h.tensors):
        t.copy_(torch.arange(t.numel()) + i)
    keep = [t.double() for t in h.tensors]
    norm = float(torch.cat(keep).square().sum().sqrt())
    assert abs(float(h.clip_grads(1.0)) - norm) <= 34 * 2.0 ** -24 * norm
    for t, k in zip(h.tensors, keep):
        assert ((t.double() - k / (norm + 1e-6)).abs() <= 41 * 2.0 ** -24 * k / norm + 1e-40).all()


@pytest.mark.gpu
def test_the_default_streams_handle():
    h, side = Holder([torch.arange(64.0).cuda()]), torch.cuda.Stream()
    norm = float(h.tensors[0].norm())
    torch.cuda.synchronize()
    seen = []
    with torch.cuda.stream(side):
        with R._current(0):
            seen.append(torch.cuda.current_stream().cuda_stream)
        with R._current(side.cuda_stream):
            seen.append(torch.cuda.current_stream().cuda_stream)
        got = h.clip_grads(1.0, stream=0)
    torch.cuda.synchronize()
    assert seen == [0, side.cuda_stream] and float(got) == pytest.approx(norm, rel=1e-6)
