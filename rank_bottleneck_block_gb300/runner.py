"""Device-buffer plumbing around the C ABI for one MLP block, one projection
group, one block stack, attention with the norm and rotation of its queries and
keys, one transformer block, and the clipping of their gradients.

torch only allocates device memory and supplies the stream; every computation
is a call into liblowrank.so through the ctypes binding.
"""
from __future__ import annotations

import contextlib
import operator
from typing import Dict, List, Optional, Sequence

import torch

from . import lowrank as L
from .inputs import MlpShape, ProjShape, QkShape

_U8 = torch.uint8


def _dt(name: str) -> int:
    return L.LR_BF16 if name == "bf16" else L.LR_F32


def _tdt(name: str) -> torch.dtype:
    return torch.bfloat16 if name == "bf16" else torch.float32


def _buf(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=_U8, device=device)


def _current(stream):
    """Makes the stream that a call names (None: the current one) torch's current stream: torch hands memory out in the
    order of that stream's work."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):  # a handle; torch makes a new stream of handle 0, the default one's
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


_READ = (torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous, operator.attrgetter("dtype"))


def _facts(tensors):
    """What a converted list of tensors rests on."""
    return [list(map(f, tensors)) for f in _READ]


class _FixedList(list):
    """A list whose elements a prepared call has converted: changing it would change nothing."""

    def _refuse(self, *args, **kw):
        raise TypeError("the list is fixed")

    __setitem__ = __delitem__ = __iadd__ = __imul__ = _refuse
    append = extend = insert = pop = remove = clear = sort = reverse = _refuse


class GradClip:
    """The norm over a list of gradient tensors, and the tensors scaled to at most max_norm.

    grads: contiguous tensors of one type (fp32 as the backward passes write them, or bf16) on one
    device, 16-byte aligned; outs: where the scaled tensors go (None: in place).  measure() leaves the
    norm in self.norm [1]; clip() leaves it there, min(1, max_norm / (norm + 1e-6)) in self.scale [1]
    and the scaled gradients in outs (all of them unset before).  Device tensors: nothing waits for the
    GPU.  stream: the one for which the results' and the workspace's memory is made (None: the current one);
    calls on others are to be ordered after it, and the object kept until they have ended.

    The lists are fixed.  Calls work on the memory that the tensors have when the object is made, and keep it
    alive: new gradients are written into it, and tensors that have been given other memory need an object of
    their own (the runners' clip_grads sees to that).  ws may be replaced, by one that several objects share.
    """

    def __init__(self, grads: Sequence[torch.Tensor], max_norm: float = 1.0,
                 outs: Optional[Sequence[torch.Tensor]] = None, stream=None):
        self.max_norm = float(max_norm)
        self._stat = self.ws = None
        self._retired = []  # buffers that graphs captured before may still write to
        self._bind(grads, outs, stream)

    grads = property(lambda self: self._grads)
    outs = property(lambda self: self._outs)
    stat = property(lambda self: self._stat)  # norm and scale
    norm = property(lambda self: self._norm)
    scale = property(lambda self: self._scale)

    def _bind(self, grads, outs=None, stream=None):
        """Takes a list of tensors; the results and, where it is long enough, the workspace stay where they are."""
        grads = _FixedList(grads)
        to_tensors = grads if outs is None else _FixedList(outs)
        if not grads:
            raise ValueError("no gradients")
        if len(to_tensors) != len(grads):
            raise ValueError(f"{len(grads)} gradients but {len(to_tensors)} outputs")
        first = grads[0]
        dt, es = L.dtype_code(first), first.element_size()
        for t in grads if outs is None else grads + to_tensors:
            if t.dtype != first.dtype or t.device != first.device or not t.is_contiguous():
                raise ValueError("gradients and outputs must be contiguous, of one type and on one device")
        n = [t.numel() for t in grads]
        to = at = [t.data_ptr() for t in grads]
        if outs is not None:
            to = [t.data_ptr() for t in to_tensors]
            if [t.numel() for t in to_tensors] != n:
                raise ValueError("an output has another number of elements than its gradient")
        # a written tensor is its own gradient, or overlaps nothing else of either list
        spans = [(o, o + k * es, 1) for o, k in zip(to, n) if k]
        spans += [(g, g + k * es, 0) for g, o, k in zip(at, to, n) if k and g != o]
        end = written = 0  # the furthest end so far, of any span and of a written one
        for lo, hi, w in sorted(spans):
            if lo < (end if w else written):
                raise ValueError("an output overlaps another output or another gradient")
            end, written = max(end, hi), max(written, hi if w else 0)
        size, stat, ws = L.lr_grad_workspace_bytes(len(grads)), self._stat, self.ws
        with _current(stream):
            if stat is None or stat.device != first.device:
                stat = torch.empty(2, dtype=torch.float32, device=first.device)
            if ws is None or ws.device != first.device or ws.numel() < size:
                ws = _buf(size, first.device)
        self._retired += [b for b, now in ((self._stat, stat), (self.ws, ws)) if b is not None and b is not now]
        self._grads, self._outs, self.dt = grads, to_tensors, dt
        # aliases keep the memory alive when a tensor is given other memory
        self._held = [t.detach() for t in (grads if outs is None else grads + to_tensors)]
        self._facts = _facts(grads)
        self._g, self._n = L.tensor_list(at, n)
        self._o = self._g if outs is None else L.tensor_list(to, n)[0]
        self._stat, self.ws = stat, ws
        self._norm, self._scale = stat[:1], stat[1:]
        self._measure = self._clip = None  # the last calls' arguments, converted

    def measure(self, stream=None) -> torch.Tensor:
        if self._measure is None or self._measure[0] is not self.ws:
            self._measure = (self.ws, L.Prepared("lr_grad_norm", self.dt, len(self._grads), self._g, self._n, self._stat,
                                                 self.ws, L._nbytes(self.ws)))
        self._measure[1](stream)
        return self._norm

    def clip(self, stream=None) -> torch.Tensor:
        made = self._clip
        if made is None or made[0] is not self.ws or made[1] != self.max_norm:
            made = self._clip = (self.ws, self.max_norm, L.Prepared(
                "lr_grad_clip", self.dt, len(self._grads), self._g, self._n, self.max_norm, self._o, self._stat, self.ws,
                L._nbytes(self.ws)))
        made[2](stream)
        return self._norm


class _Clipped:
    """clip_grads for the runners that hold gradients (they list them in grad_tensors)."""

    _clip: Optional[GradClip] = None

    def clip_grads(self, max_norm: float, stream=None) -> torch.Tensor:
        """Scale every gradient in place so that their common norm is at most max_norm; the norm [1]."""
        grads = self.grad_tensors()
        if self._clip is None:
            self._clip = GradClip(grads, stream=stream)
        elif _facts(grads) != self._clip._facts:  # the held memory makes equal addresses the same memory
            self._clip._bind(grads, stream=stream)
        self._clip.max_norm = float(max_norm)
        return self._clip.clip(stream)


class MlpBlock(_Clipped):
    """One low-rank SwiGLU MLP block resident on the device (weights, saved set, workspaces, grads)."""

    def __init__(self, shape: MlpShape, case: Dict[str, torch.Tensor], mode: int = L.LR_SAVE_CKPT,
                 device="cuda", act: int = L.LR_ACT_SILU):
        self.s, self.mode, self.device, self.act = shape, mode, device, act
        self.dt = _dt(shape.dtype)
        dev = {k: v.to(device) for k, v in case.items()}
        self.t = dev
        T, d, f, r = shape.T, shape.d, shape.f, shape.r
        self.out = torch.empty(T, d, dtype=_tdt(shape.dtype), device=device)
        self.dx = torch.empty_like(self.out)
        self.saved = _buf(L.lr_mlp_saved_bytes(self.dt, mode, T, d, f, r), device)
        self.ws_f = _buf(L.lr_mlp_fwd_workspace_bytes(self.dt, mode, T, d, f, r), device)
        self.ws_b = _buf(L.lr_mlp_bwd_workspace_bytes(self.dt, mode, T, d, f, r), device)
        f32 = dict(dtype=torch.float32, device=device)
        self.dg = torch.empty(d, **f32)
        self.grads = {}
        for k, (ri, co) in {"gate": (r, d), "up": (r, d), "down": (r, f)}.items():
            do = f if k != "down" else d
            self.grads[f"dA_{k}"] = torch.empty(ri, co, **f32)
            self.grads[f"dB_{k}"] = torch.empty(do, r, **f32)

    def pairs(self):
        t = self.t
        return (L.pair(t["A_gate"], t["B_gate"]), L.pair(t["A_up"], t["B_up"]), L.pair(t["A_down"], t["B_down"]))

    def forward(self, x: Optional[torch.Tensor] = None, stream=None, out: Optional[torch.Tensor] = None):
        s = self.s
        x = self.t["x"] if x is None else x
        out = self.out if out is None else out
        L.lr_mlp_fwd(self.dt, self.mode, s.T, s.d, s.f, s.r, s.eps, x, self.t["g"], *self.pairs(), out,
                     self.saved, self.ws_f, stream, act=self.act)
        return out

    def backward(self, dout: Optional[torch.Tensor] = None, x: Optional[torch.Tensor] = None, stream=None,
                 dx: Optional[torch.Tensor] = None):
        s, gr = self.s, self.grads
        x = self.t["x"] if x is None else x
        dout = self.t["G"] if dout is None else dout
        dx = self.dx if dx is None else dx
        L.lr_mlp_bwd(self.dt, self.mode, s.T, s.d, s.f, s.r, s.eps, x, self.t["g"], *self.pairs(), self.saved, dout,
                     dx, self.dg, L.pair_grad(gr["dA_gate"], gr["dB_gate"]),
                     L.pair_grad(gr["dA_up"], gr["dB_up"]), L.pair_grad(gr["dA_down"], gr["dB_down"]), self.ws_b,
                     stream, act=self.act)
        return dx

    def step(self, stream=None):
        self.forward(stream=stream)
        self.backward(stream=stream)

    def grad_tensors(self):
        return [self.dg, *self.grads.values()]


class DenseBlock(_Clipped):
    """The full-rank SwiGLU MLP block of the same d, f, resident on the device: the reference point
    the low-rank block is compared with."""

    def __init__(self, shape: MlpShape, case: Dict[str, torch.Tensor], device="cuda"):
        self.s, self.device = shape, device
        self.dt = _dt(shape.dtype)
        self.t = {k: v.to(device) for k, v in case.items()}
        T, d, f = shape.T, shape.d, shape.f
        self.out = torch.empty(T, d, dtype=_tdt(shape.dtype), device=device)
        self.dx = torch.empty_like(self.out)
        self.saved = _buf(L.lr_dense_saved_bytes(self.dt, T, d, f), device)
        self.ws_f = _buf(L.lr_dense_fwd_workspace_bytes(self.dt, T, d, f), device)
        self.ws_b = _buf(L.lr_dense_bwd_workspace_bytes(self.dt, T, d, f), device)
        f32 = dict(dtype=torch.float32, device=device)
        self.dg = torch.empty(d, **f32)
        self.grads = {"dW_gate": torch.empty(f, d, **f32), "dW_up": torch.empty(f, d, **f32),
                      "dW_down": torch.empty(d, f, **f32)}

    def forward(self, x: Optional[torch.Tensor] = None, stream=None):
        s, t = self.s, self.t
        x = t["x"] if x is None else x
        L.lr_dense_fwd(self.dt, s.T, s.d, s.f, s.eps, x, t["g"], t["W_gate"], t["W_up"], t["W_down"], self.out,
                       self.saved, self.ws_f, stream)
        return self.out

    def backward(self, dout: Optional[torch.Tensor] = None, x: Optional[torch.Tensor] = None, stream=None):
        s, t, gr = self.s, self.t, self.grads
        x = t["x"] if x is None else x
        dout = t["G"] if dout is None else dout
        L.lr_dense_bwd(self.dt, s.T, s.d, s.f, s.eps, x, t["g"], t["W_gate"], t["W_up"], t["W_down"], self.saved,
                       dout, self.dx, self.dg, gr["dW_gate"], gr["dW_up"], gr["dW_down"], self.ws_b, stream)
        return self.dx

    def step(self, stream=None):
        self.forward(stream=stream)
        self.backward(stream=stream)

    def grad_tensors(self):
        return [self.dg, *self.grads.values()]


class HostPipeline:
    """fwd + bwd of an MlpBlock over batches that live in (pinned) host memory.

    Step i copies x_i and dout_i to the device on a copy stream, runs the block on the
    compute stream and copies out_i and dx_i back on a second copy stream; with two device
    buffer sets the copies of steps i+1 and i-1 overlap the compute of step i.
    """

    def __init__(self, blk: MlpBlock):
        self.blk = blk
        s, dev = blk.s, blk.device
        td = _tdt(s.dtype)
        self.x = [torch.empty(s.T, s.d, dtype=td, device=dev) for _ in range(2)]
        self.G = [torch.empty(s.T, s.d, dtype=td, device=dev) for _ in range(2)]
        self.out = [torch.empty(s.T, s.d, dtype=td, device=dev) for _ in range(2)]
        self.dx = [torch.empty(s.T, s.d, dtype=td, device=dev) for _ in range(2)]
        self.h2d = torch.cuda.Stream(device=dev)
        self.d2h = torch.cuda.Stream(device=dev)
        self.ev_in = [torch.cuda.Event() for _ in range(2)]    # inputs of the set copied in
        self.ev_done = [torch.cuda.Event() for _ in range(2)]  # compute of the set finished
        self.ev_read = [torch.cuda.Event() for _ in range(2)]  # results of the set copied out

    def bytes_per_step(self):
        e = self.x[0].element_size() * self.x[0].numel()
        return 2 * e, 2 * e  # (host -> device: x, dout), (device -> host: out, dx)

    def run(self, xh: List[torch.Tensor], gh: List[torch.Tensor], outh: torch.Tensor, dxh: torch.Tensor,
            steps: int, stream=None):
        """Runs `steps` steps on batches xh[i % len], gh[i % len]; results land in outh, dxh."""
        blk = self.blk
        comp = stream if stream is not None else torch.cuda.current_stream(blk.device)
        self.h2d.wait_stream(comp)
        self.d2h.wait_stream(comp)
        for i in range(steps):
            b = i % 2
            with torch.cuda.stream(self.h2d):
                if i >= 2:
                    self.h2d.wait_event(self.ev_done[b])  # step i-2 no longer reads this input set
                self.x[b].copy_(xh[i % len(xh)], non_blocking=True)
                self.G[b].copy_(gh[i % len(gh)], non_blocking=True)
                self.ev_in[b].record(self.h2d)
            comp.wait_event(self.ev_in[b])
            if i >= 2:
                comp.wait_event(self.ev_read[b])  # step i-2's results have been copied out of this set
            blk.forward(self.x[b], stream=comp.cuda_stream, out=self.out[b])
            blk.backward(self.G[b], self.x[b], stream=comp.cuda_stream, dx=self.dx[b])
            self.ev_done[b].record(comp)
            with torch.cuda.stream(self.d2h):
                self.d2h.wait_event(self.ev_done[b])
                outh.copy_(self.out[b], non_blocking=True)
                dxh.copy_(self.dx[b], non_blocking=True)
                self.ev_read[b].record(self.d2h)
        comp.wait_stream(self.d2h)
        comp.wait_stream(self.h2d)


class ProjGroup(_Clipped):
    """A group of low-rank pairs sharing one input, optionally behind an RMSNorm."""

    def __init__(self, shape: ProjShape, case: Dict[str, object], device="cuda", act: int = L.LR_ACT_SILU):
        self.s, self.device, self.act = shape, device, act
        self.dt = _dt(shape.dtype)
        s = shape
        self.x = case["x"].to(device)
        self.g = case["g"].to(device) if case["g"] is not None else None
        self.A = [a.to(device) for a in case["A"]]
        self.B = [b.to(device) for b in case["B"]]
        self.G = [gg.to(device) for gg in case["G"]] if "G" in case else None
        td = _tdt(s.dtype)
        self.outs = [torch.empty(s.T, s.d_out, dtype=td, device=device) for _ in range(s.group)]
        self.dx = torch.empty(s.T, s.d_in, dtype=td, device=device)
        norm = self.g is not None
        self.saved = _buf(L.lr_proj_saved_bytes(self.dt, s.T, s.d_in, s.d_out, s.r, s.group, norm), device)
        self.ws_f = _buf(L.lr_proj_fwd_workspace_bytes(self.dt, s.T, s.d_in, s.d_out, s.r, s.group, norm), device)
        self.ws_b = _buf(L.lr_proj_bwd_workspace_bytes(self.dt, s.T, s.d_in, s.d_out, s.r, s.group, norm), device)
        f32 = dict(dtype=torch.float32, device=device)
        self.dg = torch.empty(s.d_in, **f32) if norm else None
        self.dA = [torch.empty(s.r, s.d_in, **f32) for _ in range(s.group)]
        self.dB = [torch.empty(s.d_out, s.r, **f32) for _ in range(s.group)]

    def pairs(self):
        return [L.pair(a, b) for a, b in zip(self.A, self.B)]

    def forward(self, stream=None):
        s = self.s
        L.lr_proj_fwd(self.dt, s.T, s.d_in, s.d_out, s.r, self.pairs(), self.g, s.eps, self.x, self.outs, self.saved,
                      self.ws_f, stream, act=self.act)
        return self.outs

    def backward(self, stream=None):
        s = self.s
        L.lr_proj_bwd(self.dt, s.T, s.d_in, s.d_out, s.r, self.pairs(), self.g, s.eps, self.x, self.saved, self.G,
                      self.dx, self.dg, [L.pair_grad(a, b) for a, b in zip(self.dA, self.dB)], self.ws_b, stream,
                      act=self.act)
        return self.dx

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    def grad_tensors(self):
        return [t for t in (self.dg, *self.dA, *self.dB) if t is not None]


class BlockStack(_Clipped):
    """A residual stack of MLP blocks trained with an MSE loss (one call per step)."""

    def __init__(self, shape: MlpShape, case: Dict[str, object], mode: int = L.LR_SAVE_CKPT, device="cuda"):
        self.s, self.mode, self.device = shape, mode, device
        self.dt = _dt(shape.dtype)
        s = shape
        self.x = case["x"].to(device)
        self.target = case["target"].to(device)
        self.blocks: List[Dict[str, torch.Tensor]] = [{k: v.to(device) for k, v in b.items()}
                                                      for b in case["blocks"]]
        n = len(self.blocks)
        self.ws = _buf(L.lr_stack_workspace_bytes(self.dt, mode, n, s.T, s.d, s.f, s.r), device)
        f32 = dict(dtype=torch.float32, device=device)
        self.loss = torch.zeros(1, **f32)
        self.dx = torch.empty(s.T, s.d, dtype=_tdt(s.dtype), device=device)
        self.dgs = [torch.empty(s.d, **f32) for _ in range(n)]
        self.grads = []
        for _ in range(n):
            gr = {}
            for k, (ri, co, do) in {"gate": (s.r, s.d, s.f), "up": (s.r, s.d, s.f), "down": (s.r, s.f, s.d)}.items():
                gr[f"dA_{k}"] = torch.empty(ri, co, **f32)
                gr[f"dB_{k}"] = torch.empty(do, s.r, **f32)
            self.grads.append(gr)

    def step(self, stream=None):
        s = self.s
        pairs, grads = [], []
        for b, gr in zip(self.blocks, self.grads):
            for k in ("gate", "up", "down"):
                pairs.append(L.pair(b[f"A_{k}"], b[f"B_{k}"]))
                grads.append(L.pair_grad(gr[f"dA_{k}"], gr[f"dB_{k}"]))
        L.lr_stack_step(self.dt, self.mode, s.T, s.d, s.f, s.r, s.eps, self.x, self.target,
                        [b["g"] for b in self.blocks], pairs, self.loss, self.dx, self.dgs, grads, self.ws, stream)
        return self.loss

    def grad_tensors(self):
        return [*self.dgs, *(t for gr in self.grads for t in gr.values())]


class GraphStep:
    """A step captured once as a CUDA graph and replayed with one launch.

    `fn` enqueues the step on torch's current stream (every runner above does when given no
    stream).  Capture records its launches, programmatic-launch edges included, with their
    arguments: the buffers the step reads and writes must stay where they are, and new inputs
    are copied into them.  Replaying removes the host cost of issuing each launch, which bounds
    steps of a few tens of microseconds.
    """

    def __init__(self, fn, warmup: int = 2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # first launches (kernel attributes, caches) outside the capture
            for _ in range(warmup):
                fn()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            fn()

    def __call__(self) -> None:
        self.graph.replay()


class Attention:
    """Causal multi-head self-attention between the projection groups, resident on the device.

    q, k, v [b*s, H*dh] bf16 (token-major, as the projections write them); forward() writes o
    and keeps the row log-sum-exp; backward() takes dout and writes dq, dk, dv.
    """

    def __init__(self, b: int, s: int, H: int, dh: int, q, k, v, device="cuda", scale: Optional[float] = None):
        self.b, self.s, self.H, self.dh = b, s, H, dh
        self.scale = float(scale if scale is not None else dh ** -0.5)
        self.q, self.k, self.v = (t.to(device=device, dtype=torch.bfloat16).contiguous() for t in (q, k, v))
        self.o = torch.empty_like(self.q)
        self.dq, self.dk, self.dv = (torch.empty_like(self.q) for _ in range(3))
        self.dout = torch.empty_like(self.q)
        self.saved = _buf(L.lr_attn_saved_bytes(b, s, H, dh), device)
        self.ws = _buf(L.lr_attn_workspace_bytes(b, s, H, dh), device)

    def forward(self, stream=None):
        L.lr_attn_fwd(L.LR_BF16, self.b, self.s, self.H, self.dh, self.scale, self.q, self.k, self.v, self.o,
                      self.saved, self.ws, stream)

    def backward(self, dout: Optional[torch.Tensor] = None, stream=None):
        if dout is not None:
            self.dout.copy_(dout)
        L.lr_attn_bwd(L.LR_BF16, self.b, self.s, self.H, self.dh, self.scale, self.q, self.k, self.v, self.o,
                      self.saved, self.dout, self.dq, self.dk, self.dv, self.ws, stream)

    def step(self, stream=None):
        self.forward(stream)
        self.backward(None, stream)


def _qk_shape(s: QkShape) -> L.lr_qk_shape:
    layouts = {"half": L.LR_PAIR_HALF, "pairs": L.LR_PAIR_ADJACENT}
    return L.qk_shape(s.Hq, s.Hk, s.dh, s.rot, s.sec, layouts[s.layout], s.seq)


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors with contiguous rows share an element."""

    def span(t):  # address, bytes of a row, bytes from row to row, bytes in all
        row = t.shape[-1] * t.element_size()
        if t.dim() < 2 or t.shape[0] < 2:
            return t.data_ptr(), row, 0, row
        step = t.stride(0) * t.element_size()
        return t.data_ptr(), row, step, (t.shape[0] - 1) * step + row

    if not a.numel() or not b.numel():
        return False
    (pa, ra, sa, na), (pb, rb, sb, nb) = span(a), span(b)
    if pa + na <= pb or pb + nb <= pa:
        return False
    if sa != sb or sa == 0:
        return True
    return (pb - pa) % sa < ra or (pa - pb) % sa < rb  # columns of one matrix


class QkRotary:
    """Norm and position rotation of queries and keys between their projections and attention.

    case: q [T, Hq*dh], k [T, Hk*dh] (rows may be further apart: columns of a packed matrix; None with 0
    heads), gq, gk [dh] (None: no norm), pos int32 [axes, T] (None: position t mod shape.seq), freq (the
    rot / 2 frequencies in radians per position) and, for backward(), dqo, dko.  forward() writes qo, ko;
    backward() writes dq, dk and, with the norm, dgq, dgk [dh] fp32.

    The tensors are attributes, and may be replaced by others of their size and type on the same device, 16-byte
    aligned (run.q = ..., run.qo = run.q for a forward in place).  The calls' arguments are converted once for
    each assignment: a tensor that is given other memory by other means is to be assigned again.  An output may take
    the place of its own input (qo of q, ko of k, dq of dqo, dk of dko) and overlaps no other tensor of its call.  The
    shape is fixed.
    """

    _FORWARD = ("turns", "pos", "gq", "gk", "q", "k", "qo", "ko")
    _BACKWARD = ("turns", "pos", "gq", "gk", "q", "k", "dqo", "dko", "dq", "dk", "dgq", "dgk", "ws")
    _TENSORS = frozenset(_FORWARD + _BACKWARD)

    def __init__(self, shape: QkShape, case: Dict[str, object], device="cuda"):
        self.s, self.dt, self.sh = shape, _dt(shape.dtype), _qk_shape(shape)
        s, td, f32 = shape, _tdt(shape.dtype), torch.float32
        q, k, g = (s.T, s.Hq * s.dh), (s.T, s.Hk * s.dh), (s.dh,)
        self._fits = {"turns": ((s.rot // 2,), torch.int64), "pos": ((len(s.sec), s.T), torch.int32), "gq": (g, td),
                      "gk": (g, td), "dgq": (g, f32), "dgk": (g, f32), "ws": (None, _U8),
                      **{n: (q, td) for n in ("q", "qo", "dqo", "dq")}, **{n: (k, td) for n in ("k", "ko", "dko", "dk")}}
        if len(case["freq"]) != s.rot // 2:
            raise ValueError(f"{len(case['freq'])} frequencies for {s.rot // 2} pairs")
        turns = L.turns_tensor(case["freq"], device)
        self._device = turns.device
        self.turns = turns
        for n in ("pos", "q", "k", "gq", "gk", "dqo", "dko"):
            t = case.get(n)
            setattr(self, n, None if t is None else self._fit(n, t).to(device))

        def fresh(H, wanted=True):
            return torch.empty(s.T, H * s.dh, dtype=td, device=device) if H and wanted else None

        self.qo, self.ko = fresh(s.Hq), fresh(s.Hk)
        back = self.dqo is not None or self.dko is not None
        self.dq, self.dk = fresh(s.Hq, back), fresh(s.Hk, back)
        self.dgq = torch.empty(s.dh, dtype=f32, device=device) if back and s.Hq and self.gq is not None else None
        self.dgk = torch.empty(s.dh, dtype=f32, device=device) if back and s.Hk and self.gk is not None else None
        self.ws = _buf(L.lr_qk_bwd_workspace_bytes(self.dt, s.T, self.sh), device) if back else None
        self._convert_forward()
        if back:
            self._convert_backward()

    def __setattr__(self, name, value):
        if name in self._TENSORS:
            if value is not None and self._fit(name, value).device != self._device:
                raise ValueError(f"{name}: a tensor on {self._device} needed, not on {value.device}")
            self.__dict__.update(_fwd=None, _bwd=None)
        elif name in ("s", "dt", "sh") and name in self.__dict__:
            raise AttributeError(f"{name} is fixed")
        object.__setattr__(self, name, value)

    def _fit(self, name, t):
        size, dtype = self._fits[name]
        if (size is not None and tuple(t.shape) != size) or t.dtype != dtype or (t.numel() and t.stride(-1) != 1):
            raise ValueError(f"{name}: {'' if size is None else list(size)} {dtype} with contiguous rows needed, not "
                             f"{list(t.shape)} {t.dtype} with strides {t.stride()}")
        if name in ("pos", "ws") and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t

    def _rows(self, *names):
        """Each tensor and its row distance."""
        for n in names:
            t = getattr(self, n)
            yield t
            yield 0 if t is None else t.stride(0) if self.s.T > 1 else t.shape[1]

    def _common(self):
        return (self.dt, self.s.T, L.ctypes.pointer(self.sh), self.s.eps, self.turns, self.pos, self.gq, self.gk,
                *self._rows("q", "k"))

    def _apart(self, names, outputs):
        """Refuses outputs that overlap one another or an input of their call."""
        tensors = {n: t for n in names if (t := getattr(self, n)) is not None}
        own = {"qo": "q", "ko": "k", "dq": "dqo", "dk": "dko"}
        for o, out in ((o, tensors[o]) for o in outputs if o in tensors):
            for n, t in tensors.items():
                if n == o or not _overlap(out, t):
                    continue
                if n == own.get(o) and out.data_ptr() == t.data_ptr() and (self.s.T == 1 or out.stride(0) == t.stride(0)):
                    continue
                raise ValueError(f"{o} overlaps {n}")

    def _prepare_forward(self):
        self._apart(self._FORWARD, ("qo", "ko"))
        return self._convert_forward()

    def _prepare_backward(self):
        if self.ws is None or (self.dqo is None and self.dko is None):
            raise ValueError("no upstream gradients dqo, dko were given")
        unused = {n for g, names in ((self.gq, ("q", "dgq")), (self.gk, ("k", "dgk"))) if g is None for n in names}
        self._apart([n for n in self._BACKWARD if n not in unused], ("dq", "dk", "dgq", "dgk", "ws"))
        return self._convert_backward()

    def _convert_forward(self):
        self._fwd = L.Prepared("lr_qk_fwd", *self._common(), *self._rows("qo", "ko"))
        return self._fwd

    def _convert_backward(self):
        self._bwd = L.Prepared("lr_qk_bwd", *self._common(), *self._rows("dqo", "dko", "dq", "dk"), self.dgq, self.dgk,
                               self.ws, L._nbytes(self.ws))
        return self._bwd

    def forward(self, stream=None):
        (self._fwd or self._prepare_forward())(stream)
        return self.qo, self.ko

    def backward(self, stream=None):
        (self._bwd or self._prepare_backward())(stream)
        return self.dq, self.dk

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)


_BLOCK_PAIRS = tuple(f"{m}_{n}" for n in ("q", "k", "v", "o", "gate", "up", "down") for m in "AB")


def _block_struct(kind, pair, g_attn, g_mlp, at):
    """lr_block_weights or lr_block_grads of the pointers of _BLOCK_PAIRS."""
    pairs = [pair(*at[i:i + 2]) for i in range(0, len(at), 2)]
    return kind(g_attn, *pairs[:4], g_mlp, *pairs[4:])


class TransformerBlock(_Clipped):
    """One low-rank transformer block (q/k/v group, causal attention, o-projection with its
    residual, MLP block in checkpoint mode) resident on the device, bf16.

    qk: the heads' position rotation (its T, Hq, Hk, dh those of the block), with case["freq"], case["pos"]
    (int32 [axes, b*s]; None or missing: positions within each sequence) and the gains case["gq"], case["gk"]
    [dh] of the queries' and keys' norms (None or missing: no norm).  The block's eps serves these norms too.

    Inputs and weights are the entries of self.t and gradients those of self.grads, dg_attn, dg_mlp, dgq and dgk, as
    they are when a call is made: each may be replaced by a tensor of its size and type."""

    def __init__(self, shape, case: Dict[str, object], device="cuda", qk: Optional[QkShape] = None):
        self.sh = shape
        self.t = {k: v.to(device).contiguous() for k, v in case.items() if isinstance(v, torch.Tensor)}
        t, bf16, f32 = self.t, torch.bfloat16, torch.float32
        self._rotation = self.dgq = self.dgk = None
        self._made, self._fits = {}, {n: (tuple(t[n].shape), bf16) for n in ("g_attn", "g_mlp", *_BLOCK_PAIRS)}
        if qk is not None:
            if (qk.T, qk.Hq, qk.Hk, qk.dh, qk.dtype) != (shape.T, shape.H, shape.H, shape.dh, "bf16"):
                raise ValueError("the rotation's tokens, heads or type are not those of the block")
            if len(case["freq"]) != qk.rot // 2:
                raise ValueError(f"{len(case['freq'])} frequencies for {qk.rot // 2} pairs")
            self._fits.update(turns=((qk.rot // 2,), torch.int64), pos=((len(qk.sec), qk.T), torch.int32),
                              gq=((qk.dh,), bf16), gk=((qk.dh,), bf16), dgq=((qk.dh,), f32), dgk=((qk.dh,), f32))
            self._rotation = _qk_shape(qk)
            self.turns = L.turns_tensor(case["freq"], device)
            self.dgq, self.dgk = (torch.empty(qk.dh, dtype=f32, device=device) if n in t else None
                                  for n in ("gq", "gk"))
        self.grads = {}
        for n in _BLOCK_PAIRS:
            self.grads["d" + n] = torch.empty(t[n].shape, dtype=f32, device=device)
        self.dg_attn = torch.empty(shape.d, dtype=f32, device=device)
        self.dg_mlp = torch.empty(shape.d, dtype=f32, device=device)
        self._fits.update({"d" + n: (self._fits[n][0], f32) for n in _BLOCK_PAIRS}, dg_attn=((shape.d,), f32),
                          dg_mlp=((shape.d,), f32))
        dims = (shape.b, shape.s, shape.H, shape.dh, shape.f, shape.ra, shape.rm)
        self.dims = dims
        self.out = torch.empty_like(t["x"])
        self.dx = torch.empty_like(t["x"])
        rotated = self._rotation is not None
        self.saved = _buf((L.lr_block_qk_saved_bytes if rotated else L.lr_block_saved_bytes)(*dims), device)
        self.ws = _buf((L.lr_block_qk_workspace_bytes if rotated else L.lr_block_workspace_bytes)(*dims), device)
        self.w, self.g, self.qk  # refuse what does not fit

    def _struct(self, kind, tensors, make):
        """What `make` builds of the tensors' pointers, kept with their memory until one of them changes."""
        given = [t for t in tensors.values() if t is not None]
        now = ([t is None for t in tensors.values()], _facts(given))
        made = self._made.get(kind)
        if made is None or made[0] != now:
            for n, t in tensors.items():
                size, dtype = self._fits[n]
                if t is not None and (tuple(t.shape) != size or t.dtype != dtype or not t.is_contiguous()
                                      or t.device != self.out.device):
                    raise ValueError(f"{n}: {list(size)} {dtype} on {self.out.device} needed, contiguous, not "
                                     f"{list(t.shape)} {t.dtype} on {t.device} with strides {t.stride()}")
            made = self._made[kind] = (now, make(*map(L._p, tensors.values())), [t.detach() for t in given])
        return made[1]

    @property
    def w(self) -> L.lr_block_weights:
        t = self.t
        return self._struct("w", {n: t[n] for n in ("g_attn", "g_mlp", *_BLOCK_PAIRS)},
                            lambda ga, gm, *p: _block_struct(L.lr_block_weights, L.pair, ga, gm, p))

    @property
    def g(self) -> L.lr_block_grads:
        gr = self.grads
        return self._struct("g", {"dg_attn": self.dg_attn, "dg_mlp": self.dg_mlp,
                                  **{"d" + n: gr["d" + n] for n in _BLOCK_PAIRS}},
                            lambda ga, gm, *p: _block_struct(L.lr_block_grads, L.pair_grad, ga, gm, p))

    @property
    def qk(self) -> Optional[L.lr_block_qk]:
        if self._rotation is None:
            return None
        t = self.t
        return self._struct("qk", {"turns": self.turns, "pos": t.get("pos"), "gq": t.get("gq"), "gk": t.get("gk")},
                            lambda *at: L.lr_block_qk(self._rotation, *at))

    def forward(self, stream=None):
        common = (L.LR_BF16, *self.dims, self.sh.eps, self.t["x"], self.w)
        if self._rotation is None:
            L.lr_block_fwd(*common, self.out, self.saved, self.ws, stream)
        else:
            L.lr_block_qk_fwd(*common, self.qk, self.out, self.saved, self.ws, stream)

    def backward(self, stream=None):
        common = (L.LR_BF16, *self.dims, self.sh.eps, self.t["x"], self.w)
        if self._rotation is None:
            L.lr_block_bwd(*common, self.saved, self.t["G"], self.dx, self.g, self.ws, stream)
        else:
            self._struct("dg", {"dgq": self.dgq, "dgk": self.dgk}, lambda *at: None)
            L.lr_block_qk_bwd(*common, self.qk, self.saved, self.t["G"], self.dx, self.g, self.dgq, self.dgk, self.ws,
                              stream)

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    def grad_tensors(self):
        gains = [g for g in (self.dg_attn, self.dg_mlp, self.dgq, self.dgk) if g is not None]
        return [*gains, *self.grads.values()]
