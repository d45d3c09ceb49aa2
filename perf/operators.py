"""What is timed of the operators around attention and after the backward of the low-rank transformer.

* ``qk``: the norm of every query and key head and the rotation by its token's position, in one pass, forward
  ("fwd") and backward ("bwd").  Token t, head vector x, gain g, 1/rms r = (mean x^2 + eps)^-1/2, n = x r g (n = x
  without the norm); channel pair p turns by pos[axis(p), t] * freq[p]; channels from ``rot`` on are not turned.
* ``clip``: the norm over all gradients of a model, norm = sqrt(sum g^2), and out = g min(1, bound / (norm + 1e-6)).

``run`` computes them from elementary torch operations, or, where ``own`` is true, by the package's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-6
LIMIT = 2_200_000_000  # bytes a drawn case may move: below the largest listed case

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _qk(direction, T, Hq, Hk, dh, rot, axes, norm, layout, dtype, packed, start, theta=10000.0):
    return dict(op="qk", dir=direction, T=T, Hq=Hq, Hk=Hk, dh=dh, rot=rot, axes=axes, norm=norm, layout=layout,
                dtype=dtype, packed=packed, start=start, theta=theta)


def _clip(tensors, dtype, bound, blocks=0, d=0, f=0, r=0, attn=False, n=0, total=0):
    return dict(op="clip", tensors=tensors, dtype=dtype, bound=bound, blocks=blocks, d=d, f=f, r=r, attn=attn, n=n,
                total=total)


def listed():
    cases = {
        # one new token of one sequence, far into its context: latency
        "qk_fwd_1_token": _qk("fwd", 1, 32, 8, 128, 128, 1, True, "half", "bf16", True, 131000),
        # one new token of each of 96 sequences, rotation alone
        "qk_fwd_96_tokens_rotation": _qk("fwd", 96, 32, 8, 128, 128, 1, False, "half", "bf16", True, 5000),
        # the training batch of the attention projections (4 sequences of 4096 tokens, 32 heads of 128)
        "qk_fwd_16384_tokens": _qk("fwd", 16384, 32, 32, 128, 128, 1, True, "half", "bf16", False, 0),
        # a video clip: time, height and width positions, shared key heads, q and k inside one packed matrix
        "qk_fwd_3_axes_packed": _qk("fwd", 12483, 20, 4, 128, 128, 3, True, "half", "bf16", True, 0),
        # an odd head width turned in part, neighbouring channels paired, fp32
        "qk_fwd_odd_f32": _qk("fwd", 1531, 7, 1, 80, 56, 1, True, "pairs", "f32", False, 17),
        # backward of a short batch
        "qk_bwd_130_tokens": _qk("bwd", 130, 32, 8, 128, 128, 1, True, "half", "bf16", False, 0),
        # backward of the training batch
        "qk_bwd_16384_tokens": _qk("bwd", 16384, 32, 32, 128, 128, 1, True, "half", "bf16", False, 0),
        # backward of the clip, two axes and a part of the channels not turned
        "qk_bwd_2_axes_odd_f32": _qk("bwd", 5003, 6, 2, 72, 40, 2, True, "half", "f32", False, 3),
        # gradients of one small MLP block (d 256, f 688, rank 64)
        "clip_small_block": _clip("model", "f32", 1.0, blocks=1, d=256, f=688, r=64),
        # gradients of one transformer block (d 4096, f 11008, ranks 1024)
        "clip_transformer_block": _clip("model", "f32", 1.0, blocks=1, d=4096, f=11008, r=1024, attn=True),
        # many tensors of uneven, odd sizes, held in bf16
        "clip_ragged_bf16": _clip("ragged", "bf16", 1.0, n=613, total=20_000_003),
        # gradients of 24 MLP blocks (d 2048, f 5632, rank 512)
        "clip_24_blocks": _clip("model", "f32", 1.0, blocks=24, d=2048, f=5632, r=512),
    }
    return [dict(c, name=k) for k, c in cases.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    if rng.random() < 0.7:
        while True:
            T = _log(rng, 1, 65536)
            dh = rng.choice([64, 128, 128, 128, 256, 8 * rng.randint(2, 32)])
            rot = dh if rng.random() < 0.6 else 8 * rng.randint(1, dh // 8)
            Hk = rng.choice([1, 2, 4, 8, rng.randint(1, 32)])
            Hq = min(64, Hk * rng.choice([1, 1, 2, 4, 5, 8]))
            c = _qk(rng.choice(["fwd", "bwd"]), T, Hq, Hk, dh, rot, min(rng.choice([1, 1, 2, 3, 4]), rot // 2),
                    rng.random() < 0.75, rng.choice(["half", "half", "pairs"]), rng.choice(["bf16", "bf16", "f32"]),
                    rng.random() < 0.4, rng.choice([0, rng.randint(0, 1 << 20)]), rng.choice([1e4, 5e5, 1e6]))
            if work(c)["bytes"] <= LIMIT:
                return c
    while True:
        dtype, bound = rng.choice(["f32", "f32", "bf16"]), rng.choice([0.5, 1.0, 1.0, 1e4])
        if rng.random() < 0.6:
            d = 8 * _log(rng, 8, 640)
            c = _clip("model", dtype, bound, blocks=_log(rng, 1, 24), d=d, f=8 * (d * rng.randint(2, 4) // 8 + 1),
                      r=8 * max(1, d // rng.choice([16, 32, 64])), attn=rng.random() < 0.5)
        else:
            n = _log(rng, 1, 700)
            c = _clip("ragged", dtype, bound, n=n, total=_log(rng, 100 * n, 200_000_000))
        if work(c)["bytes"] <= LIMIT:
            return c


def _sections(case):
    """Channel pairs of each axis: the first axis takes what the even split leaves over."""
    each = (case["rot"] // 2) // case["axes"]
    return [case["rot"] // 2 - each * (case["axes"] - 1)] + [each] * (case["axes"] - 1)


def _sizes(case):
    if case["tensors"] == "ragged":
        rng = random.Random(case["n"] * 1000003 + case["total"])
        w = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(case["n"])]
        return [1 + int((case["total"] - case["n"]) * v / sum(w)) for v in w]
    d, f, r = case["d"], case["f"], case["r"]
    block = [d, r * d, f * r, r * d, f * r, r * f, d * r]
    if case["attn"]:
        block += [d] + [r * d, d * r] * 4
    return block * case["blocks"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * n * es, "flops": 3 * n}
    n = case["T"] * (case["Hq"] + case["Hk"]) * case["dh"]
    tensors = 2 if case["dir"] == "fwd" or not case["norm"] else 3
    return {"bytes": tensors * n * es + 4 * case["axes"] * case["T"], "flops": n * (10 if case["dir"] == "fwd" else 20)}


# ------------------------------------------------------------------ inputs
def _qk_inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, Hq, Hk, dh, dt = case["T"], case["Hq"], case["Hk"], case["dh"], TYPES[case["dtype"]]

    def normal(*size):
        return torch.randn(*size, generator=gen, device="cuda")

    def rows(scaled):
        """q and k of a scale per head, as matrices of their own or as columns of the packed q, k, v."""
        wide = Hq + (2 * Hk if case["packed"] else Hk)
        m = normal(T, wide, dh) if not scaled else normal(T, wide, dh) * torch.exp(0.5 * normal(1, wide, 1))
        m = m.to(dt).reshape(T, wide * dh)
        q, k = m[:, :Hq * dh], m[:, Hq * dh:(Hq + Hk) * dh]
        return (q, k) if case["packed"] else (q.contiguous(), k.contiguous())

    s = {}
    s["q"], s["k"] = rows(True)
    s["gq"] = s["gk"] = None
    if case["norm"]:
        s["gq"], s["gk"] = (1 + 0.1 * normal(dh)).to(dt), (1 + 0.1 * normal(dh)).to(dt)
    t = torch.arange(T, device="cuda", dtype=torch.int64)
    if case["axes"] == 1:
        # decoding: every sequence at a place of its own; training: sequences of 4096 tokens
        far = torch.randint(0, max(1, case["start"]), (T,), generator=gen, device="cuda")
        pos = [far if T <= 256 and case["dir"] == "fwd" else case["start"] + t % 4096]
    else:
        # frames of a grid of 30 x 52 patches, then (4 axes) the index of the clip
        pos = [case["start"] + t // 1560, t // 52 % 30, t % 52, t // 15600][:case["axes"]]
    s["pos"] = torch.stack(pos).to(torch.int32).contiguous()
    s["freq"] = [case["theta"] ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
    s["dqo"] = s["dko"] = None
    if case["dir"] == "bwd":
        s["dqo"], s["dko"] = rows(False)
    return s


def _clip_inputs(case, seed):
    """The gradients, as a program keeps them: 16-byte aligned pieces of one flat buffer."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    sizes, at, n = _sizes(case), [], 0
    for v in sizes:
        at.append(n)
        n += (v + 7) // 8 * 8
    flat = torch.zeros(n, device="cuda", dtype=TYPES[case["dtype"]])
    scale = torch.exp(torch.randn(len(sizes), generator=gen, device="cuda") * 1.0 - 6.0).tolist()
    for o, v, sc in zip(at, sizes, scale):
        flat[o:o + v] = torch.randn(v, generator=gen, device="cuda") * sc
    return {"flat": flat, "at": at, "sizes": sizes}


def prepare(case, seed):
    s = {"case": case, "own": own}
    if case["op"] == "clip":
        s.update(_clip_inputs(case, seed))
        s["grads"] = [s["flat"][o:o + v] for o, v in zip(s["at"], s["sizes"])]
        if own:
            from rank_bottleneck_block_gb300.runner import GradClip

            s["out"] = torch.zeros_like(s["flat"])
            outs = [s["out"][o:o + v] for o, v in zip(s["at"], s["sizes"])]
            s["handle"] = GradClip(s["grads"], case["bound"], outs=outs)
        return s
    s.update(_qk_inputs(case, seed))
    if own:
        from rank_bottleneck_block_gb300.inputs import QkShape
        from rank_bottleneck_block_gb300.runner import QkRotary

        shape = QkShape(T=case["T"], Hq=case["Hq"], Hk=case["Hk"], dh=case["dh"], rot=case["rot"],
                        sec=tuple(_sections(case)), layout=case["layout"], dtype=case["dtype"], eps=EPS)
        s["handle"] = QkRotary(shape, {k: s[k] for k in ("q", "k", "gq", "gk", "pos", "freq", "dqo", "dko")})
    else:
        s["freq"] = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
        s["axis"] = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(_sections(case))).to("cuda")
    return s


# -------------------------------------------------------------- plain form
def _turn(x, cos, sin, rot, layout):
    """[T, H, dh] fp32 with the pairs of its first `rot` channels turned."""
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_qk(s):
    c = s["case"]
    rot, layout = c["rot"], c["layout"]
    angle = (s["pos"].double()[s["axis"]].T * s["freq"])[:, None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    out = {}
    for n, H in (("q", c["Hq"]), ("k", c["Hk"])):
        x, g = s[n], s["g" + n]
        dt = x.dtype
        x = x.float().reshape(-1, H, c["dh"])
        if g is not None:
            g = g.float()
            r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        if c["dir"] == "fwd":
            y = _turn(x if g is None else x * r * g, cos, sin, rot, layout)
            out[n + "o"] = y.to(dt).flatten(1)
            continue
        dn = _turn(s[f"d{n}o"].float().reshape(-1, H, c["dh"]), cos, -sin, rot, layout)
        if g is None:
            out["d" + n] = dn.to(dt).flatten(1)
            continue
        u = x * r
        w = dn * g
        out["dg" + n] = (dn * u).sum((0, 1))
        out["d" + n] = (r * (w - u * (w * u).mean(-1, keepdim=True))).to(dt).flatten(1)
    return out


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    scale = (s["case"]["bound"] / (norm + 1e-6)).clamp(max=1.0)
    out = torch.zeros_like(s["flat"])
    for g, o, v in zip(s["grads"], s["at"], s["sizes"]):
        out[o:o + v] = g.float() * scale
    return {"flat": out, "norm": norm.reshape(1), "scale": scale.reshape(1)}


def run(s):
    c = s["case"]
    if not s["own"]:
        return _plain_clip(s) if c["op"] == "clip" else _plain_qk(s)
    h = s["handle"]
    if c["op"] == "clip":
        h.clip()
        return {"flat": s["out"], "norm": h.norm, "scale": h.scale}
    if c["dir"] == "fwd":
        h.forward()
        return {"qo": h.qo, "ko": h.ko}
    h.backward()
    if not c["norm"]:
        return {"dq": h.dq, "dk": h.dk}
    return {"dq": h.dq, "dk": h.dk, "dgq": h.dgq, "dgk": h.dgk}


# ------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    """Turns as products of complex numbers and gradients by differentiating the forward, in float64."""
    if case["op"] == "clip":
        s = _clip_inputs(case, seed)
        g = s["flat"].double()
        norm = torch.linalg.vector_norm(g).reshape(1)
        scale = torch.minimum(torch.ones_like(norm), case["bound"] / (norm + 1e-6))
        return {"flat": g * scale, "norm": norm, "scale": scale}
    s = _qk_inputs(case, seed)
    half, rot = case["rot"] // 2, case["rot"]
    theta = torch.empty(case["T"], 1, half, dtype=torch.float64, device="cuda")
    p = 0
    for a, n in enumerate(_sections(case)):
        for i in range(p, p + n):
            theta[:, 0, i] = s["pos"][a].double() * s["freq"][i]
        p += n
    turn = torch.polar(torch.ones_like(theta), theta)
    if case["layout"] == "half":
        first = torch.arange(half, device="cuda")
        second = first + half
    else:
        first = torch.arange(0, rot, 2, device="cuda")
        second = first + 1
    out = {}
    for n, H in (("q", case["Hq"]), ("k", case["Hk"])):
        x = s[n].double().reshape(-1, H, case["dh"])
        g = s["g" + n].double() if case["norm"] else None
        if case["dir"] == "bwd":
            x.requires_grad_(True)
            if g is not None:
                g.requires_grad_(True)
        v = x if g is None else x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dh"] + EPS) * g
        z = torch.complex(v[..., first], v[..., second]) * turn
        y = torch.zeros_like(v)
        y = y.index_copy(-1, first, z.real).index_copy(-1, second, z.imag)
        if rot < case["dh"]:
            rest = torch.arange(rot, case["dh"], device="cuda")
            y = y.index_copy(-1, rest, v[..., rest])
        if case["dir"] == "fwd":
            out[n + "o"] = y.flatten(1)
            continue
        y.backward(s[f"d{n}o"].double().reshape(-1, H, case["dh"]))
        out["d" + n] = x.grad.flatten(1)
        if g is not None:
            out["dg" + n] = g.grad
        del x, v, z, y
    return out
