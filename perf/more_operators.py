"""What is timed of the operators that training on packed text adds to the low-rank transformer.

* ``attn``: causal attention over sequences of different lengths that lie one behind the other in the rows of q, k, v,
  with query heads that share key heads, forward ("fwd") and backward ("bwd", of the forward's o and lse).  Row t of a
  sequence, head h of q, head h // (Hq / Hk) of k and v: S_tj = scale q_t.k_j for j <= t of the same sequence,
  lse_t = log sum_j exp S_tj, o_t = sum_j exp(S_tj - lse_t) v_j.  Rows behind the last sequence stay as they are.
* ``logp``: log probabilities of given tokens under logits [T, V], the entropy of each row's distribution and its most
  probable tokens (equal logits: the lowest index first), forward and backward.  z = scale * logits,
  logp = z[target] - lse (0 where the target is negative), H = -sum p log p.

``run`` computes them from elementary torch operations, or, where ``own`` is true, by the package's calls.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FLOPS = 2_100_000_000_000  # that a drawn case may need: below the largest listed one
BYTES = 2_100_000_000  # that a drawn case may move: below the largest listed one
CHUNK = 1024  # queries that the plain form takes at a time


# ------------------------------------------------------------------ cases
def _attn(direction, T, lens, Hq, Hk, dh, n=1, used=0, packed=False):
    """lens "even": n sequences of used // n tokens; "mixed": n of uneven lengths, used tokens in all."""
    return dict(op="attn", dir=direction, T=T, lens=lens, n=n, used=used or T, Hq=Hq, Hk=Hk, dh=dh, packed=packed,
                dtype="bf16")


def _logp(direction, T, V, top, dtype, scale=1.0, entropy=True):
    return dict(op="logp", dir=direction, T=T, V=V, top=top, dtype=dtype, scale=scale, entropy=entropy)


def listed():
    cases = {
        # one short prompt: latency
        "attn_fwd_17_tokens": _attn("fwd", 17, "even", 32, 8, 128),
        # a training batch packed from texts of all lengths, shared key heads, q, k, v inside one matrix, padded rows
        "attn_fwd_mixed_packed": _attn("fwd", 16384, "mixed", 32, 8, 128, n=24, used=16300, packed=True),
        # the training batch of the attention projections (4 sequences of 4096 tokens, 32 heads of 128)
        "attn_fwd_4x4096": _attn("fwd", 16384, "even", 32, 32, 128, n=4),
        # one long text
        "attn_fwd_16384_tokens": _attn("fwd", 16384, "even", 32, 8, 128),
        # an odd head width, five query heads to a key head, many short sequences
        "attn_fwd_odd": _attn("fwd", 5003, "mixed", 10, 2, 72, n=61),
        # backward of a few short sequences
        "attn_bwd_130_tokens": _attn("bwd", 130, "mixed", 32, 8, 128, n=3),
        # backward of the packed training batch
        "attn_bwd_mixed_packed": _attn("bwd", 16384, "mixed", 32, 8, 128, n=24, used=16300, packed=True),
        # backward of the training batch of the attention projections
        "attn_bwd_4x4096": _attn("bwd", 16384, "even", 32, 32, 128, n=4),
        # the next token of one sequence, with the alternatives to it: latency
        "logp_fwd_1_token": _logp("fwd", 1, 131072, 20, "bf16"),
        # a training batch over a large vocabulary
        "logp_fwd_4096_tokens": _logp("fwd", 4096, 131072, 0, "bf16"),
        # rollouts scored at a temperature, odd vocabulary, fp32, five alternatives
        "logp_fwd_odd_f32": _logp("fwd", 515, 50021, 5, "f32", scale=1.25),
        # the gradient of a training batch's loss with an entropy term
        "logp_bwd_4096_tokens": _logp("bwd", 4096, 131072, 0, "bf16"),
    }
    return [dict(c, name=k) for k, c in cases.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    if rng.random() < 0.65:
        while True:
            T = _log(rng, 1, 32768)
            Hk = rng.choice([1, 2, 4, 8, rng.randint(1, 16)])
            Hq = min(64 // Hk, rng.choice([1, 1, 2, 4, 4, 5, 7, 8, 16])) * Hk
            dh = rng.choice([64, 128, 128, 128, 8 * rng.randint(2, 16)])
            used = T if rng.random() < 0.7 else rng.randint(max(1, T // 2), T)
            n = 1 if rng.random() < 0.3 else min(used, _log(rng, 1, 200))
            c = _attn(rng.choice(["fwd", "bwd"]), T, rng.choice(["even", "mixed", "mixed"]), Hq, Hk, dh, n=n, used=used,
                      packed=rng.random() < 0.5)
            if work(c)["flops"] <= FLOPS and work(c)["bytes"] <= BYTES:
                return c
    while True:
        V = rng.choice([32000, 50021, 65536, 131072, _log(rng, 100, 262144)])
        c = _logp(rng.choice(["fwd", "fwd", "bwd"]), _log(rng, 1, 16384), V, rng.choice([0, 0, 1, 5, 20, 32]),
                  rng.choice(["bf16", "bf16", "f32"]), rng.choice([1.0, 1.0, 0.7, 1.25]), rng.random() < 0.6)
        if work(c)["bytes"] <= BYTES:
            return c


def _lengths(case):
    """Tokens of each sequence; they add up to case["used"]."""
    n, used = case["n"], case["used"]
    if case["lens"] == "even":
        return [used // n + (i < used % n) for i in range(n)]
    rng = random.Random(used * 1000003 + n)
    w = [math.exp(rng.uniform(0.0, 4.0)) for _ in range(n)]
    ends = [round(used * sum(w[:i + 1]) / sum(w)) for i in range(n)]
    return [e - b for b, e in zip([0] + ends, ends)]


def work(case):
    es, T = (2 if case["dtype"] == "bf16" else 4), case["T"]
    if case["op"] == "logp":
        n = T * case["V"]
        if case["dir"] == "bwd":
            return {"bytes": 2 * n * es + 16 * T, "flops": 6 * n}
        return {"bytes": n * es + T * (16 + 8 * case["top"]), "flops": 5 * n}
    pairs = sum(s * (s + 1) // 2 for s in _lengths(case)) * case["Hq"] * case["dh"]
    rows, dh, lse = case["used"], case["dh"], 4 * case["used"] * case["Hq"]
    if case["dir"] == "fwd":
        return {"bytes": rows * 2 * (case["Hq"] + case["Hk"]) * dh * es + lse, "flops": 4 * pairs}
    return {"bytes": rows * 4 * (case["Hq"] + case["Hk"]) * dh * es + lse, "flops": 10 * pairs}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _attn_inputs(case, seed):
    gen = _generator(seed)
    T, Hq, Hk, dh, dt = case["T"], case["Hq"], case["Hk"], case["dh"], TYPES[case["dtype"]]
    # heads of different sharpness: scores of a standard deviation around one
    m = torch.randn(T, Hq + 2 * Hk, dh, generator=gen, device="cuda")
    m = m * torch.exp(0.3 * torch.randn(1, Hq + 2 * Hk, 1, generator=gen, device="cuda"))
    m = m.to(dt).reshape(T, (Hq + 2 * Hk) * dh)
    s = dict(zip("qkv", m.split([Hq * dh, Hk * dh, Hk * dh], dim=1)))
    if not case["packed"]:
        s = {n: t.contiguous() for n, t in s.items()}
    offs = [0]
    for n in _lengths(case):
        offs.append(offs[-1] + n)
    s["offs"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
    s["dout"] = None
    if case["dir"] == "bwd":
        s["dout"] = torch.randn(T, Hq * dh, generator=gen, device="cuda").to(dt)
    return s, offs


def _logp_inputs(case, seed):
    gen = _generator(seed)
    T, V = case["T"], case["V"]
    z = torch.randn(T, V, generator=gen, device="cuda").mul_(2.5)
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # most tokens are predicted well: their logits stand out by a few units
    z[torch.arange(T, device="cuda"), target] += 8 + 4 * torch.randn(T, generator=gen, device="cuda")
    counted = torch.rand(T, generator=gen, device="cuda") < 0.9
    s = {"logits": z.to(TYPES[case["dtype"]]), "target": torch.where(counted, target, -100).to(torch.int32),
         "dlogp": None, "dentropy": None}
    if case["dir"] == "bwd":
        s["dlogp"] = -torch.exp(0.5 * torch.randn(T, generator=gen, device="cuda")) / T
        if case["entropy"]:
            s["dentropy"] = torch.full((T,), 0.01 / T, device="cuda")
    return s


def prepare(case, seed):
    if case["op"] == "logp":
        s = _logp_inputs(case, seed)
        given = {}
        if case["dir"] == "bwd":  # what the forward left behind
            z = s["logits"].float() * case["scale"]
            given["lse"] = z.logsumexp(-1)
            lp = z.sub_(given["lse"][:, None])
            given["entropy"] = -(lp.exp() * lp).sum(-1)
            del z, lp
        if own:
            from rank_bottleneck_block_gb300.inputs import LogProbShape
            from rank_bottleneck_block_gb300.runner import TokenLogProbs

            shape = LogProbShape(T=case["T"], V=case["V"], top=case["top"], scale=case["scale"], dtype=case["dtype"])
            h = TokenLogProbs(shape, s)
            if given:
                h.lse, h.entropy = given["lse"], given["entropy"]
            return {"case": case, "own": True, "handle": h}
        return {"case": case, "own": False, **s, **given}
    s, offs = _attn_inputs(case, seed)
    given = {}
    if case["dir"] == "bwd":
        given = _plain_attn_fwd(case, s, offs)
    if own:
        from rank_bottleneck_block_gb300.inputs import PackedShape
        from rank_bottleneck_block_gb300.runner import PackedAttention

        shape = PackedShape(T=case["T"], nseq=case["n"], Hq=case["Hq"], Hk=case["Hk"], dh=case["dh"])
        h = PackedAttention(shape, s)
        for n in ("o", "lse") if case["dir"] == "fwd" else ("dq", "dk", "dv"):
            getattr(h, n).zero_()  # rows behind the last sequence are not written
        if given:
            h.o, h.lse = given["o"], given["lse"]
        return {"case": case, "own": True, "handle": h}
    return {"case": case, "own": False, "where": offs, **s, **given}


# -------------------------------------------------------------- plain form
def _heads(x, case, H):
    """[T, H * dh] as fp32 [Hk, T, H / Hk, dh]."""
    x = x.float().reshape(x.shape[0], case["Hk"], H // case["Hk"], case["dh"])
    return x.permute(1, 0, 2, 3)


def _walk(case, q, k, offs):
    """Of each sequence, run after run of queries: its first row, the run's rows, and the run's scores
    [Hk, rows * group, keys], -inf behind each query's own position."""
    group, scale = case["Hq"] // case["Hk"], case["dh"] ** -0.5
    for b, e in zip(offs, offs[1:]):
        for r in range(b, e, CHUNK):
            t = min(e, r + CHUNK)
            S = (q[:, r:t].flatten(1, 2) @ k[:, b:t, 0].transpose(1, 2)) * scale
            place = torch.arange(r, t, device=S.device).repeat_interleave(group)
            late = torch.arange(b, t, device=S.device)[None, :] > place[:, None]
            yield b, r, t, S.masked_fill_(late, float("-inf"))


def _plain_attn_fwd(case, s, offs):
    T, Hq, dh = case["T"], case["Hq"], case["dh"]
    q, k, v = _heads(s["q"], case, Hq), _heads(s["k"], case, case["Hk"]), _heads(s["v"], case, case["Hk"])
    o = torch.zeros(T, Hq * dh, dtype=s["q"].dtype, device="cuda")
    lse = torch.zeros(T, Hq, device="cuda")
    for b, r, t, S in _walk(case, q, k, offs):
        m = S.amax(-1, keepdim=True)
        p = S.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        y = (p @ v[:, b:t, 0]) / total
        o[r:t] = y.unflatten(1, (t - r, -1)).transpose(0, 1).reshape(t - r, Hq * dh).to(o.dtype)
        lse[r:t] = (m + total.log()).unflatten(1, (t - r, -1)).transpose(0, 1).reshape(t - r, Hq)
    return {"o": o, "lse": lse}


def _plain_attn_bwd(case, s, offs):
    Hq, Hk, scale = case["Hq"], case["Hk"], case["dh"] ** -0.5
    q, k, v = _heads(s["q"], case, Hq), _heads(s["k"], case, Hk), _heads(s["v"], case, Hk)
    o, do = _heads(s["o"], case, Hq), _heads(s["dout"], case, Hq)
    D = (o * do).sum(-1)
    lse = s["lse"].reshape(case["T"], Hk, Hq // Hk).permute(1, 0, 2)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, r, t, S in _walk(case, q, k, offs):
        p = S.sub_(lse[:, r:t].flatten(1)[..., None]).exp_()
        g = do[:, r:t].flatten(1, 2)
        dv[:, b:t, 0] += p.transpose(1, 2) @ g
        ds = (g @ v[:, b:t, 0].transpose(1, 2)).sub_(D[:, r:t].flatten(1)[..., None]).mul_(p).mul_(scale)
        dq[:, r:t] = (ds @ k[:, b:t, 0]).unflatten(1, (t - r, -1))
        dk[:, b:t, 0] += ds.transpose(1, 2) @ q[:, r:t].flatten(1, 2)
    rows = {"dq": dq, "dk": dk, "dv": dv}
    return {n: x.permute(1, 0, 2, 3).reshape(case["T"], -1).to(s["q"].dtype) for n, x in rows.items()}


def _plain_logp(s):
    c = s["case"]
    z = s["logits"].float() * c["scale"]
    counted = s["target"] >= 0
    at = s["target"].clamp(min=0).long()[:, None]
    if c["dir"] == "bwd":
        lp = z.sub_(s["lse"][:, None])
        p = lp.exp()
        dlogp = torch.where(counted, s["dlogp"], torch.zeros_like(s["dlogp"]))
        d = p * -dlogp[:, None]
        d.scatter_add_(1, at, dlogp[:, None])
        if s["dentropy"] is not None:
            d -= s["dentropy"][:, None] * p * (lp + s["entropy"][:, None])
        return {"dlogits": (d * c["scale"]).to(s["logits"].dtype)}
    m = z.amax(-1, keepdim=True)
    lse = m + (z - m).exp().sum(-1, keepdim=True).log()
    lp = z - lse
    out = {"logp": torch.where(counted, lp.gather(1, at)[:, 0], torch.zeros_like(m[:, 0])),
           "entropy": -(lp.exp() * lp).sum(-1), "lse": lse[:, 0]}
    if c["top"]:
        ids = s["logits"].sort(dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        out["top_ids"], out["top_logp"] = ids.to(torch.int32), lp.gather(1, ids)
    return out


def run(s):
    c = s["case"]
    if not s["own"]:
        if c["op"] == "logp":
            return _plain_logp(s)
        return _plain_attn_fwd(c, s, s["where"]) if c["dir"] == "fwd" else _plain_attn_bwd(c, s, s["where"])
    h = s["handle"]
    if c["op"] == "logp":
        if c["dir"] == "bwd":
            return {"dlogits": h.backward()}
        h.forward()
        out = {"logp": h.logp, "entropy": h.entropy, "lse": h.lse}
        return dict(out, top_ids=h.top_ids, top_logp=h.top_logp) if c["top"] else out
    if c["dir"] == "fwd":
        h.forward()
        return {"o": h.o, "lse": h.lse}
    h.backward()
    return {"dq": h.dq, "dk": h.dk, "dv": h.dv}


# ------------------------------------------------------- definition in 64 bits
def _exact_logp(case, seed):
    s = _logp_inputs(case, seed)
    names = ["dlogits"] if case["dir"] == "bwd" else ["logp", "entropy", "lse"]
    parts = {n: [] for n in names + (["top_ids", "top_logp"] if case["top"] and case["dir"] == "fwd" else [])}
    for r in range(0, case["T"], 256):
        x = s["logits"][r:r + 256].double().requires_grad_(case["dir"] == "bwd")
        z = x * case["scale"]
        lse = torch.logsumexp(z, -1)
        prob = torch.softmax(z, -1)
        lp = torch.log_softmax(z, -1)
        entropy = -(prob * lp).sum(-1)
        target = s["target"][r:r + 256].long()
        onehot = torch.arange(case["V"], device="cuda")[None, :] == target[:, None]
        logp = torch.where(onehot, lp, torch.zeros_like(lp)).sum(-1)
        if case["dir"] == "bwd":
            total = (logp * s["dlogp"][r:r + 256]).sum()
            if case["entropy"]:
                total = total + (entropy * s["dentropy"][r:r + 256]).sum()
            total.backward()
            parts["dlogits"].append(x.grad)
            continue
        for n, t in zip(names, (logp, entropy, lse)):
            parts[n].append(t)
        if case["top"]:
            ids = torch.argsort(-x, dim=-1, stable=True)[:, :case["top"]]
            parts["top_ids"].append(ids.to(torch.int32))
            parts["top_logp"].append(lp.gather(1, ids))
        del x, z, prob, lp, onehot
    return {n: torch.cat(t) for n, t in parts.items()}


def exact(case, seed):
    """Softmax over each query's own keys, a head at a time, and gradients by differentiating it, in float64."""
    if case["op"] == "logp":
        return _exact_logp(case, seed)
    back = case["dir"] == "bwd"
    if sum(n * n for n in _lengths(case)) * case["Hq"] * case["dh"] * (12 if back else 4) > 8e12:
        return None
    s, offs = _attn_inputs(case, seed)
    T, Hq, Hk, dh = case["T"], case["Hq"], case["Hk"], case["dh"]
    q, k, v = (s[n].double().reshape(T, -1, dh) for n in "qkv")
    out = {n: torch.zeros_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v))} if back else {
        "o": torch.zeros_like(q), "lse": torch.zeros(T, Hq, dtype=torch.float64, device="cuda")}
    for b, e in zip(offs, offs[1:]):
        if b == e:
            continue
        seen = torch.ones(e - b, e - b, dtype=torch.bool, device="cuda").tril()
        for h in range(Hq):
            hk = h * Hk // Hq
            qs, ks, vs = (x[b:e, i].clone().requires_grad_(back) for x, i in ((q, h), (k, hk), (v, hk)))
            S = torch.where(seen, qs @ ks.T / math.sqrt(dh), torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
            y = torch.softmax(S, -1) @ vs
            if not back:
                out["o"][b:e, h], out["lse"][b:e, h] = y, torch.logsumexp(S, -1)
                continue
            y.backward(s["dout"][b:e, h * dh:(h + 1) * dh].double())
            out["dq"][b:e, h] = qs.grad
            out["dk"][b:e, hk] += ks.grad
            out["dv"][b:e, hk] += vs.grad
            del S, y
    return {n: t if n == "lse" else t.flatten(1) for n, t in out.items()}
