"""fp64 CPU oracle for the norm and position rotation of queries and keys, and for gradient clipping.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``): only ``tests/`` imports it, and it shares no code
with the CUDA library.

Per token t and head, x in R^dh, gain g (or none), pair p = (i, j) of the first rot channels, a(p) its axis:

    n = x r g,  r = (mean(x^2) + eps)^(-1/2)        (n = x without a gain)
    theta = pos[a(p), t] * freq[p]
    y_i = n_i cos - n_j sin,  y_j = n_i sin + n_j cos,  y_c = n_c for c >= rot

The backward of sum(y * dy) by the chain rule: dn is dy turned by -theta, dg = sum dn x r,
w = dn g, dx = r w - x r^3 mean(w x) (dx = dn without a gain).

Angles of far positions are reduced in exact rational arithmetic (``angles``): float64 products of a
position near 2^31 with a frequency lose some 1e-7 radians.

Clipping: norm = sqrt(sum g^2) over all tensors, scale = min(1, max_norm / (norm + 1e-6)), out = scale g.

Pins (tests/test_qk_oracle.py): central finite differences of every gradient, rotation of a pair of unit
vectors by hand, invariance of inner products under a shift of all positions, unit root mean square after
the norm.
"""
from __future__ import annotations

from fractions import Fraction
from typing import Dict, List, Optional, Sequence

import numpy as np

F64 = np.float64
# 2 pi to 60 digits
TWO_PI = Fraction(628318530717958647692528676655900576839433879875021164194988, 10 ** 59)

__all__ = ["TWO_PI", "angles", "pairs", "qk_fwd", "qk_bwd", "magnitudes", "clip", "block_fwd", "block_bwd"]


def angles(pos: np.ndarray, freq: Sequence[float], sec: Sequence[int]) -> np.ndarray:
    """theta [T, pairs] in [0, 2 pi) from pos [axes, T] (integers) and freq [pairs]."""
    pos = np.asarray(pos)
    out = np.empty((pos.shape[1], len(freq)), dtype=F64)
    axis = [a for a, n in enumerate(sec) for _ in range(n)]
    scale = 1 << 120
    for p, f in enumerate(freq):
        turns = Fraction(f) / TWO_PI
        turns = int(turns * scale) % scale  # one position's turn, to 2^-120
        for t in range(pos.shape[1]):
            out[t, p] = float(Fraction(int(pos[axis[p], t]) * turns % scale, scale) * TWO_PI)
    return out


def pairs(rot: int, layout: str):
    """Channel indices i, j of the rot / 2 pairs."""
    p = np.arange(rot // 2)
    return (p, p + rot // 2) if layout == "half" else (2 * p, 2 * p + 1)


def _turn(x, theta, rot, layout, sign):
    i, j = pairs(rot, layout)
    c, s = np.cos(theta)[:, None, :], sign * np.sin(theta)[:, None, :]
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def _heads(x, dh):
    x = np.asarray(x, dtype=F64)
    return x.reshape(x.shape[0], -1, dh)


def _rstd(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def qk_fwd(x, g: Optional[np.ndarray], theta, dh: int, rot: int, layout: str, eps: float) -> np.ndarray:
    """x [T, H*dh] -> y, same shape."""
    x = _heads(x, dh)
    n = x if g is None else x * _rstd(x, eps) * np.asarray(g, dtype=F64)
    return _turn(n, theta, rot, layout, 1.0).reshape(x.shape[0], -1)


def qk_bwd(x, g: Optional[np.ndarray], theta, dy, dh: int, rot: int, layout: str, eps: float) -> Dict[str, np.ndarray]:
    """dx [T, H*dh] and, with a gain, dg [dh]."""
    dn = _turn(_heads(dy, dh), theta, rot, layout, -1.0)
    if g is None:
        return {"dx": dn.reshape(dn.shape[0], -1)}
    x, g = _heads(x, dh), np.asarray(g, dtype=F64)
    r = _rstd(x, eps)
    w = dn * g
    dx = r * w - x * r ** 3 * np.mean(w * x, axis=-1, keepdims=True)
    return {"dx": dx.reshape(x.shape[0], -1), "dg": np.sum(dn * x * r, axis=(0, 1))}


def magnitudes(x, g, dy, dh: int, rot: int, layout: str, eps: float) -> Dict[str, np.ndarray]:
    """Magnitudes of the terms each result sums, for error bounds of rounded arithmetic: y (|n_i| + |n_j| of the
    channel's pair), dx and dg likewise (of dy's pairs)."""
    i, j = pairs(rot, layout)

    def both(v):
        v = np.abs(v)
        out = v.copy()
        out[..., i] = out[..., j] = v[..., i] + v[..., j]
        return out

    out = {}
    xh = None if x is None else _heads(x, dh)
    T = (dy if x is None else x).shape[0]
    if g is None:
        if xh is not None:
            out["y"] = both(xh).reshape(T, -1)
        if dy is not None:
            out["dx"] = both(_heads(dy, dh)).reshape(T, -1)
        return out
    r, ag = _rstd(xh, eps), np.abs(np.asarray(g, dtype=F64))
    out["y"] = both(xh * r * ag).reshape(T, -1)
    if dy is not None:
        d = both(_heads(dy, dh))
        w = d * ag
        out["dx"] = (r * (w + np.abs(xh) * r ** 2 * np.mean(w * np.abs(xh), axis=-1, keepdims=True))).reshape(T, -1)
        out["dg"] = np.sum(d * np.abs(xh) * r, axis=(0, 1))
    return out


def clip(grads: List[np.ndarray], max_norm: float):
    """(norm, scale, scaled tensors)."""
    top = max([float(np.max(np.abs(g))) for g in grads if g.size] or [0.0])
    unit = top if top > 0 and np.isfinite(top) else 1.0  # squares stay inside the fp64 range
    total = sum(float(np.sum(np.square(np.asarray(g, dtype=F64) / unit))) for g in grads)
    norm = unit * np.sqrt(total)
    scale = min(1.0, max_norm / (norm + 1e-6))
    return norm, scale, [scale * np.asarray(g, dtype=F64) for g in grads]


# ---------------------------------------------------------------------------
# The low-rank transformer block with norm and rotation of q and k before attention.
# ---------------------------------------------------------------------------
def block_fwd(x, W: Dict, rot: Dict, b: int, s: int, H: int, dh: int, eps: float = 1e-6):
    """attention_oracle.block_fwd with q, k normed and rotated; rot: theta [T, pairs], rot, layout, gq, gk."""
    from . import attention_oracle as A
    from . import lowrank_oracle as O

    x = O.to64(x)
    qkv, s_qkv = O.proj_group_fwd(x, W["g_attn"], [W["A_q"], W["A_k"], W["A_v"]],
                                  [W["B_q"], W["B_k"], W["B_v"]], eps)
    qr, kr = (qk_fwd(t, rot[g], rot["theta"], dh, rot["rot"], rot["layout"], eps)
              for t, g in ((qkv[0], "gq"), (qkv[1], "gk")))
    o, s_att = A.attention_fwd(qr, kr, qkv[2], b, s, H, dh, dh ** -0.5)
    (y,), s_o = O.proj_group_fwd(o, None, [W["A_o"]], [W["B_o"]], eps)
    x1 = x + y
    mlp = {k: W[k] for k in ("A_gate", "B_gate", "A_up", "B_up", "A_down", "B_down")}
    out, s_mlp = O.mlp_block_fwd(x1, W["g_mlp"], mlp, eps, O.FULL)
    return out, dict(qkv=qkv, qr=qr, kr=kr, s_qkv=s_qkv, o=o, s_att=s_att, s_o=s_o, mlp=mlp, s_mlp=s_mlp)


def block_bwd(W: Dict, saved: Dict, rot: Dict, G, b: int, s: int, H: int, dh: int, eps: float = 1e-6):
    """Gradients of sum(out * G), with dgq and dgk where the gains are given."""
    from . import attention_oracle as A
    from . import lowrank_oracle as O

    gm = O.mlp_block_bwd(W["g_mlp"], saved["mlp"], saved["s_mlp"], O.to64(G), eps)
    dx1 = gm["dx"]
    go = O.proj_group_bwd(None, [W["A_o"]], [W["B_o"]], saved["s_o"], [dx1])
    ga = A.attention_bwd(saved["qr"], saved["kr"], saved["qkv"][2], saved["o"], saved["s_att"], go["dx"], b, s, H, dh,
                         dh ** -0.5)
    q, k = (qk_bwd(saved["qkv"][i], rot[g], rot["theta"], ga[d], dh, rot["rot"], rot["layout"], eps)
            for i, g, d in ((0, "gq", "dq"), (1, "gk", "dk")))
    gq = O.proj_group_bwd(W["g_attn"], [W["A_q"], W["A_k"], W["A_v"]], [W["B_q"], W["B_k"], W["B_v"]],
                          saved["s_qkv"], [q["dx"], k["dx"], ga["dv"]])
    out = {"dx": dx1 + gq["dx"], "dg_attn": gq["dg"], "dg_mlp": gm["dg"]}
    for n, g in (("dgq", q), ("dgk", k)):
        if "dg" in g:
            out[n] = g["dg"]
    for i, n in enumerate("qkv"):
        out[f"dA_{n}"], out[f"dB_{n}"] = gq["dA"][i], gq["dB"][i]
    out["dA_o"], out["dB_o"] = go["dA"][0], go["dB"][0]
    for n in ("gate", "up", "down"):
        out[f"dA_{n}"], out[f"dB_{n}"] = gm[f"dA_{n}"], gm[f"dB_{n}"]
    return out
