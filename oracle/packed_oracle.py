"""fp64 CPU oracle for causal attention over packed sequences with grouped heads.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``): only ``tests/`` imports it, and it shares no code
with the CUDA library.

Sequence i is rows offs[i] .. offs[i+1]-1; query head h reads key head h // (Hq / Hk).  Within a sequence

    S_tj = scale q_t.k_j (j <= t),  lse_t = log sum_j exp S_tj,  P = exp(S - lse),  o_t = sum_j P_tj v_j
    D_t = dout_t.o_t,  dS = scale P (dout_t.v_j - D_t)
    dq_t = sum_j dS_tj k_j,  dk_j = sum dS_tj q_t,  dv_j = sum P_tj dout_t   (over t and the group's heads)

The backward takes o and lse, as the library's does.  Rows of no sequence are NaN in every result.

Pins (tests/test_packed_oracle.py): a loop over single elements, central finite differences of every gradient, one
sequence after the other, equal heads.
"""
from __future__ import annotations

from typing import Dict, Sequence

import numpy as np

F64 = np.float64

__all__ = ["attn_fwd", "attn_bwd"]


def _heads(x, H):
    x = np.asarray(x, dtype=F64)
    return x.reshape(x.shape[0], H, -1)


def _sequences(offs: Sequence[int]):
    return [(int(b), int(e)) for b, e in zip(offs, offs[1:]) if e > b]


def _scores(q, k, scale):
    """S [n, n] of one head, -inf above the diagonal."""
    return np.where(np.tril(np.ones((len(q), len(q)), dtype=bool)), scale * (q @ k.T), -np.inf)


def attn_fwd(q, k, v, offs, Hq: int, Hk: int, scale: float) -> Dict[str, np.ndarray]:
    """o [T, Hq*dh], lse [T, Hq], and the magnitudes that rounding errors scale with: mag_o = sum P |v| and
    mag_s [T, Hq] = the largest scale sum_c |q_c k_c| of a row."""
    q, k, v = _heads(q, Hq), _heads(k, Hk), _heads(v, Hk)
    out = {"o": np.full(q.shape, np.nan), "lse": np.full(q.shape[:2], np.nan), "mag_o": np.full(q.shape, np.nan),
           "mag_s": np.full(q.shape[:2], np.nan)}
    for b, e in _sequences(offs):
        for h in range(Hq):
            hk = h * Hk // Hq
            S = _scores(q[b:e, h], k[b:e, hk], scale)
            m = S.max(1, keepdims=True)
            p = np.exp(S - m)
            total = p.sum(1, keepdims=True)
            p /= total
            out["lse"][b:e, h] = (m + np.log(total))[:, 0]
            out["o"][b:e, h] = p @ v[b:e, hk]
            out["mag_o"][b:e, h] = p @ np.abs(v[b:e, hk])
            out["mag_s"][b:e, h] = np.tril(scale * np.abs(q[b:e, h]) @ np.abs(k[b:e, hk]).T).max(1)
    return {n: x.reshape(x.shape[0], -1) for n, x in out.items()}


def attn_bwd(q, k, v, o, lse, dout, offs, Hq: int, Hk: int, scale: float, rel_p: float = 0.0, rel_s: float = 0.0,
             abs_d: float = 0.0, rel_d: float = 0.0) -> Dict[str, np.ndarray]:
    """dq, dk, dv, and bounds err_dq, err_dk, err_dv of their errors when P and dS are rounded by rel_p of themselves,
    P is off by rel_s besides, and dout.v - D by abs_d of its terms' magnitudes, o by rel_d of itself."""
    q, k, v = _heads(q, Hq), _heads(k, Hk), _heads(v, Hk)
    o, dout, lse = _heads(o, Hq), _heads(dout, Hq), np.asarray(lse, dtype=F64)
    out = {"dq": np.full(q.shape, np.nan), "dk": np.full(k.shape, np.nan), "dv": np.full(k.shape, np.nan)}
    out.update({"err_" + n: np.full(x.shape, np.nan) for n, x in list(out.items())})
    for b, e in _sequences(offs):
        for n, x in out.items():
            x[b:e] = 0.0
        for h in range(Hq):
            hk = h * Hk // Hq
            qs, ks, vs, g = q[b:e, h], k[b:e, hk], v[b:e, hk], dout[b:e, h]
            with np.errstate(over="ignore"):
                P = np.exp(_scores(qs, ks, scale) - lse[b:e, h, None])
            d = g @ vs.T - (g * o[b:e, h]).sum(1)[:, None]
            terms = np.abs(g) @ np.abs(vs).T + (np.abs(g) * np.abs(o[b:e, h])).sum(1)[:, None]
            dS = scale * P * d
            err_S = (rel_p + rel_s) * np.abs(dS) + scale * P * abs_d * terms
            err_S += scale * P * rel_d * (np.abs(g) * np.abs(o[b:e, h])).sum(1)[:, None]
            err_P = (rel_p + rel_s) * P
            out["dq"][b:e, h] = dS @ ks
            out["dk"][b:e, hk] += dS.T @ qs
            out["dv"][b:e, hk] += P.T @ g
            out["err_dq"][b:e, h] = err_S @ np.abs(ks)
            out["err_dk"][b:e, hk] += err_S.T @ np.abs(qs)
            out["err_dv"][b:e, hk] += err_P.T @ np.abs(g)
    return {n: x.reshape(x.shape[0], -1) for n, x in out.items()}
