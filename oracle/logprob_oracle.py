"""fp64 CPU oracle for the log probabilities of tokens, the entropy and the largest logits of each row.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``): only ``tests/`` imports it, and it shares no code
with the CUDA library.

z = scale logits; lse = log sum_j exp z_j, p = exp(z - lse), logp = z_target - lse (0 without a target), entropy =
-sum p log p; and of sum(dlogp logp + dentropy entropy), with H the entropy,

    dlogits_j = scale (dlogp (1[j = target] - p_j) - dentropy p_j (log p_j + H)).

A row of -inf alone has lse = -inf, entropy 0 and no gradient; a row that holds a NaN or +inf has NaN throughout.

Pins (tests/test_logprob_oracle.py): central finite differences, uniform and one-hot rows, shifts of a row.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np

F64 = np.float64

__all__ = ["fwd", "bwd", "top"]


def fwd(logits, target, scale: float) -> Dict[str, np.ndarray]:
    z = scale * np.asarray(logits, dtype=F64)
    T, V = z.shape
    target = np.asarray(target)
    out = {n: np.zeros(T) for n in ("logp", "entropy", "lse")}
    for t in range(T):
        has = 0 <= target[t] < V
        m = z[t].max()  # NaN if there is one
        if not m < np.inf:
            for x in out.values():
                x[t] = np.nan
            continue
        if m == -np.inf:
            out["lse"][t] = -np.inf
            out["logp"][t] = -np.inf if has else 0.0
            continue
        d = z[t] - m
        total = np.exp(d).sum()
        p = np.exp(d) / total
        out["lse"][t] = m + np.log(total)
        out["logp"][t] = d[target[t]] - np.log(total) if has else 0.0
        out["entropy"][t] = np.log(total) - (p[p > 0] * d[p > 0]).sum()
    return out


def bwd(logits, target, lse, entropy, dlogp, dentropy: Optional[np.ndarray], scale: float) -> Dict[str, np.ndarray]:
    """dlogits, and the magnitude of its terms."""
    z = scale * np.asarray(logits, dtype=F64)
    T, V = z.shape
    d, mag = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        if lse[t] == -np.inf:
            continue
        lp = z[t] - lse[t]
        p = np.exp(lp)
        dl = dlogp[t] if 0 <= target[t] < V else 0.0
        d[t] = -dl * p
        mag[t] = np.abs(dl) * p
        if dentropy is not None:
            live = p > 0
            d[t, live] -= dentropy[t] * p[live] * (lp[live] + entropy[t])
            mag[t, live] += np.abs(dentropy[t]) * p[live] * (np.abs(lp[live]) + entropy[t])
        if 0 <= target[t] < V:
            d[t, target[t]] += dl
            mag[t, target[t]] += np.abs(dl)
    return {"dlogits": scale * d, "mag": scale * mag}


def top(logits, k: int) -> np.ndarray:
    """Places of each row's k largest logits: NaN first, then by value, equal ones by their place."""
    x = np.asarray(logits, dtype=F64)
    key = np.where(np.isnan(x), np.inf, x)
    return np.stack([np.lexsort((np.arange(x.shape[1]), -key[t], ~np.isnan(x[t])))[:k] for t in range(x.shape[0])])
