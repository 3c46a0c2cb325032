"""Log probabilities of given tokens, entropy and top alternatives, in float64 (TEST INFRASTRUCTURE
ONLY, see the package docstring).  Rows whose token is outside the vocabulary are not scored."""
from __future__ import annotations

import numpy as np


def logprobs(logits, tokens, temperature=1.0, top_n=0):
    z = np.asarray(logits, np.float64)
    R, V = z.shape
    lp = np.zeros(R)
    H = np.zeros(R)
    ids = np.full((R, top_n), -1, np.int64)
    top = np.full((R, top_n), -np.inf)
    for r in range(R):
        t = int(tokens[r])
        if t < 0 or t >= V:
            continue
        if np.isnan(z[r]).any() or np.isposinf(z[r]).any() or np.isneginf(z[r]).all():
            lp[r] = H[r] = np.nan
            top[r] = np.nan
            continue
        x = z[r] / temperature
        x = x - x.max()
        with np.errstate(divide="ignore"):
            l = x - np.log(np.exp(x).sum())
        p = np.exp(l)
        lp[r] = l[t]
        H[r] = -(p[p > 0] * l[p > 0]).sum()
        order = np.lexsort((np.arange(V), -z[r]))[:top_n]
        ids[r], top[r] = order, l[order]
    return lp, H, ids, top
