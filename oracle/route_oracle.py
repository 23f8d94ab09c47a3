"""fp64 oracle of the router by scores: scores, selection bias, groups of
experts, top-K with the lower index first on equal keys, gates.  Token by token
in plain Python sorts; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def route_select(logits, bias, K, sigmoid, n_groups=1, keep=1, group_top=1, renorm=True, scale=1.0):
    l = np.asarray(logits, dtype=np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, FLT_MAX)
    B, E = l.shape
    size = E // n_groups
    ids = np.zeros((B, K), dtype=np.int32)
    gates = np.zeros((B, K))
    for t in range(B):
        masked = np.isneginf(l[t])
        with np.errstate(over="ignore"):
            if sigmoid:
                s = 1 / (1 + np.exp(-l[t]))
            elif masked.all():
                s = np.zeros(E)
            else:
                s = np.exp(l[t] - l[t].max())
                s /= s.sum()
        with np.errstate(invalid="ignore"):
            sel = s if bias is None else s + np.asarray(bias, dtype=np.float64)
        sel = np.where(masked | np.isnan(sel), -np.inf, sel)
        key = l[t] if bias is None else sel
        score = []
        for g in range(n_groups):
            top = sorted(sel[g * size:(g + 1) * size], reverse=True)[:group_top]
            live = [v for v in top if v != -np.inf]
            score.append(sum(live) if live else -np.inf)
        stay = sorted(range(n_groups), key=lambda g: (-score[g], g))[:keep] if n_groups > 1 else [0]
        cand = [e for e in range(E) if e // size in stay] if n_groups > 1 else range(E)
        pick = sorted(cand, key=lambda e: (-key[e], e))[:K]
        g = s[pick]
        if renorm:
            g = g / g.sum() if g.sum() > 0 else np.zeros(K)
        ids[t], gates[t] = pick, g * scale
    return ids, gates
