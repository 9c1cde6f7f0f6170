"""Verification of drafted tokens at a temperature, top-k and top-p.

Graft page §2 (third gear) asks for one lossless rule for draft and retrieved
nodes; SpecOPD page §03 gives the acceptance probability under exact rejection
sampling.  The rule (reading, in full) is in ``include/tv.h``, accept_sampled:
children in index order; a child drawn from the drafter's q is accepted iff
u q(x) < p'(x), and a rejection leaves max(0, p' - q); a child proposed without
a distribution is accepted iff u < p'(x), and a rejection removes its token; the
bonus token maximises p'(v) / race(v).  Arithmetic: float64.
"""
from __future__ import annotations

import numpy as np

from .sampling import _row


def target_probs(logits, temperature=1.0, top_k=0, top_p=1.0):
    """The target's distribution over one row (zeros if no logit is above -inf)."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    p = np.zeros(x.size)
    if x.max() == -np.inf:
        return p
    if not temperature > 0:
        p[int(np.argmax(x))] = 1.0
        return p
    x = np.minimum(x, np.finfo(np.float32).max)
    keep = np.ones(x.size, bool)
    if 0 < top_k < x.size:
        keep = x >= np.sort(x)[::-1][top_k - 1]
    w = np.where(keep, np.exp((x - x.max()) / temperature), 0.0)
    if top_p < 1:
        value, group = np.unique(x, return_inverse=True)
        mass = np.bincount(group, weights=w)
        above = mass.sum() - np.cumsum(mass)                   # mass of the higher classes
        on = above < top_p * mass.sum()
        on[-1] = True
        w = np.where(on[group], w, 0.0)
    return w / w.sum()


def verify(parent, tok, p_logits, node_off, u_node, race, max_depth, q_prob=None, drawn=None, temperature=None, top_k=None,
           top_p=None):
    """accept_len, best_node int32 [B], path int32 [B, max_depth + 1], bonus int32 [B], and per request the smallest
    relative distance between the two sides of a comparison that it took (decisions nearer than an implementation's
    rounding may go either way)."""
    B = len(node_off) - 1
    acc, best, bonus = (np.full(B, -1, np.int32) for _ in range(3))
    path = np.full((B, max_depth + 1), -1, np.int32)
    margin = np.full(B, np.inf)
    for r in range(B):
        a, n = int(node_off[r]), int(node_off[r + 1] - node_off[r])
        if n == 0:
            continue
        T = 1.0 if temperature is None else float(temperature[r])
        k = 0 if top_k is None else int(top_k[r])
        tp = 1.0 if top_p is None else float(top_p[r])
        cur, depth = 0, 0
        path[r, 0] = 0
        while True:
            p = target_probs(_row(p_logits, a + cur), T, k, tp)
            left, nxt = p.copy(), -1
            for c in range(1, n):
                if int(parent[a + c]) != cur:
                    continue
                x = int(tok[a + c])
                inside = 0 <= x < p.size
                is_drawn = q_prob is not None and (drawn is None or bool(drawn[a + c]))
                px = left[x] if inside else 0.0
                if not T > 0:
                    if px > 0:
                        nxt = c
                        break
                    continue
                side = float(u_node[a + c]) * ((float(q_prob[a + cur, x]) if inside else 0.0) if is_drawn else 1.0)
                if max(side, px) > 0:
                    margin[r] = min(margin[r], abs(side - px) / max(side, px))
                if side < px:
                    nxt = c
                    break
                if is_drawn:
                    left = np.maximum(0.0, left - np.asarray(q_prob[a + cur], np.float64))
                elif inside:
                    left[x] = 0.0
                s = left.sum()
                left = left / s if s > 0 else p.copy()
            if nxt < 0:
                with np.errstate(divide="ignore", invalid="ignore"):
                    f = np.where(left > 0, left / race[r].astype(np.float64), 0.0)
                order = np.sort(f)[::-1]
                if order[0] > 0:
                    bonus[r] = int(np.argmax(f))
                    if T > 0 and f.size > 1:
                        margin[r] = min(margin[r], 1 - order[1] / order[0] if np.isfinite(order[0]) else np.inf)
                break
            cur, depth = nxt, depth + 1
            if depth <= max_depth:
                path[r, depth] = cur
        acc[r], best[r] = depth, cur
    return acc, best, path, bonus, margin
