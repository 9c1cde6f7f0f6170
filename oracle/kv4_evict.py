"""Eviction from the paged 4-bit cache: accumulated attention weights, the
choice of the tokens that stay, and their move.

Sources: none of the pages describes it; the definition is the library's own
(``include/tv.h``, "Eviction from the paged 4-bit KV cache").  Weights are in
fp64 over the values that the codes stand for; choice and move are exact.
"""
from __future__ import annotations

import numpy as np

from .kv4 import f32


def rows_of(row_off, path, r, max_rows):
    """Source rows of request r, in order."""
    if path is None:
        return list(range(int(row_off[r]), min(int(row_off[r + 1]), int(row_off[r]) + max_rows)))
    rows = []
    for j in path[r][:max_rows]:
        if j < 0:
            break
        rows.append(int(row_off[r]) + int(j))
    return rows


def attn_mass(q, lse, keys, cache_len, row_off, max_rows, score_in, columns, old_len=None, path=None, vis=None,
              causal=False, scale=None, decay=1.0, page_ok=None):
    """(score_out fp64 [B, Hkv, columns], tolerance); NaN where nothing is written.

    ``keys``: per request fp32 [tokens, Hkv, d].  The tolerance counts the
    roundings of an fp32 evaluation: a score's sum of d products is off by at
    most (d + 8) 2^-24 of sum |q k| scale, the exponent's factors and its
    rounding by 2^-22 of |score| + |lse| + 1, the base-2 exponential by 2^-22;
    the sum of n weights by n 2^-24 of itself, the decayed term by 2^-22."""
    q = f32(q).astype(np.float64)
    n, Hq, d = q.shape
    B, Hkv = len(cache_len), keys[0].shape[1]
    g = Hq // Hkv
    scale = 1.0 / np.sqrt(d) if scale is None else float(np.float32(scale))
    out = np.full((B, Hkv, columns), np.nan)
    tol = np.zeros_like(out)
    for r in range(B):
        L = int(cache_len[r])
        old = L if old_len is None else max(int(old_len[r]), 0)
        K = keys[r][:L].astype(np.float64)
        m = np.zeros((Hkv, L))
        e = np.zeros((Hkv, L))
        rows = rows_of(row_off, path, r, max_rows)
        for j, src in enumerate(rows):
            if not 0 <= src < n:
                continue
            see = min(L, old + j + 1) if causal else L
            if vis is not None:
                see = min(see, max(int(vis[src]), 0))
            for hq in range(Hq):
                l = float(lse[src, hq])
                if l == -np.inf or see == 0:
                    continue
                h = hq // g
                with np.errstate(invalid="ignore", over="ignore"):
                    s = K[:see, h] @ q[src, hq] * scale
                    w = np.exp(s - l)
                    a = np.abs(K[:see, h]) @ np.abs(q[src, hq]) * scale
                    rel = (d + 8) * 2.0 ** -24 * a + 2.0 ** -22 * (np.abs(s) + abs(l) + 2)
                    m[h, :see] += w
                    e[h, :see] += w * rel
        if page_ok is not None:
            m = np.where(page_ok[r][None, :L], m, 0.0)
        before = np.zeros((Hkv, L))
        if score_in is not None and decay != 0:
            k = min(old, L)
            before[:, :k] = np.float32(decay) * score_in[r, :, :k].astype(np.float64)
        out[r, :, :L] = before + m
        with np.errstate(invalid="ignore"):
            tol[r, :, :L] = e + (len(rows) * g * 2.0 ** -24) * m + 2.0 ** -22 * (np.abs(before) + m) + 1e-35
    return out, tol


def _order(x):
    """Sort key, highest score first: (NaN last, value descending); zeros alike."""
    x = np.asarray(x, np.float64) + 0.0
    return np.where(np.isnan(x), 1, 0), np.where(np.isnan(x), 0.0, -x)


def evict_select(score, cache_len, budget, n_sink, n_recent, idx_ld):
    """(idx int32 [B, Hkv, idx_ld], scores: list per (request, head), new_len int32 [B])."""
    B, H, _ = score.shape
    idx = np.full((B, H, idx_ld), -1, np.int32)
    kept = {}
    new_len = np.zeros(B, np.int32)
    for r in range(B):
        L = int(cache_len[r])
        n = min(L, max(int(budget[r]), 0), idx_ld)
        new_len[r] = n
        first = min(n_sink, n)
        last = min(n_recent, n - first)
        for h in range(H):
            middle = np.arange(first, L - last)
            nan, neg = _order(score[r, h, middle])
            pick = middle[np.lexsort((middle, neg, nan))[:n - first - last]]
            t = np.sort(np.concatenate([np.arange(first), pick, np.arange(L - last, L)])).astype(np.int32)
            idx[r, h, :n] = t
            kept[r, h] = score[r, h, t]
    return idx, kept, new_len
