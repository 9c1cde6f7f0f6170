"""The paged 4-bit KV cache and what is done with it: rotation, quantisation,
append, read-back, and attention over it.

Sources: none of the pages describes a cache format; the definition is the
library's own (``include/tv.h``, "Paged 4-bit KV cache").  Rotation and
quantisation are defined in fp32 with each operation rounded by itself, so
they are restated here in NumPy float32 and compared bit for bit; attention is
in fp64 over the values that the codes stand for.

Blocks are packed and unpacked item by item through an explicit (byte, nibble)
address, not by the word shuffles that the kernels use.
"""
from __future__ import annotations

import numpy as np

SCALE_MIN = np.float32(2.0 ** -100)


def f32(x) -> np.ndarray:
    """Widen raw bf16 patterns (uint16) or pass fp32 through."""
    x = np.asarray(x)
    if x.dtype == np.uint16:
        return (x.astype(np.uint32) << np.uint32(16)).view(np.float32)
    return x.astype(np.float32)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """float32 -> bf16 bits, nearest even; NaN stays NaN."""
    x = np.ascontiguousarray(x, np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


# ------------------------------------------------------------------ rotation
def rope_table(max_pos: int, rot: int, base: float = 10000.0) -> np.ndarray:
    inv = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    ang = np.arange(max_pos, dtype=np.float64)[:, None] * inv[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rotate(x: np.ndarray, pos, table: np.ndarray | None, interleaved: bool) -> np.ndarray:
    """x [n, H, d] -> float32, pair by pair."""
    y = f32(x).copy()
    if table is None or table.shape[1] == 0:
        return y
    half = table.shape[1] // 2
    for t, p in enumerate(np.asarray(pos)):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = table[p, i], table[p, half + i]
            xa, xb = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a] = xa * c - xb * s
            y[t, :, b] = xb * c + xa * s
    return y


# -------------------------------------------------------------- quantisation
def row_scale(x: np.ndarray) -> np.ndarray:
    """Scale of each row of float32 x [..., d]."""
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(x).max(-1).astype(np.float32)
    out = np.empty(a.shape, np.float32)
    flat, o = a.reshape(-1), out.reshape(-1)
    for i, v in enumerate(flat):
        if not np.isfinite(v):
            o[i] = np.nan
            continue
        t = np.float32(v / np.float32(7.0))
        bits = int(t.view(np.uint32))
        up = bits if bits % 65536 == 0 else (bits // 65536 + 1) * 65536
        o[i] = max(np.uint32(up).view(np.float32), SCALE_MIN)
    return out


def quantise(x: np.ndarray):
    """float32 rows [..., d] -> (n int64 in -7..7, scale float32)."""
    s = row_scale(x)
    with np.errstate(invalid="ignore"):
        n = np.rint((x / s[..., None]).astype(np.float32))
    n = np.where(np.isfinite(n), n, 0)
    return np.clip(n, -7, 7).astype(np.int64), s


def values(n, s):
    return n.astype(np.float32) * s[..., None].astype(np.float32)


# -------------------------------------------------------------------- blocks
def _k_at(P, slot, dim):
    """(byte, shift) of key dim ``dim`` of token ``slot``."""
    e = dim % 8
    nib = e // 2 + 4 * (e % 2)
    return (dim // 32) * P * 16 + slot * 16 + (dim % 32) // 8 * 4 + nib // 2, 4 * (nib % 2)


def _v_at(P, d, slot, dim):
    e = slot % 8
    nib = e // 2 + 4 * (e % 2)
    return P * d // 2 + (slot // 16 * d + dim) * 8 + (slot % 16) // 8 * 4 + nib // 2, 4 * (nib % 2)


def write_row(block: np.ndarray, P: int, d: int, slot: int, kn, ks, vn, vs):
    """Writes one token of one head into its block (uint8 [P * (d + 4)])."""
    for dim in range(d):
        for (byte, sh), n in ((_k_at(P, slot, dim), kn[dim]), (_v_at(P, d, slot, dim), vn[dim])):
            block[byte] = (int(block[byte]) & ~(15 << sh) & 255) | (int(n + 8) << sh)
    for off, s in ((P * d, ks), (P * d + 2 * P, vs)):
        b = int(bf16_bits(np.array([s], np.float32))[0])
        block[off + 2 * slot], block[off + 2 * slot + 1] = b & 255, b >> 8


def read_block(block: np.ndarray, P: int, d: int):
    """(kn, ks, vn, vs) of a block: int64 [P, d], float32 [P]."""
    slot, dim = np.meshgrid(np.arange(P), np.arange(d), indexing="ij")
    out = []
    for at, off in ((_k_at(P, slot, dim), P * d), (_v_at(P, d, slot, dim), P * d + 2 * P)):
        n = ((block[at[0]].astype(np.int64) >> at[1]) & 15) - 8
        b = block[off:off + 2 * P].astype(np.uint16)
        s = ((b[0::2] | (b[1::2] << np.uint16(8))).astype(np.uint32) << np.uint32(16)).view(np.float32)
        out += [n, s]
    return out


def append(cache, P, table, cache_len, k, v, row_off, path=None, pos=None, rope=None, interleaved=False):
    """Appends in place; returns new_len.  Rows whose page is bad are skipped."""
    Hkv, d = cache.shape[1], cache.shape[2] // P - 4
    new_len = np.array(cache_len, np.int32).copy()
    for r in range(len(cache_len)):
        if path is None:
            rows = list(range(int(row_off[r]), int(row_off[r + 1])))
        else:
            rows = []
            for j in path[r]:
                if j < 0:
                    break
                rows.append(int(row_off[r]) + int(j))
        for j, src in enumerate(rows):
            t = int(cache_len[r]) + j
            new_len[r] += 1
            page = int(table[r, t // P]) if t // P < table.shape[1] else -1
            if not 0 <= page < cache.shape[0]:
                continue
            p = t if pos is None else int(pos[src])
            kr = rotate(k[src:src + 1], [p], rope, interleaved)[0]
            kn, ks = quantise(kr)
            vn, vs = quantise(f32(v[src]))
            for h in range(Hkv):
                write_row(cache[page, h], P, d, t % P, kn[h], ks[h], vn[h], vs[h])
    return new_len


def gather(cache, P, table, start, count):
    """Per request (K, V) float32 [count, Hkv, d] of tokens start .. start+count-1."""
    Hkv, d = cache.shape[1], cache.shape[2] // P - 4
    out = []
    for r in range(len(count)):
        K = np.zeros((count[r], Hkv, d), np.float32)
        V = np.zeros_like(K)
        blocks = {}
        for i in range(count[r]):
            t = int(start[r]) + i
            page = int(table[r, t // P])
            if page not in blocks:
                blocks[page] = [read_block(cache[page, h], P, d) for h in range(Hkv)]
            for h in range(Hkv):
                kn, ks, vn, vs = blocks[page][h]
                with np.errstate(over="ignore", invalid="ignore"):      # stale slots may hold any scale
                    K[i, h] = kn[t % P].astype(np.float32) * ks[t % P]
                    V[i, h] = vn[t % P].astype(np.float32) * vs[t % P]
        out.append((K, V))
    return out


# ----------------------------------------------------------------- attention
def attention(q, prefix, k_tree, v_tree, node_off, see, vis=None, node_cnt=None, scale=None, page_ok=None):
    """Attention of every node over what it sees.

    prefix: per request (K, V) values; ``see`` bool [n, max_nodes], the
    ancestor relation in request-local indices; ``page_ok``: per request a
    bool per token, False where the token's page is bad.  Returns out, lse
    (NaN rows: not computed), and per output the two sums that bound rounding:
    sum_j w_j |v_j| [n, Hq, d] and max_j scale * sum_i |q_i k_ji| [n, Hq]."""
    q, k_tree, v_tree = (f32(x).astype(np.float64) for x in (q, k_tree, v_tree))
    n, Hq, d = q.shape
    Hkv = k_tree.shape[1]
    g = Hq // Hkv
    scale = 1.0 / np.sqrt(d) if scale is None else float(np.float32(scale))
    out = np.full((n, Hq, d), np.nan)
    lse = np.full((n, Hq), np.nan)
    absv = np.zeros((n, Hq, d))
    abss = np.zeros((n, Hq))
    for r in range(len(node_off) - 1):
        n0, n1 = int(node_off[r]), int(node_off[r + 1])
        cnt = n1 - n0 if node_cnt is None else int(node_cnt[r])
        K, V = (x.astype(np.float64) for x in prefix[r])
        for i in range(cnt):
            gi = n0 + i
            m = len(K) if vis is None else min(max(int(vis[gi]), 0), len(K))
            t = np.arange(m)
            if page_ok is not None:
                t = t[page_ok[r][:m]]
            js = n0 + np.nonzero(see[gi, :cnt])[0]
            keys = np.concatenate([K[t], k_tree[js]])
            vals = np.concatenate([V[t], v_tree[js]])
            for h in range(Hq):
                if len(keys) == 0:
                    out[gi, h], lse[gi, h] = 0.0, -np.inf
                    continue
                kh, vh = keys[:, h // g], vals[:, h // g]
                with np.errstate(invalid="ignore"):
                    s = kh @ q[gi, h] * scale
                    w = np.exp(s - s.max())
                    lse[gi, h] = s.max() + np.log(w.sum())
                    w /= w.sum()
                    out[gi, h] = w @ vh
                    absv[gi, h] = w @ np.abs(vh)
                    abss[gi, h] = (np.abs(kh) @ np.abs(q[gi, h])).max() * scale
    return out, lse, absv, abss


def attention_tolerance(out, lse, absv, abss, d, bf16):
    """Bounds on |out| and |lse| errors.

    A score is a sum of d fp32 products: off by at most (d + 8) 2^-24 of
    sum |q k| scale (products, sums, the scale factors); a weight by twice that
    relatively (its own score and the normaliser's) plus 2^-20 for the base-2
    exponential, its argument's rounding and the summation.  bf16 rows: each
    weight times the value's scale is rounded to bf16 (at most 2^-8), and the
    output once more."""
    ds = (d + 8) * 2.0 ** -24 * abss + 2.0 ** -20
    tol = absv * (2 * ds[..., None] + (2.0 ** -8 if bf16 else 0.0))
    tol = tol + (np.abs(out) + tol) * (2.0 ** -8 if bf16 else 2.0 ** -22) + 1e-30
    return tol, ds + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
