"""GPU parity of eviction from the paged 4-bit cache (kv4_attn_mass,
kv4_evict_select, kv4_compact) against oracle/kv4_evict.py: choice and move
exactly, weights within the tolerance derived there."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from oracle import kv4 as ok
from oracle import kv4_evict as oe
from oracle import sampled as osm
from test_gpu_kv4 import act, bits, forest, fused, prefixes, random_pool, tables

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


# -------------------------------------------------------------------- weights
class Mass:
    """One kv4_attn_mass call and what the oracle says about it."""

    def __init__(self, seed, lens, counts, Hq, Hkv, d, P, bf16=True, path=False, causal=True, vis=False, decay=1.0,
                 score=True, scale=None):
        rng = np.random.default_rng(seed)
        self.rng, self.P, self.lens, self.decay, self.scale, self.causal = rng, P, list(lens), decay, scale, causal
        self.table, n_pages = tables(rng, lens, P)
        self.pool = random_pool(rng, n_pages, Hkv, P, d)
        held = [c + 2 if path else c for c in counts]
        self.off = np.concatenate([[0], np.cumsum(held)]).astype(np.int32)
        n = int(self.off[-1])
        (self.q, _, _), (self.hq, _, _) = fused(rng, n, Hq, Hkv, d, bf16)
        self.path = None
        if path:
            self.path = np.full((len(lens), max(counts) + 1), -1, np.int32)
            for r, c in enumerate(counts):
                self.path[r, :c] = np.sort(rng.permutation(held[r])[:c])
        self.old = np.array([max(0, m - c) for m, c in zip(lens, counts)], np.int32)
        self.vis = rng.integers(-2, max(max(lens), 1) + 3, n).astype(np.int32) if vis else None
        self.max_rows = max(max(counts), 1)
        # of the size that an attention over this many tokens gives; some rows saw nothing
        self.lse = (np.log(max(max(lens), 1)) + rng.standard_normal((n, Hq))).astype(np.float32)
        if n > 3:
            self.lse[2] = -INF
        self.cols = max(lens) + 5
        self.score = rng.random((len(lens), Hkv, self.cols), np.float32) if score else None
        self.page_ok = None

    def keys(self):
        return [k for k, _ in prefixes(self.pool, self.table, self.lens, self.P)]

    def run(self, tv, **kw):
        args = dict(score=dev(self.score), old_len=dev(self.old), path=dev(self.path), vis_prefix=dev(self.vis),
                    causal=self.causal, scale=self.scale, decay=self.decay) | kw
        if args["score"] is None and "score_out" not in args:
            args["score_out"] = torch.full((len(self.lens), self.pool[0].shape[1], self.cols), -7.0, device="cuda")
        return tv.kv4_attn_mass(self.q, dev(self.lse), dev(self.pool[0]), self.P, dev(self.table),
                                dev(np.array(self.lens, np.int32)), dev(self.off), self.max_rows, **args)

    def check(self, out, before=None):
        want, tol = oe.attn_mass(self.hq, self.lse, self.keys(), self.lens, self.off, self.max_rows, self.score, self.cols,
                                 self.old, self.path, self.vis, self.causal, self.scale, self.decay, self.page_ok)
        got = host(out).astype(np.float64)
        for r, L in enumerate(self.lens):
            w, t, x = want[r, :, :L], tol[r, :, :L], got[r, :, :L]
            assert np.array_equal(np.isnan(w), np.isnan(x))
            m = ~np.isnan(w)
            assert (np.abs(x - w)[m] <= t[m]).all(), np.nanmax(np.abs(x - w)[m] / t[m])
            rest = got[r, :, L:]
            assert (rest == (0.0 if before is None else host(before)[r, :, L:])).all()      # not written


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("lens,counts,Hq,Hkv,d,P,kw", [
    ([1], [1], 1, 1, 64, 16, {}),
    ([128], [60], 4, 1, 64, 16, {}),
    ([300, 0, 17, 129], [1, 1, 1, 1], 8, 2, 128, 64, dict(decay=0.5)),
    ([40, 257, 33], [0, 16, 5], 8, 8, 128, 16, dict(path=True)),
    ([64, 200], [7, 64], 14, 2, 64, 32, dict(causal=False, vis=True, score=False)),
    ([131, 90], [33, 21], 16, 1, 128, 128, dict(vis=True, decay=0.0, scale=0.31)),
    ([500], [200], 12, 3, 64, 64, dict()),
    ([129], [129], 1, 1, 128, 16, dict()),
    ([1100, 0, 513], [300, 0, 513], 8, 2, 128, 32, dict(decay=0.5)),
    ([260, 40], [150, 40], 10, 2, 64, 16, dict(path=True, vis=True)),
    ([700], [90], 128, 2, 64, 64, dict(causal=False)),
    ([610], [600], 16, 1, 64, 32, dict()),
    ([300, 61], [48, 48], 8, 2, 128, 64, dict()),                # the most rows of the kernel for few
    ([300, 61], [49, 49], 8, 2, 128, 64, dict()),
    ([90, 35], [20, 35], 6, 2, 128, 32, dict(path=True, vis=True)),
])
def test_mass_matches(tv, lens, counts, Hq, Hkv, d, P, kw, bf16):
    m = Mass(sum(lens) + Hq, lens, counts, Hq, Hkv, d, P, bf16, **kw)
    start = torch.full((len(lens), Hkv, m.cols), 3.25, device="cuda")
    out, err = m.run(tv, score_out=start.clone())
    m.check(out, start)
    assert int(err) == 0
    again, _ = m.run(tv, score_out=start.clone())
    assert torch.equal(torch.nan_to_num(again), torch.nan_to_num(out))


def test_mass_in_place_and_strided_rows(tv):
    m = Mass(5, [150, 70], [16, 9], 8, 2, 128, 64)
    s = dev(m.score)
    out, err = m.run(tv, score=s, score_out=s)
    assert out.data_ptr() == s.data_ptr() and int(err) == 0
    m.check(out, dev(m.score))


def test_mass_bad_pages_rows_and_bounds(tv):
    m = Mass(6, [100, 50], [8, 8], 4, 2, 64, 16, causal=False)
    m.table[0, 2], m.table[1, 0] = -1, 10 ** 6
    m.page_ok = [np.arange(100) // 16 != 2, np.arange(50) // 16 != 0]
    out, err = m.run(tv)
    assert int(err) == 1
    want, tol = oe.attn_mass(m.hq, m.lse, m.keys(), m.lens, m.off, 8, m.score, m.cols, m.old, None, None, False,
                             page_ok=m.page_ok)
    for r, L in enumerate(m.lens):
        assert (np.abs(host(out)[r, :, :L] - want[r, :, :L]) <= tol[r, :, :L]).all()
    # tokens past max_len are not touched; rows past max_rows are left out; rows outside the tensor give nothing
    m = Mass(7, [100], [8], 4, 2, 64, 16, causal=False)
    before = torch.full((1, 2, m.cols), 9.0, device="cuda")
    out, err = m.run(tv, max_len=70, score_out=before.clone())
    assert int(err) == 1 and bool((out[:, :, 70:] == 9).all())
    m.max_rows = 5
    out, err = m.run(tv)
    assert int(err) == 1
    m.off = np.array([0, 5], np.int32)
    m.check(out)
    m = Mass(8, [60], [4], 4, 2, 64, 16, path=True, causal=False)
    m.path[0, :4] = [1, 100, 0, 3]
    out, err = m.run(tv)
    m.check(out)
    assert int(err) == 1


def test_mass_without_rows_or_pages_only_decays(tv):
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    s = torch.rand(1, 2, 40, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        for pages, table in ((3, [[0, 1, 2]]), (0, [[0, 1, 2]])):
            q = torch.zeros((0, 4, 64), dtype=dt, device="cuda")
            cache = torch.zeros((pages, 2, 16 * 68), dtype=torch.uint8, device="cuda")
            out, err = tv.kv4_attn_mass(q, torch.zeros(0, 4, device="cuda"), cache, 16, i32(*table), i32(40), i32(0, 0), 4,
                                        score=s, decay=0.5)
            assert torch.equal(out, 0.5 * s) and int(err) == (pages == 0)


def test_mass_nan_reaches_only_what_sees_it(tv):
    for bf16 in (True, False):
        m = Mass(9, [90], [6], 4, 2, 64, 16, bf16, causal=False, vis=True)
        m.vis[:] = [30, 60, 10, 60, 90, 0]
        m.lse[2] = 1.0
        m.lse[5] = NAN                                   # sees nothing
        cache, kn, ks, vn, vs = m.pool
        page, slot = m.table[0, 70 // 16], 70 % 16       # a key whose scale is NaN, seen by row 4 alone
        cache[page, 1, 16 * 64 + 2 * slot:16 * 64 + 2 * slot + 2] = [0xC0, 0x7F]
        ks[page, 1, slot] = NAN
        out, err = m.run(tv)
        m.check(out)
        assert int(err) == 0 and bool(out[0, 1, 70].isnan()) and int(out.isnan().sum()) == 1
        m.lse[1, 3] = NAN                                # a row of KV head 1 that sees 60 tokens
        out, _ = m.run(tv)
        m.check(out)
        assert bool(out[0, 1, :60].isnan().all()) and not bool(out[0, 0].isnan().any())


def test_mass_agrees_with_the_attention(tv):
    """Weights of all rows over everything they see sum to one per head: prefix alone (an empty tree row has no such
    thing, so the tree's own share is what is missing)."""
    rng = np.random.default_rng(10)
    lens, N, Hq, Hkv, d, P = [700, 130], 16, 8, 2, 128, 64
    table, n_pages = tables(rng, lens, P)
    pool = random_pool(rng, n_pages, Hkv, P, d)
    _, off, anc, _ = forest(rng, [N, N], "chain")
    (q, k, v), _ = fused(rng, 2 * N, Hq, Hkv, d, True)
    clen = dev(np.array(lens, np.int32))
    # a tree whose keys weigh nothing: their products are far below the prefix's
    k = torch.zeros_like(k) - 0.0
    out, lse, _ = tv.tree_verify_attn_kv4(q, dev(pool[0]), P, dev(table), clen, k, v, dev(off), dev(anc.view(np.int64)), N)
    s, err = tv.kv4_attn_mass(q, lse, dev(pool[0]), P, dev(table), clen, dev(off), N, max_len=700)
    depth = np.tile(np.arange(1, N + 1), 2)                                     # tree keys of weight exp(0 - lse)
    share = 1 - (depth[:, None] * np.exp(-host(lse).astype(np.float64)))
    for r in range(2):
        want = share[N * r:N * r + N].reshape(N, Hkv, -1).sum((0, 2))
        got = host(s)[r, :, :lens[r]].astype(np.float64).sum(-1)
        assert np.abs(got - want).max() <= 2.0 ** -16 * N * Hq and int(err) == 0


# --------------------------------------------------------------------- choice
@pytest.mark.parametrize("lens,budget,sink,recent,kind", [
    ([1], [1], 0, 0, "float"), ([5, 0, 9], [3, 4, 20], 1, 1, "float"), ([4000, 333, 1024], [700, 333, 1023], 4, 128, "ties"),
    ([4097, 12], [2048, 1], 3, 4000, "float"), ([9000, 8193], [1, 5000], 0, 0, "ties"), ([40000], [12345], 17, 100, "wild"),
    ([131072, 77], [16384, 50], 4, 1024, "wild"), ([300], [0], 4, 4, "wild"), ([300] * 70, [37] * 70, 4, 4, "same"),
    ([393216], [70001], 4, 1000, "float")])
def test_select_matches(tv, lens, budget, sink, recent, kind):
    rng = np.random.default_rng(sum(lens))
    H, ld = 2, max(lens) + 3
    x = np.exp(3 * rng.standard_normal((len(lens), H, ld))).astype(np.float32)
    if kind == "ties":
        x = rng.integers(0, 5, x.shape).astype(np.float32)
    elif kind == "same":
        x[:] = 0.0
    elif kind == "wild":
        u = rng.random(x.shape)
        for i, v in enumerate([NAN, INF, -INF, 0.0, -0.0, -1.5, 1e-42]):
            x[(u > i / 20) & (u < (i + 1) / 20)] = v
    keep = max(1, max(min(a, b) for a, b in zip(lens, budget)))
    idx, kept, new_len = oe.evict_select(x, lens, budget, sink, recent, keep)
    i32 = lambda a: dev(np.array(a, np.int32))  # noqa: E731
    t, s, n, err = tv.kv4_evict_select(dev(x), i32(lens), i32(budget), max(lens), sink, recent, max_keep=keep)
    assert np.array_equal(host(t), idx) and np.array_equal(host(n), new_len) and int(err) == 0
    same = dev(x)
    t2, s2, _, _ = tv.kv4_evict_select(same, i32(lens), i32(budget), max(lens), sink, recent, max_keep=keep, score_out=same)
    assert torch.equal(t2, t)
    for (r, h), v in kept.items():
        assert np.array_equal(bits(s[r, h, :len(v)]), v.view(np.int32))
        assert np.array_equal(bits(s2[r, h, :len(v)]), v.view(np.int32))
        assert np.array_equal(bits(s2[r, h, len(v):]), x[r, h, len(v):].view(np.int32))      # left as they were


def test_select_bad_lengths_and_budgets(tv):
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    x = torch.rand(4, 1, 50, device="cuda")
    t, _, n, err = tv.kv4_evict_select(x, i32(-3, 51, 40, 40), i32(5, 5, -2, 20), 50, max_keep=8)
    assert int(err) == 1 and n.tolist() == [-3, 51, 0, 8]
    assert bool((t[:3] == -1).all()) and bool((t[3] >= 0).all())


# ----------------------------------------------------------------------- move
def codes(tv, cache, P, table, lens):
    """Cached values of every request, float32 [tokens, Hkv, d] pairs."""
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v, err = tv.kv4_gather(cache, P, dev(table), dev(off), max(max(lens), 1), total_rows=int(off[-1]),
                              dtype=torch.float32)
    assert int(err) == 0
    return [(k[a:b], v[a:b]) for a, b in zip(off, off[1:])]


def choose(rng, lens, kept, H, cols):
    idx = np.full((len(lens), H, cols), -1, np.int32)
    for r, (n, k) in enumerate(zip(lens, kept)):
        for h in range(H):
            idx[r, h, :k] = np.sort(rng.permutation(n)[:k])
    return idx


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,kept,H,d,P", [
    ([1], [1], 1, 64, 16), ([40, 0, 33], [13, 0, 33], 2, 64, 16), ([500, 129], [100, 128], 3, 128, 64),
    ([5000, 300], [4100, 7], 2, 64, 128), ([9000], [4000], 1, 128, 32), ([700] * 40, [333] * 40, 8, 64, 64)])
def test_compact_matches(tv, lens, kept, H, d, P, in_place):
    rng = np.random.default_rng(sum(lens) + d)
    pages = [(k + P - 1) // P for k in kept]
    table, n_pages = tables(rng, lens, P, spare=sum(pages) + 1)
    free = np.setdiff1d(np.arange(n_pages), table.ravel())
    dst = np.full((len(lens), max(pages) + 1), -1, np.int32)
    for r, u in enumerate(pages):
        dst[r, :u] = free[sum(pages[:r]):sum(pages[:r]) + u]
    pool = random_pool(rng, n_pages, H, P, d)
    cache = dev(pool[0])
    idx = choose(rng, lens, kept, H, max(kept) + 2)
    i32 = lambda a: dev(np.array(a, np.int32))  # noqa: E731
    was = codes(tv, cache, P, table, lens)
    err = tv.kv4_compact(cache, P, dev(table), i32(lens), dev(idx), i32(kept), max(kept),
                         dst_table=None if in_place else dev(dst))
    assert int(err) == 0
    now = codes(tv, cache, P, table if in_place else dst, kept)
    for r, k in enumerate(kept):
        t = torch.from_numpy(idx[r, :, :k].astype(np.int64)).cuda()
        for a, b in zip(was[r], now[r]):
            assert torch.equal(torch.stack([a[t[h], h] for h in range(H)], 1), b)
    if in_place:                                             # tokens behind the kept ones are left as they were
        for r, (a, b) in enumerate(zip(was, codes(tv, cache, P, table, lens))):
            assert torch.equal(a[0][kept[r]:], b[0][kept[r]:]) and torch.equal(a[1][kept[r]:], b[1][kept[r]:])
    else:                                                    # sources, and the rest of the last page
        for a, b in zip(was, codes(tv, cache, P, table, lens)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        full = [u * P for u in pages]
        old = codes(tv, dev(pool[0]), P, dst, full)
        for r, (a, b) in enumerate(zip(old, codes(tv, cache, P, dst, full))):
            assert torch.equal(a[0][kept[r]:], b[0][kept[r]:]) and torch.equal(a[1][kept[r]:], b[1][kept[r]:])


def test_compact_skips_what_is_bad(tv):
    rng = np.random.default_rng(3)
    P, H, d = 16, 2, 64
    table, n_pages = tables(rng, [64], P, spare=3)
    free = np.setdiff1d(np.arange(n_pages), table.ravel())
    pool = random_pool(rng, n_pages, H, P, d)
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    dst = np.array([[free[0], 10 ** 6, free[1]]], np.int32)
    idx = choose(rng, [64], [48], H, 48)
    idx[0, 0, 3], idx[0, 1, 40] = 64, -5
    src = table.copy()
    src[0, 1] = -1
    cache = dev(pool[0])
    err = tv.kv4_compact(cache, P, dev(src), i32(64), dev(idx), i32(48), 48, dst_table=dev(dst))
    assert int(err) == 1
    a = codes(tv, dev(pool[0]), P, table, [64])[0]
    for page, j0 in ((0, 0), (2, 32)):
        t = np.array([[dst[0, page]]], np.int32)
        new, old = codes(tv, cache, P, t, [16])[0], codes(tv, dev(pool[0]), P, t, [16])[0]
        for x, y, z in zip(a, new, old):
            for h in range(H):
                for j in range(16):
                    s = idx[0, h, j0 + j]
                    moved = 0 <= s < 64 and not 16 <= s < 32
                    assert torch.equal(y[j, h], x[s, h] if moved else z[j, h])
    # the request's own table as the destination is in place
    cache, same = dev(pool[0]), dev(pool[0])
    idx = choose(rng, [64], [48], H, 48)
    t = dev(table)
    assert int(tv.kv4_compact(cache, P, t, i32(64), dev(idx), i32(48), 48, dst_table=t)) == 0
    assert int(tv.kv4_compact(same, P, t, i32(64), dev(idx), i32(48), 48)) == 0
    assert torch.equal(cache, same)
    # more than max_keep: the first max_keep
    cache = dev(pool[0])
    err = tv.kv4_compact(cache, P, dev(table), i32(64), dev(idx), i32(48), 20)
    now = codes(tv, cache, P, table, [64])[0]
    assert int(err) == 1
    for h in range(H):
        assert torch.equal(now[0][:20, h], a[0][torch.from_numpy(idx[0, h, :20].astype(np.int64)).cuda(), h])
        assert torch.equal(now[0][20:, h], a[0][20:, h])


def test_pages_beyond_four_gigabytes(tv):
    """The same tokens on the last pages of a cache of 5.4 GB: weights on every path and the move are the same."""
    m = Mass(40, [300, 130], [60, 20], 8, 2, 128, 128)
    small = m.pool[0]
    far = 160000
    cache = torch.empty((far + len(small), 2, 128 * 132), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    table = np.where(m.table >= 0, m.table + far, m.table).astype(np.int32)
    i32 = lambda a: dev(np.array(a, np.int32))  # noqa: E731
    idx = choose(np.random.default_rng(0), m.lens, [100, 77], 2, 100)
    for q, rows in ((m.q, 60), (m.q, 8), (m.q.float(), 60)):
        out = []
        for c, t, base in ((dev(small), m.table, 0), (cache, table, far)):
            c[base:base + len(small)] = dev(small)
            s, err = tv.kv4_attn_mass(q, dev(m.lse), c, 128, dev(t), i32(m.lens), dev(m.off), rows, max_len=300)
            assert int(err) == int(rows == 8)
            e = tv.kv4_compact(c, 128, dev(t), i32(m.lens), dev(idx), i32([100, 77]), 100)
            assert int(e) == 0
            out.append((s, c[base:base + len(small)].clone()))
        assert torch.equal(torch.nan_to_num(out[0][0]), torch.nan_to_num(out[1][0])) and torch.equal(out[0][1], out[1][1])


# ------------------------------------------------------------------- together
def serve(tv, d, steps, graph=False):
    """Verification steps of two requests that go over their budget: attention, sampled acceptance, append, weights,
    eviction.  The oracle keeps a cache of its own."""
    rng = np.random.default_rng(d)
    B, N, Hq, Hkv, P, V, budget = 2, 6, 4, 2, 16, 64, 40
    counts = [38, 29]
    rope = ok.rope_table(256, d)
    off0 = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    table = np.array([[7, 2, 9, 0], [5, 1, 3, 8]], np.int32)
    kx = ok.f32(ok.bf16_bits(rng.standard_normal((sum(counts), 2, Hkv, d)).astype(np.float32)))
    bf = lambda x: dev(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)  # noqa: E731
    i32 = lambda a: dev(np.array(a, np.int32))  # noqa: E731
    cache = tv.kv4_new_cache(10, P, Hkv, d)
    clen, err = tv.kv4_append(bf(kx[:, 0]), bf(kx[:, 1]), cache, P, dev(table), i32([0, 0]), dev(off0), max(counts),
                              rope=dev(rope))
    ocache = np.zeros((10, Hkv, P * (d + 4)), np.uint8)
    olen = ok.append(ocache, P, table, np.zeros(B, np.int32), kx[:, 0], kx[:, 1], off0, rope=rope)
    score = torch.zeros(B, Hkv, 64, device="cuda")
    oscore = np.zeros((B, Hkv, 64))
    slack = np.zeros((B, Hkv, 64))
    position = np.array(counts)
    par = np.tile(np.array([-1, 0, 1, 1, 0, 4], np.int32), B)
    node = np.array([0, N, 2 * N], np.int32)
    see = np.zeros((2 * N, N), bool)
    for r in range(B):
        for i in range(N):
            j = i
            while j >= 0:
                see[r * N + i, j] = True
                j = par[j]
    for _ in range(steps):
        x = ok.f32(ok.bf16_bits(rng.standard_normal((2 * N, Hq + 2 * Hkv, d)).astype(np.float32)))
        depth, pos, anc, _, _ = tv.tv_tree_prep(dev(par), dev(node), i32(position), None, N, 1)
        q, k, _ = tv.tv_rope(bf(x[:, :Hq]), bf(x[:, Hq:Hq + Hkv]), pos, dev(rope), err=err)
        v = bf(x[:, Hq + Hkv:])
        out, lse, _ = tv.tree_verify_attn_kv4(q, cache, P, dev(table), clen, k, v, dev(node), anc, N, err=err)
        logits = (2 * rng.standard_normal((2 * N, V))).astype(np.float32)
        tok = np.argsort(-logits, 1)[:, :3][np.clip(np.tile(par[:N], 2), 0, None) + np.repeat(node[:2], N),
                                            rng.integers(0, 3, 2 * N)].astype(np.int32)
        u, race = rng.random(2 * N).astype(np.float32), rng.exponential(size=(B, V)).astype(np.float32)
        acc, best, path, bonus = tv.accept_sampled(dev(par), dev(tok), dev(logits), dev(node), dev(u), dev(race),
                                                   temperature=dev(np.array([0.7, 1.1], np.float32)),
                                                   top_k=i32([20, 0]), top_p=dev(np.array([0.9, 1.0], np.float32)),
                                                   max_nodes=N, max_depth=N - 1)
        oacc, _, opath, obonus, margin = osm.verify(par, tok, logits, node, u, race, N - 1, None, None, [0.7, 1.1], [20, 0],
                                                    [0.9, 1.0])
        assert margin.min() > 1e-5                        # (of these inputs)
        assert np.array_equal(host(acc), oacc) and np.array_equal(host(path), opath) and np.array_equal(host(bonus), obonus)
        old = clen
        clen, _ = tv.kv4_append(k, v, cache, P, dev(table), old, dev(node), N, path=path, err=err)
        tv.kv4_attn_mass(q, lse, cache, P, dev(table), clen, dev(node), N, score=score, old_len=old, path=path, causal=True,
                         decay=0.9, score_out=score, err=err)
        opos = np.concatenate([position[r] + np.array([0, 1, 2, 2, 1, 2]) for r in range(B)])
        rot = lambda y: ok.f32(ok.bf16_bits(ok.rotate(y, opos, rope, False)))  # noqa: E731
        oq, okk, ov = rot(x[:, :Hq]), rot(x[:, Hq:Hq + Hkv]), x[:, Hq + Hkv:]
        oo, ol, av, sa = ok.attention(oq, ok.gather(ocache, P, table, [0, 0], olen), okk, ov, node, see)
        tol, ltol = ok.attention_tolerance(oo, ol, av, sa, d, True)
        assert (np.abs(out.float().cpu().numpy() - oo) <= tol).all()
        before = olen
        olen = ok.append(ocache, P, table, olen, okk, ov, node, path=opath)
        keys = [kk for kk, _ in ok.gather(ocache, P, table, [0, 0], olen)]
        # the weights follow the device's lse, itself within ltol of the oracle's
        assert (np.abs(host(lse) - ol) <= ltol).all()
        m, mtol = oe.attn_mass(oq, host(lse), keys, olen, node, N, oscore.astype(np.float32), 64, before, opath, None, True,
                               None, 0.9)
        for r in range(B):
            L = olen[r]
            slack[r, :, :L] = 0.9 * np.where(np.arange(L) < before[r], slack[r, :, :L], 0) + mtol[r, :, :L] + \
                2.0 ** -23 * np.abs(m[r, :, :L])
            oscore[r, :, :L] = m[r, :, :L]
            assert (np.abs(host(score)[r, :, :L] - m[r, :, :L]) <= slack[r, :, :L]).all()
        # the choice goes by the device's own scores
        mine = host(score)
        oidx, _, on = oe.evict_select(mine, olen, [budget] * B, 4, 8, budget)
        idx, _, new_len, _ = tv.kv4_evict_select(score, clen, i32([budget] * B), 64, 4, 8, max_keep=budget, score_out=score,
                                                 err=err)
        assert np.array_equal(host(idx), oidx) and np.array_equal(host(new_len), on)
        tv.kv4_compact(cache, P, dev(table), clen, idx, new_len, budget, err=err)
        full = ok.gather(ocache, P, table, [0, 0], olen)
        blocks = {(r, h, j): [z[j % P] for z in ok.read_block(ocache[table[r, j // P], h], P, d)]
                  for r in range(B) for h in range(Hkv) for j in range(olen[r])}
        for r in range(B):
            for h in range(Hkv):
                for j in range(on[r]):
                    kn, ks, vn, vs = blocks[r, h, int(oidx[r, h, j])]
                    ok.write_row(ocache[table[r, j // P], h], P, d, j % P, kn, ks, vn, vs)
                oscore[r, h, :on[r]] = oscore[r, h, oidx[r, h, :on[r]]]
                slack[r, h, :on[r]] = slack[r, h, oidx[r, h, :on[r]]]
        assert len(full) == B and np.array_equal(host(cache), ocache)
        position = position + oacc + 1
        clen, olen = new_len, on
    assert int(err) == 0 and position.max() > budget


@pytest.mark.parametrize("d", [64, 128])
def test_steps_of_a_cache_that_evicts(tv, d):
    serve(tv, d, 5)


def test_captured_on_another_stream(tv):
    """Weights, choice and move in one graph, replayed on new inputs, beside the same calls made eagerly."""
    m = Mass(21, [300, 260], [16, 12], 8, 2, 128, 64, path=True)
    pool, budget = dev(m.pool[0]), dev(np.array([200, 100], np.int32))
    q, lse, table, clen = m.q.clone(), dev(m.lse), dev(m.table), dev(np.array(m.lens, np.int32))
    off, old, path = dev(m.off), dev(m.old), dev(m.path)

    def step(cache, score, idx, new_len, err):
        tv.kv4_attn_mass(q, lse, cache, 64, table, clen, off, m.max_rows, score=score, old_len=old, path=path, causal=True,
                         score_out=score, err=err)
        tv.kv4_evict_select(score, clen, budget, 300, 4, 16, idx=idx, score_out=score, new_len=new_len, err=err)
        tv.kv4_compact(cache, 64, table, clen, idx, new_len, 200, err=err)

    def buffers():
        return [pool.clone(), dev(m.score), torch.empty((2, 2, 200), dtype=torch.int32, device="cuda"),
                torch.empty(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")]
    a, b = buffers(), buffers()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(*buffers())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(*a)
        for scale in (1.0, 0.5):
            q.mul_(scale)
            for x, y in zip(a, buffers()):
                x.copy_(y)
            b = buffers()
            g.replay()
            step(*b)
    stream.synchronize()
    assert int(a[4]) == 0
    for x, y in zip(a, b):
        assert torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float()))
