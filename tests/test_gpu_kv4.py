"""GPU parity of the paged 4-bit KV cache calls (tv_rope, kv4_append,
kv4_gather, tree_verify_attn_kv4) against oracle/kv4.py.

Rotation, append and gather are compared bit for bit: the definition fixes
every rounding.  Attention is compared with the fp64 oracle within
``kv4.attention_tolerance`` (bounds derived there from the roundings)."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from oracle import kv4 as ok
from oracle import tree as otree

pytestmark = pytest.mark.gpu
NAN = float("nan")


# ------------------------------------------------------------------- helpers
def act(x, bf16):
    """float32 array -> (device tensor, the float32 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    t = t.to(torch.bfloat16) if bf16 else t
    return t, t.float().cpu().numpy()


def bits(t):
    t = t.contiguous()
    return host(t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32))


def rounded(x, bf16):
    """float32 values -> the bits of the rows' type."""
    return ok.bf16_bits(x).view(np.int16) if bf16 else np.ascontiguousarray(x, np.float32).view(np.int32)


def fused(rng, n, Hq, Hkv, d, bf16):
    """q, k, v as slices of one projection's rows: [n, Hq + 2 Hkv, d]."""
    t, x = act(rng.standard_normal((n, Hq + 2 * Hkv, d)), bf16)
    cut = (slice(0, Hq), slice(Hq, Hq + Hkv), slice(Hq + Hkv, None))
    return [t[:, c] for c in cut], [x[:, c] for c in cut]


def random_pool(rng, n_pages, H, P, d):
    """(cache uint8, kn, ks, vn, vs) of a pool with a quantised row in every slot."""
    kn, vn = rng.integers(-7, 8, (2, n_pages, H, P, d))
    ks, vs = ok.f32(ok.bf16_bits(rng.uniform(0.2, 0.4, (2, n_pages, H, P)).astype(np.float32)))
    cache = np.zeros((n_pages, H, P * (d + 4)), np.uint8)
    slot, dim = np.meshgrid(np.arange(P), np.arange(d), indexing="ij")
    for at, n in ((ok._k_at(P, slot, dim), kn), (ok._v_at(P, d, slot, dim), vn)):
        byte, sh = (np.asarray(x).ravel() for x in at)
        code = ((n + 8).reshape(n_pages, H, -1) << sh).astype(np.uint8)
        for nib in (0, 4):
            m = sh == nib
            cache[:, :, byte[m]] |= code[:, :, m]
    for off, s in ((P * d, ks), (P * d + 2 * P, vs)):
        b = ok.bf16_bits(s)
        cache[:, :, off:off + 2 * P:2] = b & 255
        cache[:, :, off + 1:off + 2 * P:2] = b >> 8
    return cache, kn, ks, vn, vs


def tables(rng, lens, P, spare=1, extra_cols=1):
    """Block table over randomly ordered pages (unused entries -1) and the page count."""
    used = [(n + P - 1) // P for n in lens]
    n_pages = sum(used) + spare
    perm = rng.permutation(n_pages)
    t = np.full((len(lens), max(used) + extra_cols), -1, np.int32)
    o = 0
    for r, u in enumerate(used):
        t[r, :u] = perm[o:o + u]
        o += u
    return t, n_pages


def prefixes(pool, table, lens, P):
    """Per request the (K, V) values of its cached tokens."""
    _, kn, ks, vn, vs = pool
    out = []
    for r, n in enumerate(lens):
        t = np.arange(n)
        pg, sl = np.clip(table[r, t // P], 0, len(kn) - 1), t % P   # (a bad page: masked by its caller)
        out.append((ok.values(kn[pg, :, sl], ks[pg, :, sl]), ok.values(vn[pg, :, sl], vs[pg, :, sl])))
    return out


def forest(rng, counts, kind):
    """(parent, node_off, anc, see) of one tree per request."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    words = max(1, (max(counts) + 63) // 64)
    par, anc, see = [], np.zeros((off[-1], words), np.uint64), np.zeros((off[-1], max(max(counts), 1)), bool)
    for r, n in enumerate(counts):
        for i in range(n):
            if kind == "chain":
                p = i - 1
            elif kind == "roots":
                p = -1 if i % 5 == 0 else i - 1
            else:
                p = -1 if i == 0 else int(rng.integers(0, i))
            par.append(p)
            g = off[r] + i
            if p >= 0:
                see[g] = see[off[r] + p]
                anc[g] = anc[off[r] + p]
            see[g, i] = True
            anc[g, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return np.array(par, np.int32), off, anc, see


class Case:
    """One tree_verify_attn_kv4 call and what the oracle says about it."""

    def __init__(self, seed, counts, lens, Hq, Hkv, d, P, bf16=True, kind="random", vis=False, node_cnt=None,
                 scale=None):
        rng = np.random.default_rng(seed)
        self.d, self.P, self.bf16, self.lens, self.scale, self.node_cnt = d, P, bf16, list(lens), scale, node_cnt
        self.table, n_pages = tables(rng, lens, P)
        self.pool = random_pool(rng, n_pages, Hkv, P, d)
        self.cache = self.pool[0].copy()
        _, self.off, self.anc, self.see = forest(rng, counts, kind)
        n = int(self.off[-1])
        (self.q, self.k, self.v), (self.hq, self.hk, self.hv) = fused(rng, n, Hq, Hkv, d, bf16)
        self.max_nodes = max(counts)
        self.vis = None
        if vis:
            self.vis = np.concatenate([rng.integers(-2, m + 3, c) for m, c in zip(lens, counts)]).astype(np.int32)
        self.page_ok = None

    def prefix(self):
        return prefixes(self.pool, self.table, self.lens, self.P)

    def args(self):
        return (self.q, dev(self.cache), self.P, dev(self.table), dev(np.array(self.lens, np.int32)), self.k, self.v,
                dev(self.off), dev(self.anc.view(np.int64)), self.max_nodes)

    def kwargs(self):
        nc = None if self.node_cnt is None else dev(np.array(self.node_cnt, np.int32))
        return dict(vis_prefix=dev(self.vis), node_cnt=nc, scale=self.scale)

    def oracle(self):
        return ok.attention(self.hq, self.prefix(), self.hk, self.hv, self.off, self.see, self.vis, self.node_cnt,
                            self.scale, self.page_ok)

    def check(self, out, lse, want=None):
        o, l, av, sa = want or self.oracle()
        tol, ltol = ok.attention_tolerance(o, l, av, sa, self.d, self.bf16)
        got, gl = out.float().cpu().numpy().astype(np.float64), host(lse).astype(np.float64)
        rows = ~np.isnan(l)
        err = np.abs(got - o)[rows]
        assert (err <= tol[rows]).all(), f"out: {np.nanmax(err / tol[rows]):.3f} of the tolerance"
        fin = rows & np.isfinite(l)
        assert np.array_equal(gl[rows & ~fin], l[rows & ~fin])
        ratio = np.abs(gl[fin] - l[fin]) / ltol[fin]
        assert (ratio <= 1).all(), f"lse: {ratio.max():.3f} of the tolerance"

    def run(self, tv, **kw):
        out, lse, err = tv.tree_verify_attn_kv4(*self.args(), **(self.kwargs() | kw))
        return out, lse, err


# ------------------------------------------------------------------ rotation
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n,Hq,Hkv,d,rot,inter", [
    (1, 32, 8, 128, 128, False), (37, 4, 1, 64, 64, True), (130, 7, 7, 128, 64, False), (5, 1, 3, 64, 16, True),
    (9, 3, 0, 256, 96, False), (2, 2, 2, 16, 0, False)])
def test_rope_matches_bit_for_bit(tv, n, Hq, Hkv, d, rot, inter, bf16):
    rng = np.random.default_rng(n + rot)
    table = ok.rope_table(200, rot) if rot else None
    pos = rng.integers(0, 200, n).astype(np.int32)
    (q, k, _), (hq, hk, _) = fused(rng, n, Hq, max(Hkv, 1), d, bf16)
    k = k if Hkv else None
    qo, ko, err = tv.tv_rope(q, k, dev(pos), dev(table), interleaved=inter)
    assert int(err) == 0
    assert np.array_equal(bits(qo), rounded(ok.rotate(hq, pos, table, inter), bf16))
    if Hkv:
        assert np.array_equal(bits(ko), rounded(ok.rotate(hk, pos, table, inter), bf16))


def test_rope_skips_rows_with_a_bad_position(tv):
    rng = np.random.default_rng(0)
    (q, k, _), (hq, _, _) = fused(rng, 6, 4, 2, 64, True)
    pos = np.array([0, -1, 7, 8, 2 ** 31 - 1, 3], np.int32)
    table = ok.rope_table(8, 64)
    out = tuple(torch.full((6, h, 64), 3.0, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    qo, ko, err = tv.tv_rope(q, k, dev(pos), dev(table), outputs=out)
    assert int(err) == 1
    good = [0, 2, 5]
    assert np.array_equal(bits(qo)[good], rounded(ok.rotate(hq[good], pos[good], table, False), True))
    bad = [1, 3, 4]
    assert (qo[bad] == 3).all() and (ko[bad] == 3).all()


# ------------------------------------------------------------ append, gather
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("P,H,d,lens,counts,rot,inter", [
    (16, 2, 64, [0, 5, 31], [1, 40, 3], 64, False),
    (64, 1, 128, [63, 64, 10], [1, 130, 0], 128, True),
    (32, 3, 128, [17], [200], 64, False),
    (128, 1, 64, [127, 3], [2, 1], 0, False)])
def test_append_and_gather_match_bit_for_bit(tv, P, H, d, lens, counts, rot, inter, bf16):
    rng = np.random.default_rng(P + d)
    table, n_pages = tables(rng, [a + b for a, b in zip(lens, counts)], P)
    cache = rng.integers(0, 256, (n_pages, H, P * (d + 4))).astype(np.uint8)   # stale codes everywhere
    n = sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    (_, k, v), (_, hk, hv) = fused(rng, n, 1, H, d, bf16)
    rope = ok.rope_table(512, rot) if rot else None
    want = cache.copy()
    want_len = ok.append(want, P, table, lens, hk, hv, off, rope=rope, interleaved=inter)
    c = dev(cache)
    new_len, err = tv.kv4_append(k, v, c, P, dev(table), dev(np.array(lens, np.int32)), dev(off), max(counts),
                                 rope=dev(rope), interleaved=inter)
    assert int(err) == 0 and np.array_equal(host(new_len), want_len)
    assert np.array_equal(host(c), want)
    start = dev(np.array(lens, np.int32))
    dt = torch.bfloat16 if bf16 else torch.float32
    K, V, err = tv.kv4_gather(c, P, dev(table), dev(off), max(counts), start=start, total_rows=n, dtype=dt)
    assert int(err) == 0
    parts = ok.gather(want, P, table, lens, counts)
    assert np.array_equal(bits(K), rounded(np.concatenate([p[0] for p in parts]), bf16))
    assert np.array_equal(bits(V), rounded(np.concatenate([p[1] for p in parts]), bf16))


def test_append_by_path_with_given_positions(tv):
    rng = np.random.default_rng(3)
    P, H, d, B, N = 16, 2, 128, 3, 7
    lens = [15, 0, 30]
    path = np.array([[0, 2, 3, 6, -1, 5], [-1, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 6]], np.int32)
    table, n_pages = tables(rng, [40, 10, 40], P)
    off = (np.arange(B + 1) * N).astype(np.int32)
    pos = rng.integers(0, 100, B * N).astype(np.int32)
    (_, k, v), (_, hk, hv) = fused(rng, B * N, 4, H, d, True)
    rope = ok.rope_table(100, d)
    for max_new in (6, 4):
        cache = np.zeros((n_pages, H, P * (d + 4)), np.uint8)
        want_len = ok.append(cache, P, table, lens, hk, hv, off, path[:, :max_new], pos, rope)
        c = torch.zeros(cache.shape, dtype=torch.uint8, device="cuda")
        new_len, err = tv.kv4_append(k, v, c, P, dev(table), dev(np.array(lens, np.int32)), dev(off), max_new,
                                     path=dev(path), pos=dev(pos), rope=dev(rope))
        assert int(err) == 0 and np.array_equal(host(new_len), want_len)
        assert np.array_equal(host(c), cache)


def test_append_rows_with_nan_infinity_zero_and_extreme_values(tv):
    rng = np.random.default_rng(4)
    P, H, d = 16, 1, 64
    x = rng.standard_normal((8, H, d)).astype(np.float32)
    x[0, 0, 5] = np.nan
    x[1, 0, 60] = np.inf
    x[2, 0, 0] = -np.inf
    x[3] = 0
    x[4] *= np.float32(1e-35)
    x[5] *= np.float32(5e37)
    x[6, 0] = np.linspace(-7, 7, d).round() / 2          # exact ties
    table = np.array([[0]], np.int32)
    cache = np.zeros((1, H, P * (d + 4)), np.uint8)
    ok.append(cache, P, table, [2], x, x, [0, 8])
    c = torch.zeros(cache.shape, dtype=torch.uint8, device="cuda")
    _, err = tv.kv4_append(dev(x), dev(x), c, P, dev(table), dev(np.array([2], np.int32)),
                           dev(np.array([0, 8], np.int32)), 8)
    assert int(err) == 0
    got, want = ok.read_block(host(c)[0, 0], P, d), ok.read_block(cache[0, 0], P, d)
    for g, w in zip(got, want):
        finite = ~np.isnan(w) if w.ndim == 1 else ~np.isnan(want[1])[:, None] & np.ones_like(w, bool)
        assert np.array_equal(np.isnan(g), np.isnan(w)) and np.array_equal(g[finite], w[finite])


def test_append_and_gather_skip_what_is_out_of_range(tv):
    rng = np.random.default_rng(5)
    P, H, d, B = 16, 1, 64, 4
    lens = np.array([10, 30, -3, 5], np.int32)
    counts = [20, 8, 4, 4]
    table = np.array([[0, -1], [1, 2], [3, 4], [99, 5]], np.int32)    # a missing page, a short table, a page id too large
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    (_, k, v), (_, hk, hv) = fused(rng, 36, 1, H, d, True)
    before = rng.integers(0, 256, (6, H, P * (d + 4))).astype(np.uint8)
    want = before.copy()
    ok.append(want, P, table[[0, 1, 3]], lens[[0, 1, 3]], hk[[*range(28), *range(32, 36)]],
              hv[[*range(28), *range(32, 36)]], [0, 20, 28, 32])
    c = dev(before)
    new_len, err = tv.kv4_append(k, v, c, P, dev(table), dev(lens), dev(off), 20)
    assert int(err) == 1 and host(new_len).tolist()[:2] == [30, 38]
    assert np.array_equal(host(c), want)
    # a path that points outside the rows
    path = np.array([[0, 1000, 2], [0, 1, -1], [0, 0, 0], [-1, 0, 0]], np.int32)
    c = dev(before)
    lens2 = np.array([0, 0, 0, 0], np.int32)
    _, err = tv.kv4_append(k, v, c, P, dev(np.array([[0], [1], [2], [3]], np.int32)), dev(lens2), dev(off), 3,
                           path=dev(path))
    assert int(err) == 1
    got = host(c)
    want = before.copy()
    ok.append(want, P, np.array([[1], [2]]), [0, 0], hk, hv, [20, 28, 36], path[1:3])
    assert np.array_equal(got[1:], want[1:])
    # gather: a bad page and a start past the table leave their rows as they were
    for start, tbl in (([0, 16], [[0, -1], [1, 2]]), ([0, 28], [[0, 3], [1, 2]])):
        K, V = (torch.full((32, H, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        _, _, err = tv.kv4_gather(dev(want), P, dev(np.array(tbl, np.int32)), dev(np.array([0, 24, 32], np.int32)), 24,
                                  start=dev(np.array(start, np.int32)), outputs=(K, V))
        assert int(err) == 1
        w = ok.gather(want, P, np.array(tbl), [0], [16 if tbl[0][1] < 0 else 24])[0][0]
        assert np.array_equal(bits(K)[:len(w)], rounded(w, True))
        assert (K[len(w):24] == 9).all() and (tbl[0][1] < 0 or (K[28:] == 9).all())
    K, V = (torch.full((32, H, d), 9.0, device="cuda") for _ in range(2))
    _, _, err = tv.kv4_gather(dev(want), P, dev(table), dev(np.array([0, 8, 8, 8, 40], np.int32)), 40,
                              outputs=(K, V))                        # out_off past the outputs
    assert int(err) == 1 and (K[8:] == 9).all() and (K[:8] != 9).any()


# ----------------------------------------------------------------- attention
ATTN = [
    # counts, lens, Hq, Hkv, d, P, kind, vis
    ([1], [1], 1, 1, 128, 16, "chain", False),
    ([1], [0], 4, 1, 64, 16, "chain", False),
    ([1, 1, 1], [129, 5, 777], 32, 8, 128, 64, "chain", False),
    ([16, 16], [200, 385], 8, 2, 128, 64, "chain", False),
    ([60], [128], 4, 1, 64, 16, "random", False),
    ([61, 3], [300, 0], 8, 2, 128, 128, "random", False),
    ([113, 20, 1], [130, 128, 127], 4, 1, 128, 16, "random", True),
    ([33], [512], 7, 1, 128, 32, "random", True),
    ([9, 2], [1000, 255], 28, 4, 64, 64, "roots", True),
    ([150], [140], 2, 2, 128, 32, "chain", True),
    ([5], [260], 64, 1, 128, 16, "roots", False),
    ([4, 4], [96, 17], 48, 1, 64, 32, "chain", False),
    # few rows per KV head: 3 to 16, one and two blocks of eight
    ([3, 1, 2], [64, 200, 65], 8, 2, 128, 16, "chain", True),
    ([2], [1000], 16, 4, 64, 128, "roots", False),
    ([4, 3, 1], [300, 1, 63], 32, 8, 128, 32, "random", False),
    ([16, 9], [130, 128], 1, 1, 128, 128, "random", True),
    ([1, 1], [65, 129], 16, 1, 128, 64, "chain", True),
    ([2, 2], [40, 700], 7, 1, 64, 16, "chain", False),
    # 17 rows and one more tile of 64
    ([17], [127], 1, 1, 64, 64, "roots", False),
    ([65], [100], 2, 2, 128, 64, "random", False),
]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts,lens,Hq,Hkv,d,P,kind,vis", ATTN)
def test_attention_matches_the_oracle(tv, counts, lens, Hq, Hkv, d, P, kind, vis, bf16):
    c = Case(len(counts) * 1000 + lens[0], counts, lens, Hq, Hkv, d, P, bf16, kind, vis)
    out, lse, err = c.run(tv)
    assert int(err) == 0
    c.check(out, lse)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts", [[20, 3], [2, 1], [4, 4]])
def test_attention_large_logits_and_scale(tv, counts, bf16):
    c = Case(7, counts, [300, 140], 8, 2, 128, 64, bf16, scale=2.5)   # peaked softmax, growing maxima
    out, lse, _ = c.run(tv)
    c.check(out, lse)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts,kind", [([40, 3], "random"), ([150, 33], "chain"), ([4, 2], "chain"), ([2, 1], "roots")])
def test_attention_tree_scores_far_above_the_cached_ones(tv, counts, kind, bf16):
    """Nodes' keys 16 times as long: the running maxima grow in the tree's own tiles, under its masks."""
    c = Case(20, counts, [300, 64], 8, 2, 128, 32, bf16, kind)
    c.k, c.hk = c.k * 16, c.hk * 16            # exact
    out, lse, _ = c.run(tv)
    c.check(out, lse)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts,cnt", [([16, 16, 9], [5, 0, 9]), ([4, 2, 3], [1, 0, 3]),
                                        ([110, 60, 9], [5, 0, 9])])
def test_attention_node_cnt_leaves_other_rows(tv, counts, cnt, bf16):
    c = Case(8, counts, [100, 300, 64], 8, 2, 128, 32, bf16, "chain", node_cnt=cnt)
    n = int(c.off[-1])
    out = torch.full((n, 8, 128), 5.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((n, 8), 5.0, device="cuda")
    c.run(tv, out=out, lse=lse)
    c.check(out, lse)
    left = [c.off[r] + i for r in range(3) for i in range(cnt[r], counts[r])]
    assert (out[left] == 5).all() and (lse[left] == 5).all()
    without, none, _ = c.run(tv, want_lse=False)
    assert none is None and torch.equal(without[:cnt[0]], out[:cnt[0]])


@pytest.mark.parametrize("bf16", [True, False])
def test_attention_rows_that_see_nothing(tv, bf16):
    c = Case(9, [12, 6], [50, 0], 8, 2, 128, 16, bf16, "chain")
    c.vis = np.zeros(18, np.int32)
    c.vis[3] = 20
    for i in (1, 3, 14):                       # no ancestor bits at all, not even the node itself
        c.anc[i] = 0
        c.see[i] = False
    out, lse, _ = c.run(tv)
    c.check(out, lse)
    assert (out[[1, 14]] == 0).all() and torch.isneginf(lse[[1, 14]]).all()


@pytest.mark.parametrize("bf16", [True, False])
def test_attention_few_rows_that_see_nothing_or_late(tv, bf16):
    """Rows whose first visible key comes after many masked ones, and rows without any, among few rows."""
    c = Case(19, [4, 2], [200, 70], 8, 2, 128, 64, bf16, "chain", vis=True)
    c.vis[:] = [0, 200, 0, 1, 0, 70]
    for i in (0, 4):
        c.anc[i] = 0
        c.see[i] = False
    out, lse, _ = c.run(tv)
    c.check(out, lse)
    assert (out[[0, 4]] == 0).all() and torch.isneginf(lse[[0, 4]]).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts", [[24, 24, 10], [4, 4, 3], [110, 24, 10]])
def test_attention_ignores_whatever_it_does_not_see(tv, counts, bf16):
    """NaN and infinities in tree rows that a node does not see, in rows of other requests, in rows beyond node_cnt,
    and NaN scales behind the end of the cached tokens."""
    half = counts[1] // 2
    c = Case(10, counts, [70, 129, 33], 8, 2, 128, 64, bf16, "random", node_cnt=[counts[0], half, counts[2]])
    clean = c.run(tv)
    want = c.oracle()
    d, P = c.d, c.P
    for r, n in enumerate(c.lens):             # stale tokens: NaN scales, any codes
        pg = c.table[r, n // P] if n % P else -1
        if pg >= 0:
            c.cache[pg, :, P * d + 2 * (n % P):P * d + 2 * P] = 0xFF
            c.cache[pg, :, P * d + 2 * P + 2 * (n % P):] = 0xFF
    gone = list(range(int(c.off[1]) + half, int(c.off[2])))    # nodes that node_cnt leaves out
    for i, bad in zip(gone, (NAN, float("inf"), -float("inf"))):
        c.k[i], c.v[i], c.q[i] = bad, bad, bad
    leaf = counts[0] - 1                       # the last node is nobody's ancestor
    c.k[leaf], c.v[leaf] = NAN, NAN
    out, lse, err = c.run(tv)
    assert int(err) == 0
    rows = [i for i in range(sum(counts)) if i != leaf and i not in gone]
    assert torch.equal(out[rows], clean[0][rows]) and torch.equal(lse[rows], clean[1][rows])
    assert torch.isnan(out[leaf]).all() and torch.isnan(lse[leaf]).all()
    c.check(clean[0], clean[1], want)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts", [[10, 6], [4, 3], [80, 60]])
def test_attention_nan_and_infinity_reach_exactly_the_rows_that_see_them(tv, counts, bf16):
    n0, n = counts[0], sum(counts)
    c = Case(11, counts, [40, 40], 8, 2, 128, 16, bf16, "chain")
    clean = c.run(tv)
    a, b = n0 // 2 - 1, n0 - 2
    c.v[a, 1, 7] = float("inf")                # a node of request 0, KV head 1, dim 7
    c.v[b, 0, 3] = NAN
    out, lse, _ = c.run(tv)
    exp = clean[0].clone()
    exp[a:n0, 4:, 7] = float("inf")
    exp[b:n0, :4, 3] = NAN
    assert torch.equal(torch.isnan(out), torch.isnan(exp)) and torch.equal(torch.isinf(out), torch.isinf(exp))
    ok_ = torch.isfinite(exp)
    assert torch.equal(out[ok_], exp[ok_]) and torch.equal(lse, clean[1])
    # a cached token whose key was not finite: every row that sees it is NaN, the others are as they were
    c = Case(11, counts, [40, 40], 8, 2, 128, 16, bf16, "chain", vis=True)
    c.vis[:] = 40
    c.vis[n0] = 35                             # tokens 0 .. 34: token 35 is not among them
    clean = c.run(tv)
    pg = c.table[1, 2]
    c.cache[pg, 0, c.P * 128 + 2 * 3:c.P * 128 + 2 * 3 + 2] = [0xC0, 0x7F]
    out, lse, _ = c.run(tv)
    assert torch.isnan(out[n0 + 1:, :4]).all() and torch.isnan(lse[n0 + 1:, :4]).all()
    assert torch.equal(out[:n0 + 1], clean[0][:n0 + 1]) and torch.equal(out[n0 + 1:, 4:], clean[0][n0 + 1:, 4:])
    # ... whose value was not: outputs are NaN, the sums are not
    c.cache[pg, 0, c.P * 128 + 2 * 3:c.P * 128 + 2 * 3 + 2] = c.pool[0][pg, 0, c.P * 128 + 6:c.P * 128 + 8]
    c.cache[pg, 0, c.P * 130 + 2 * 3:c.P * 130 + 2 * 3 + 2] = [0xC0, 0x7F]
    out, lse, _ = c.run(tv)
    assert torch.isnan(out[n0 + 1:, :4]).all() and torch.equal(lse, clean[1])
    assert torch.equal(out[:n0 + 1], clean[0][:n0 + 1])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts", [[5, 5], [2, 1], [4, 4], [80, 70]])
def test_attention_bad_pages_are_not_visible(tv, counts, bf16):
    c = Case(12, counts, [200, 90], 8, 2, 128, 32, bf16)
    c.table[0, 2] = -1
    c.table[1, 1] = 10 ** 6
    c.page_ok = [np.arange(200) // 32 != 2, np.arange(90) // 32 != 1]
    out, lse, err = c.run(tv)
    assert int(err) == 1
    c.check(out, lse)


def test_attention_clamps_lengths(tv):
    c = Case(13, [4, 4], [96, 64], 8, 2, 128, 32)
    args = list(c.args())
    c.table = c.table[:, :3].copy()
    args[3] = dev(c.table)
    args[4] = dev(np.array([1000, -7], np.int32))     # 3 pages of 32 hold 96 tokens
    out, lse, err = tv.tree_verify_attn_kv4(*args)
    assert int(err) == 1
    c.lens = [96, 0]
    c.check(out, lse)


@pytest.mark.parametrize("counts", [[16, 16, 1], [1, 1, 1], [3, 2, 4]])
def test_attention_is_the_same_twice_on_another_stream_and_in_a_graph(tv, counts):
    c = Case(14, counts, [900, 1300, 40], 32, 8, 128, 64, True, "chain")
    args, kw = c.args(), c.kwargs()
    ws = [tv.tree_verify_attn_kv4_workspace(3, max(counts), 32, 8, 128) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = tv.tree_verify_attn_kv4(*args, **kw, ws=ws[0], err=err)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        two = tv.tree_verify_attn_kv4(*args, **kw, ws=ws[1], err=err)
    three = tv.tree_verify_attn_kv4(*args, **kw, ws=ws[0], err=err)    # at the same time, in its own workspace
    torch.cuda.synchronize()
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1]) and torch.equal(one[0], three[0])
    out, lse = torch.empty_like(one[0]), torch.empty_like(one[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tv.tree_verify_attn_kv4(*args, **kw, out=out, lse=lse, ws=ws[0], err=err)
    for lens in ([900, 1300, 40], [1, 129, 0], [640, 5, 33]):          # lengths change between replays
        args[4].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.lens = lens
        c.check(out, lse)
    assert int(err) == 0 and int(ws[0][:4].view(torch.int32)) == 0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("counts,lens", [([1], [40000]), ([20], [40000]), ([1, 2, 1], [1, 30000, 17])])
def test_attention_one_long_prefix_among_short_ones(tv, counts, lens, bf16):
    """Units cut into hundreds of pieces beside units of a tile."""
    c = Case(24, counts, lens, 4, 1, 128, 128, bf16)
    out, lse, _ = c.run(tv)
    c.check(out, lse)


def test_two_graphs_at_once_with_a_workspace_each(tv):
    """Replays on two streams: other requests, other rows, one cache."""
    cs = [Case(21, n, [700, 129], 8, 2, 128, 64, True, "chain") for n in ([30, 9], [4, 1])]
    runs = []
    for c in cs:
        args, kw = c.args(), c.kwargs()
        want = tv.tree_verify_attn_kv4(*args, **kw)
        out, lse, err = (torch.zeros_like(t) for t in want)
        ws = tv.tree_verify_attn_kv4_workspace(2, c.max_nodes, 8, 2, 128)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tv.tree_verify_attn_kv4(*args, **kw, out=out, lse=lse, err=err, ws=ws)
        runs.append((g, torch.cuda.Stream(), args, kw, want, out, lse, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, *_ in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (_, _, _, _, want, out, lse, _) in zip(cs, runs):
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        c.check(out, lse)


def test_one_workspace_for_the_largest_trees_serves_all_calls(tv):
    ws = tv.tree_verify_attn_kv4_workspace(8, 113, 32, 8, 128)
    for seed, counts in enumerate(([113, 4], [1, 1, 1], [4, 2], [3], [60])):
        c = Case(50 + seed, counts, [200] * len(counts), 32, 8, 128, 64, True, "chain")
        out, lse, err = c.run(tv, ws=ws)
        assert int(err) == 0
        c.check(out, lse)


def test_append_takes_no_more_rows_than_max_new(tv):
    rng = np.random.default_rng(22)
    P, H, d = 16, 2, 64
    table, n_pages = tables(rng, [40, 40], P)
    off = np.array([0, 9, 12], np.int32)
    (_, k, v), (_, hk, hv) = fused(rng, 12, 2, H, d, True)
    cache = np.zeros((n_pages, H, P * (d + 4)), np.uint8)
    c = torch.zeros(cache.shape, dtype=torch.uint8, device="cuda")
    take = [0, 1, 2, 3, 4, 9, 10, 11]
    want = ok.append(cache, P, table, [14, 0], hk[take], hv[take], np.array([0, 5, 8]))
    new_len, err = tv.kv4_append(k, v, c, P, dev(table), dev(np.array([14, 0], np.int32)), dev(off), 5)
    assert int(err) == 1                       # told, and the first five are there
    assert np.array_equal(host(new_len), want) and np.array_equal(host(c), cache)


def test_append_tells_of_rows_beyond_a_max_new_of_zero(tv):
    P, H, d = 16, 1, 64
    (_, k, v), _ = fused(np.random.default_rng(25), 4, 1, H, d, True)
    for off, want in (([0, 0, 4], 1), ([0, 0, 0], 0)):
        c = torch.zeros((2, H, P * (d + 4)), dtype=torch.uint8, device="cuda")
        lens = dev(np.array([3, 5], np.int32))
        new_len, err = tv.kv4_append(k, v, c, P, dev(np.array([[0], [1]], np.int32)), lens, dev(np.array(off, np.int32)), 0)
        assert int(err) == want and torch.equal(new_len, lens) and (c == 0).all()


def test_append_counts_skipped_rows_and_leaves_negative_lengths(tv):
    rng = np.random.default_rng(23)
    P, H, d = 16, 1, 64
    table = np.array([[0], [7], [1]], np.int32)          # the second request's page is bad
    (_, k, v), _ = fused(rng, 9, 1, H, d, True)
    c = torch.zeros((2, H, P * (d + 4)), dtype=torch.uint8, device="cuda")
    new_len, err = tv.kv4_append(k, v, c, P, dev(table), dev(np.array([15, 2, -2], np.int32)),
                                 dev(np.array([0, 3, 6, 9], np.int32)), 3)
    assert int(err) == 1 and host(new_len).tolist() == [18, 5, -2]
    assert (host(c)[1] == 0).all() and (host(c)[0] != 0).any()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("by_path", [True, False])
@pytest.mark.parametrize("idle_len", [20, 16, 0, 48])
def test_append_leaves_an_idle_request_alone(tv, idle_len, by_path, bf16):
    """A request that appends nothing needs no table entry: its pages may have been given back (-1, or a page that is
    another request's by now), its length kept."""
    rng = np.random.default_rng(idle_len)
    P, H, d, N = 16, 2, 64, 3
    table = np.array([[-1, -1, -1], [3, 1, 0], [99, 99, 1]], np.int32)
    lens = np.array([idle_len, 15, idle_len], np.int32)
    path = np.array([[-1, 0, 1], [0, 2, -1], [-1, -1, -1]], np.int32) if by_path else None
    off = np.array([0, N, 2 * N, 3 * N] if by_path else [0, 0, N, N], np.int32)
    (_, k, v), (_, hk, hv) = fused(rng, int(off[-1]), 1, H, d, bf16)
    before = rng.integers(0, 256, (4, H, P * (d + 4))).astype(np.uint8)
    want = before.copy()
    want_len = ok.append(want, P, table, lens, hk, hv, off, path)
    c = dev(before)
    new_len, err = tv.kv4_append(k, v, c, P, dev(table), dev(lens), dev(off), N, path=dev(path))
    assert int(err) == 0 and np.array_equal(host(new_len), want_len) and np.array_equal(host(c), want)
    # nobody appends: by the bound, by the rows
    for kk, vv, o, m in ((k, v, off, 0), (k[:0], v[:0], np.zeros(4, np.int32), N)):
        c = dev(before)
        new_len, err = tv.kv4_append(kk, vv, c, P, dev(np.full_like(table, -1)), dev(lens), dev(o * 0), m)
        assert int(err) == 0 and np.array_equal(host(new_len), lens) and np.array_equal(host(c), before)


def test_cache_offsets_pass_32_bits(tv):
    """Pages behind the first 4 GB of the pool."""
    P, H, d = 128, 8, 128
    n_pages = 32500                            # 135168 bytes each: 4.39 GB
    cache = torch.empty((n_pages, H, P * (d + 4)), dtype=torch.uint8, device="cuda")
    c = Case(15, [3], [130], 32, H, d, P)
    far = np.array([[n_pages - 1, n_pages - 3, -1]], np.int32)
    for i in range(2):
        cache[int(far[0, i])] = dev(c.cache[c.table[0, i]])
    args = list(c.args())
    args[1], args[3] = cache, dev(far)
    out, lse, err = tv.tree_verify_attn_kv4(*args)
    assert int(err) == 0
    c.check(out, lse)
    K, V, err = tv.kv4_gather(cache, P, dev(far), dev(np.array([0, 130], np.int32)), 130, total_rows=130)
    want = c.prefix()[0]
    assert np.array_equal(bits(K), rounded(want[0], True)) and np.array_equal(bits(V), rounded(want[1], True))
    rng = np.random.default_rng(0)
    (_, k, v), (_, hk, hv) = fused(rng, 6, 1, H, d, True)
    tv.kv4_append(k, v, cache, P, dev(far), dev(np.array([126], np.int32)), dev(np.array([0, 6], np.int32)), 6)
    K, V, err = tv.kv4_gather(cache, P, dev(far), dev(np.array([0, 6], np.int32)), 6,
                              start=dev(np.array([126], np.int32)), total_rows=6)
    assert np.array_equal(bits(K), rounded(ok.values(*ok.quantise(hk)), True))
    assert np.array_equal(bits(V), rounded(ok.values(*ok.quantise(hv)), True))


def test_gathered_prefix_feeds_the_contiguous_attention(tv):
    """The same step over the 4-bit cache and over its gathered bf16 rows: the values are the same but for the rows'
    rounding to bf16 (at most 2^-8 of each key and value)."""
    c = Case(16, [16, 16], [300, 520], 32, 8, 128, 64, True, "chain")
    out, lse, _ = c.run(tv)
    off = np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32)
    K, V, _ = tv.kv4_gather(dev(c.cache), c.P, dev(c.table), dev(off), max(c.lens), total_rows=int(off[-1]))
    args = c.args()
    o2, l2 = tv.tree_verify_attn(c.q.contiguous(), K, V, dev(off), c.k.contiguous(), c.v.contiguous(), dev(c.off),
                                 args[8], 16, max(c.lens))
    _, _, av, sa = c.oracle()
    # keys off by 2^-8 move a score by 2^-8 sum|q k| and a weight by twice that relatively; values by 2^-8;
    # both calls round weights and outputs to bf16
    bound = av * (2 * 2.0 ** -8 * sa[..., None] + 5 * 2.0 ** -8)
    assert (np.abs((out - o2).float().cpu().numpy()) <= bound + 1e-6).all()
    assert (np.abs(host(lse) - host(l2)) <= 2.0 ** -8 * sa + 1e-4).all()


# -------------------------------------------------- rows whose maximum is zero
def scale_keys(c, r, tokens, factor):
    """Multiplies the cached keys of these tokens by a power of two; 0: zero rows as kv4_append leaves them."""
    _, kn, ks, _, _ = c.pool
    pg, sl = c.table[r, tokens // c.P], tokens % c.P
    heads = np.arange(ks.shape[1])
    if factor:
        ks[pg, :, sl] *= np.float32(factor)
    else:
        kn[pg, :, sl], ks[pg, :, sl] = 0, ok.SCALE_MIN
        byte = ok._k_at(c.P, sl[:, None], np.arange(c.d))[0]
        c.cache[pg[:, None, None], heads[:, None], byte[:, None]] = 0x88
    b = ok.bf16_bits(ks[pg, :, sl])
    at = (c.P * c.d + 2 * sl)[:, None]
    c.cache[pg[:, None], heads, at] = b & 255
    c.cache[pg[:, None], heads, at + 1] = b >> 8


def zero_queries(c, nodes, heads):
    c.q[nodes], c.hq[nodes] = 0, 0
    c.q[:, heads], c.hq[:, heads] = 0, 0


ZERO_ROWS = [([20, 9], [400, 300]), ([40], [260]), ([4, 2], [400, 300]), ([2], [260]),   # row tiles of 64; few rows
             ([20] * 64, list(range(257, 385, 2)))]      # several tiles of a unit in one run


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("vis", [False, True])
@pytest.mark.parametrize("counts,lens", ZERO_ROWS)
def test_attention_zero_queries_among_growing_rows(tv, counts, lens, vis, d, bf16):
    """Queries of zeros (padded nodes, a head of zeros): their scores are zero throughout, while the other rows' maxima
    grow in a later tile of keys and in the tree.  With prefixes per node, one row of the tile sees no prefix."""
    c = Case(30, counts, lens, 8, 2, d, 64, bf16, "chain", vis=vis)
    zero_queries(c, [1, counts[0] - 1], [3])
    for r, n in enumerate(lens):
        scale_keys(c, r, np.arange(128, n), 16)
    c.k, c.hk = c.k * 64, c.hk * 64            # exact
    if vis:
        c.vis[:] = np.repeat(lens, counts)
        c.vis[0] = 0
    out, lse, err = c.run(tv)
    assert int(err) == 0
    c.check(out, lse)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("vis", [False, True])
@pytest.mark.parametrize("factor", [2, 16])
@pytest.mark.parametrize("counts,lens", ZERO_ROWS)
def test_attention_zero_keys_before_larger_scores(tv, counts, lens, factor, vis, d, bf16):
    """128 cached keys of zeros (padding that was appended), then keys whose scores are somewhat or far above."""
    c = Case(31, counts, lens, 8, 2, d, 32, bf16, "roots", vis=vis)
    for r, n in enumerate(lens):
        scale_keys(c, r, np.arange(128), 0)
        scale_keys(c, r, np.arange(128, n), factor)
    if vis:
        c.vis[:] = np.repeat(lens, counts)
        c.vis[counts[0] // 2] = 130
    out, lse, err = c.run(tv)
    assert int(err) == 0
    c.check(out, lse)


@pytest.mark.parametrize("vis", [False, True])
@pytest.mark.parametrize("counts,d", [([20] * 8, 128), ([20] * 8, 64), ([4] * 24, 128)])
def test_attention_zero_rows_in_units_that_are_cut(tv, counts, d, vis):
    """The same in units that several runs share, a run having a few tiles of each."""
    n = 4000
    c = Case(32, counts, [n] * len(counts), 8, 2, d, 128, True, "chain", vis=vis)
    zero_queries(c, [3, sum(counts) - 1], [5])
    for r in range(len(counts)):
        if r % 2:
            scale_keys(c, r, np.arange(128), 0)
        t = np.arange(128, n)
        scale_keys(c, r, t[t // 128 % 3 == 1], 4)       # every third tile above the one before it
    if vis:
        c.vis[:] = n
        c.vis[1] = 0
    out, lse, err = c.run(tv)
    assert int(err) == 0
    c.check(out, lse)


def test_attention_expired_wait_reports_failure_in_subprocess(tv):
    """When a bounded wait of the tensor-core kernels runs out, every row of the call is NaN, *err is 1 and the status
    word is not zero; rows that node_cnt leaves out stay.  The failure is planted on the host (TV_TEST_ATTN_KV4_STATUS
    sets the status word where the call would clear it), so no wait runs out."""
    import os
    import subprocess
    import sys
    code = """
import sys
sys.path[:0] = ['tests', '.']
import numpy as np, torch, speculative_decoding_tree_02_gb300 as tv
from test_gpu_kv4 import Case
for counts, cnt in (([40, 12, 3], [40, 0, 2]), ([2, 1, 4], [1, 0, 4]), ([150, 3, 1], [150, 2, 1])):
    for vis in (False, True):
        c = Case(40, counts, [300, 20, 0], 8, 2, 128, 32, True, 'chain', vis=vis, node_cnt=cnt)
        n = sum(counts)
        ws = tv.tree_verify_attn_kv4_workspace(3, max(counts), 8, 2, 128)
        out = torch.full((n, 8, 128), 5.0, dtype=torch.bfloat16, device='cuda')
        lse = torch.full((n, 8), 5.0, device='cuda')
        _, _, err = c.run(tv, out=out, lse=lse, ws=ws)
        torch.cuda.synchronize()
        assert int(err) == 1 and int(ws[:4].view(torch.int32)) == 3
        live = [int(c.off[r]) + i for r in range(3) for i in range(cnt[r])]
        left = [i for i in range(n) if i not in live]
        assert torch.isnan(out[live]).all() and torch.isnan(lse[live]).all()
        assert (out[left] == 5).all() and (lse[left] == 5).all()
        out, lse, err = c.run(tv, want_lse=False)
        assert int(err) == 1 and lse is None and torch.isnan(out[live]).all()
print('failure reported')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, TV_TEST_ATTN_KV4_STATUS="3"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "failure reported" in r.stdout, r.stderr[-3000:]


# ------------------------------------------------------------ a run together
@pytest.mark.parametrize("Hq,Hkv,d,P", [(8, 2, 128, 16), (4, 1, 64, 32)])
def test_prompt_then_verification_steps(tv, Hq, Hkv, d, P):
    """Prompts into the cache, then steps of: node positions, rotation, attention over the cache, acceptance, append
    of the accepted path with the lengths kept on the device; the oracle keeps its own cache."""
    rng = np.random.default_rng(d)
    B, N, V, steps = 3, 12, 50, 4
    prompt = [20, 1, 70]
    table, n_pages = tables(rng, [p + steps * N for p in prompt], P, spare=0)
    rope = ok.rope_table(256, d)
    cache = np.zeros((n_pages, Hkv, P * (d + 4)), np.uint8)
    c = torch.zeros(cache.shape, dtype=torch.uint8, device="cuda")
    off = np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32)
    (_, k, v), (_, hk, hv) = fused(rng, int(off[-1]), Hq, Hkv, d, True)
    zero = np.zeros(B, np.int32)
    lens = ok.append(cache, P, table, zero, hk, hv, off, rope=rope)
    dlen, err = tv.kv4_append(k, v, c, P, dev(table), dev(zero), dev(off), max(prompt), rope=dev(rope))
    tab, dt = dev(table), dev(rope)
    for step in range(steps):
        par, noff, anc, see = forest(rng, [N] * B, "random")
        (q, k, v), (hq, hk, hv) = fused(rng, B * N, Hq, Hkv, d, True)
        tok = rng.integers(0, V, B * N).astype(np.int32)
        amax = rng.integers(0, V, B * N).astype(np.int32)
        for i in range(B * N):                 # most children carry their parent's choice
            p = par[i]
            if p >= 0 and rng.random() < 0.7:
                tok[i] = amax[noff[i // N] + p]
        depth, pos, danc, _, _ = tv.tv_tree_prep(dev(par), dev(noff), dlen, None, N)
        rd, rpos, _, _ = otree.tree_prep(par, noff, lens)
        assert np.array_equal(host(pos), rpos)
        qr, kr, _ = tv.tv_rope(q, k, pos, dt, err=err)
        out, lse, _ = tv.tree_verify_attn_kv4(qr, c, P, tab, dlen, kr, v, dev(noff), danc, N, err=err)
        hqr = ok.f32(ok.bf16_bits(ok.rotate(hq, rpos, rope, False)))
        hkr = ok.f32(ok.bf16_bits(ok.rotate(hk, rpos, rope, False)))
        pre = ok.gather(cache, P, table, zero, lens)
        o, l, av, sa = ok.attention(hqr, pre, hkr, hv, noff, see)
        tol, ltol = ok.attention_tolerance(o, l, av, sa, d, True)
        assert (np.abs(out.float().cpu().numpy() - o) <= tol).all() and (np.abs(host(lse) - l) <= ltol).all()
        acc, _, path, _, _ = tv.accept_longest_path(dev(par), dev(tok), dev(amax), dev(noff), max_nodes=N)
        # the cache takes the rotated rows; acceptance gives the path as it is
        hpath = host(path)
        lens = ok.append(cache, P, table, lens, hkr, hv, noff, hpath)
        dlen, _ = tv.kv4_append(kr, v, c, P, tab, dlen, dev(noff), N, path=path, err=err)
        assert np.array_equal(host(dlen), lens) and int(err) == 0
        assert np.array_equal(host(c), cache)
