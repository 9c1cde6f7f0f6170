"""GPU tests of accept_sampled at the edges of what its contract allows, against oracle/sampled.py (fp64)."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from oracle import kv4 as ok
from oracle import sampled as osm
from test_gpu_sampled import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(T=[0.7], k=[20], p=[0.9])])
def test_no_nodes_by_max_nodes(tv, kw):
    """max_nodes 0: no request has a node, whatever the offsets say, and neither a row nor the workspace is touched."""
    c = Case(50, [3, 5], 100, **kw)
    acc, best, path, bonus = c.run(tv, max_nodes=0, max_depth=2, ws=torch.empty(0, dtype=torch.uint8, device="cuda"))
    for t in (acc, best, path, bonus):
        assert bool((t == -1).all())


def test_nodes_beyond_max_nodes_are_left_out(tv):
    """The same as the requests without those nodes."""
    c = Case(51, [9, 4, 12], 300, T=[0.8], p=[0.95])
    got = c.run(tv, max_nodes=5)
    keep = np.concatenate([np.arange(a, min(a + 5, b)) for a, b in zip(c.off, c.off[1:])])
    for name in ("parent", "tok", "logits", "q", "drawn", "u"):
        setattr(c, name, getattr(c, name)[keep])
    c.off = np.array([0, 5, 9, 14], np.int32)
    for a, b in zip(got, c.run(tv)):
        assert np.array_equal(host(a), host(b))
    c.check(got, most=0.4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k,total", [(1000, 0, 4e-5), (1024, 1000, 4e-5), (20000, 900, 4e-5), (20000, 0, 2e-4), (3000, 0, 1e-3)])
def test_a_nucleus_of_many_small_tokens(tv, V, k, total, dtype):
    """One token holds nearly everything, the others 1e-8 to 1e-6 each, and top-p ends among them.  The masses that are
    compared are sums of at most 100 + V / 2048 roundings (2^-24 of the whole each), so every token whose class lies
    further than that from the border is kept, or is not: the token of each request that race favours by 1e12 is then the
    answer, or the first is."""
    B = 48
    rng = np.random.default_rng(V + k)
    w = rng.uniform(0.5, 1.0, (B, V))
    w *= (total / np.sort(w, 1)[:, -(k or V):].sum(1))[:, None]
    first = rng.integers(0, V, B)
    w[np.arange(B), first] = 1.0
    x = np.log(w).astype(np.float32)
    if dtype == "bf16":
        x = ok.f32(ok.bf16_bits(x))
    top_p = (1 - total * rng.uniform(0.3, 0.7, B)).astype(np.float32)
    race, want = np.ones((B, V), np.float32), first.copy()
    probes = np.zeros(B, int)
    for r in range(B):
        p = osm.target_probs(x[r], 1.0, k)
        value, group = np.unique(p, return_inverse=True)
        mass = np.bincount(group, weights=p)
        off = ((mass.sum() - np.cumsum(mass)) - float(top_p[r]))[group]      # above the class, less the border
        sure = np.flatnonzero((np.abs(off) > (100 + V / 2048) * 2.0 ** -24) & (p > 0) & (np.arange(V) != first[r]))
        t = int(rng.choice(sure))
        race[r, t] = 1e-12
        probes[r] = off[t] < 0
        if off[t] < 0:
            want[r] = t
    assert probes.mean() > 0.2 and (dtype == "bf16" or probes.mean() < 0.8)
    one = np.arange(B + 1, dtype=np.int32)
    p = dev(ok.bf16_bits(x)).view(torch.bfloat16) if dtype == "bf16" else dev(x)
    got = tv.accept_sampled(dev(np.full(B, -1, np.int32)), dev(np.zeros(B, np.int32)), p, dev(one), dev(np.zeros(B, np.float32)),
                            dev(race), top_k=dev(np.full(B, k, np.int32)), top_p=dev(top_p), max_nodes=1)
    assert np.array_equal(host(got[3]), want)


def remainder_case(seed, top, dtype, B=96, V=1000, kids=6, T=1.0, **kw):
    """Stars whose root gives its first child's token a probability near ``top``; that child is refused, those behind it
    meet uniforms within 1e-4..1e-1 (relative) of what they are compared with.  All are proposals."""
    c = Case(seed, [1 + kids] * B, V, "star", dtype="f32", q=None, T=[T], spread=1.0, **kw)
    rng = np.random.default_rng(seed)
    x = c.logits
    if dtype == "bf16":
        x = ok.f32(ok.bf16_bits(x))
    for r in range(B):
        a = c.off[r]
        e = np.exp(x[a].astype(np.float64) / T)
        first = int(rng.integers(0, V))
        x[a, first] = T * np.log((e.sum() - e[first]) * top / (1 - top))
        if dtype == "bf16":
            x[a, first] = ok.f32(ok.bf16_bits(x[a, first:first + 1]))[0]
        p = osm.target_probs(x[a], T, 0 if c.k is None else int(c.k[r]), 1.0 if c.p is None else float(c.p[r]))
        others = np.setdiff1d(np.argsort(-p)[:60], [first])
        c.tok[a + 1:a + 1 + kids] = [first, *rng.permutation(others)[:kids - 1]]
        c.u[a + 1] = np.nextafter(np.float32(1), np.float32(0))
        left = p.copy()
        left[first] = 0.0
        for i in range(a + 2, a + 1 + kids):
            left /= left.sum()
            t = c.tok[i]
            # mostly above (refused, so that the next child is tried too)
            side = 10.0 ** rng.uniform(-4, -1) * rng.choice([1, 1, 1, 1, -1])
            c.u[i] = min(left[t] * (1 + side), 0.99)
            left[t] = 0.0
    c.logits = ok.bf16_bits(x) if dtype == "bf16" else x
    return c


def other_nuclei(c, r):
    """Answers for request r where top-p at the root keeps as much within 40 2^-24 of the whole mass: the sums of at most
    40 roundings each that it compares cannot tell these apart.  The tokens there hold 1e-8..1e-7 of the mass, and what is
    left after the first child 1e-4, so one of them more or less moves p' by up to 1e-3."""
    a, b = int(c.off[r]), int(c.off[r + 1])
    T, k = 1.0 if c.T is None else float(c.T[r]), 0 if c.k is None else int(c.k[r])
    x = ok.f32(c.logits[a:b]) if c.logits.dtype == np.uint16 else c.logits[a:b]
    kept = np.stack([np.where(osm.target_probs(row, T, k, float(c.p[r])) > 0, row, -np.inf) for row in x])
    p = osm.target_probs(x[0], T, k)
    order = np.argsort(-p, kind="stable")
    p = p[order]
    for m in np.flatnonzero(np.abs(np.cumsum(p) - float(c.p[r])) <= 40 * 2.0 ** -24 + p) + 1:
        kept[0] = -np.inf
        kept[0, order[:m]] = x[0, order[:m]]
        yield osm.verify(c.parent[a:b], c.tok[a:b], kept, [0, b - a], c.u[a:b], c.race[r:r + 1], c.depth, None, None, [T])[:4]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top,kw", [(0.9, {}), (0.999, {}), (0.9999, {}), (0.99997, {}), (0.999, dict(T=0.5)),
                                    (0.999, dict(k=[300])), (0.9999, dict(k=[900], p=[0.99999])), (0.7, {})])
def test_little_is_left_after_a_refused_proposal(tv, top, kw, dtype):
    """Relative to one another the remaining probabilities are off by twice 30 2^-23 ln 2 for exponents up to 30, 2^-22 for
    the exponential each, and the remainder's sum of at most 40 roundings by 40 2^-24 of itself, up to four times that
    after further refusals: 5.0e-6 + 0.5e-6 + 9.6e-6 < 1.6e-5.  Decisions nearer than 2e-5 are left out; the inputs
    have next to none."""
    for B in (3, 96):                                # (in the second, rows out of reach are left out)
        c = remainder_case(60, top, dtype, B=B, **kw)
        got = c.run(tv)
        want = osm.verify(c.parent, c.tok, c.logits, c.off, c.u, c.race, c.depth, None, None, c.T, c.k, c.p)
        sure = want[4] > 2e-5
        assert (~sure).mean() <= 0.05
        same = np.all([(host(g) == w).reshape(B, -1).all(1) for g, w in zip(got, want[:4])], 0)
        if c.p is not None:                          # (see other_nuclei)
            for r in np.flatnonzero(sure & ~same):
                same[r] = any(all(np.array_equal(host(g)[r], w[0]) for g, w in zip(got, o)) for o in other_nuclei(c, r))
        assert same[sure].all()


@pytest.mark.parametrize("kw", [{}, dict(T=[0.5]), dict(k=[490])])
def test_a_remainder_that_rounding_would_swallow(tv, kw):
    """Proposals that leave a thousandth of what was left each time, down to 1e-9 of the target's mass: all are refused,
    stay refused, and what is left decides.  Exponents reach 45, so 8e-6 + 0.5e-6 + 9.6e-6 < 2e-5 (as above)."""
    V, B = 500, 64
    for most in (B, 3):
        c = Case(61, [7] * B, V, "star", dtype="f32", q=None, **kw)
        T = 1.0 if c.T is None else float(c.T[0])
        rng = np.random.default_rng(61)
        for r in range(B):
            a = c.off[r]
            t = rng.permutation(V)[:6]
            x = 0.3 * rng.standard_normal(V) - 21 - np.log(V)
            x[t[:3]] = [0.0, -7.0, -14.0]
            c.logits[a] = x * T
            c.tok[a + 1:a + 7] = t
            c.u[a + 1:a + 4] = np.nextafter(np.float32(1), np.float32(0))
            c.u[a + 4:a + 7] = rng.random(3) * 0.005             # (the others hold 1 / 500 each)
        n = int(c.off[most])
        c.off = c.off[:most + 1]
        for name in ("parent", "tok", "logits", "u"):
            setattr(c, name, getattr(c, name)[:n])
        for name in ("race", "T", "k"):
            setattr(c, name, None if getattr(c, name) is None else getattr(c, name)[:most])
        got = c.run(tv)
        want = osm.verify(c.parent, c.tok, c.logits, c.off, c.u, c.race, c.depth, None, None, c.T, c.k)
        sure = want[4] > 2e-5
        assert (~sure).mean() <= 0.05 and (most == 3 or len(set(want[1].tolist())) > 2)
        for g, w in zip(got, want[:4]):
            assert np.array_equal(host(g)[sure], w[sure])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("noise", [0.1, 0.02, 0.005])
def test_a_draft_near_the_target(tv, noise, dtype):
    """Two draws from a q whose total variation to p is small, the first refused: what is left are differences, whose
    numbers are off by 5e-6 (p + p') / z, z the masses that the refusals left multiplied together.  Every decision and
    every last token lies on the side, or is a maximum, that this allows; most decisions allow one alone."""
    B, V = 256, 2000
    c = Case(70, [3] * B, V, "star", dtype="f32", q="drawn", spread=1.0)
    rng = np.random.default_rng(70)
    x = c.logits if dtype == "f32" else ok.f32(ok.bf16_bits(c.logits))
    draft = x.astype(np.float64) + noise * rng.standard_normal(x.shape)
    e = np.exp(draft - draft.max(1, keepdims=True))
    c.q = (e / e.sum(1, keepdims=True)).astype(np.float32)
    p = [osm.target_probs(x[c.off[r]]) for r in range(B)]
    for r in range(B):
        a = c.off[r]
        q = c.q[a].astype(np.float64)
        worse = np.flatnonzero(q > p[r] * (1 + noise / 4))
        c.tok[a + 1] = rng.choice(worse)                             # drawn where q is above p: nothing of it is left
        c.u[a + 1] = np.nextafter(np.float32(1), np.float32(0))
        rest = np.maximum(0.0, p[r] - q)
        ratio = rest / rest.sum() / q
        c.tok[a + 2] = rng.choice(np.flatnonzero((ratio > 0.2) & (ratio < 0.9)))
        t = c.tok[a + 2]
        c.u[a + 2] = np.clip(ratio[t] * (1 + 10.0 ** rng.uniform(-3, 0) * rng.choice([-1, 1])), 0, 0.999)
    c.logits = ok.bf16_bits(x) if dtype == "bf16" else x
    acc, best, _, bonus = (host(t) for t in c.run(tv))
    alone = 0
    for r in range(B):
        a = c.off[r]
        q, t = c.q[a].astype(np.float64), int(c.tok[a + 2])
        r1 = np.maximum(0.0, p[r] - q)
        z = r1.sum()
        r1 /= z
        side = float(c.u[a + 2]) * q[t]
        tol = 5e-6 * (p[r][t] + r1[t]) / z
        yes = acc[r] == 1
        assert acc[r] == 0 or best[r] == 2
        if abs(side - r1[t]) > tol:
            assert yes == (side < r1[t])
            alone += 1
        if not yes:
            left = np.maximum(0.0, r1 - q)
            z2 = left.sum()
            left /= z2
            slack = 5e-6 * (p[r] / z + left) / (z * z2)              # (p' before it: at most p / z)
            f, s = left / c.race[r], slack / c.race[r]
            v = int(bonus[r])
            assert f[v] + s[v] >= (f - s).max()
    assert alone > 0.6 * B and 0.2 * B < (acc == 1).sum() < 0.8 * B


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k,top_p,masked", [(3100, 3000, 1.0, 0.0), (4347, 3000, 1.0, 0.3), (4347, 3000, 0.99, 0.3),
                                              (5700, 0, 0.9999, 0.0), (20000, 19000, 1.0, 0.0), (151936, 150000, 1.0, 0.0),
                                              (9000, 0, 0.99999, 0.5), (700, 690, 1.0, 0.0)])
def test_a_threshold_below_a_65536th_of_the_highest(tv, V, k, top_p, masked, dtype):
    """Truncations that end far below the highest logit, positive and negative logits around them.  As above, one token of
    each request is favoured by race; its class lies away from the border."""
    B = 24
    rng = np.random.default_rng(V)
    x = (3 * rng.standard_normal((B, V)) + rng.uniform(-3, 9, (B, 1))).astype(np.float32)
    x[np.arange(B), rng.integers(0, V, B)] = x.max(1) + 3
    x[rng.random(x.shape) < masked] = -np.inf
    if dtype == "bf16":
        x = ok.f32(ok.bf16_bits(x))
    race, want, probes = np.ones((B, V), np.float32), np.zeros(B, np.int64), np.zeros(B, bool)
    for r in range(B):
        p = osm.target_probs(x[r], 1.0, k)
        value, group = np.unique(p, return_inverse=True)
        mass = np.bincount(group, weights=p)
        off = ((mass.sum() - np.cumsum(mass)) - float(np.float32(top_p)))[group] if top_p < 1 else np.where(p > 0, -1.0, 1.0)
        sure = (np.abs(off) > (100 + V / 2048) * 2.0 ** -24) & np.isfinite(x[r])
        kept = sure & (off < 0)
        # near the border on either side, where the last ones kept or the first ones left out are
        order = np.argsort(-x[r], kind="stable")
        pool = order[kept[order]][-40:] if r % 2 else order[(sure & (off > 0))[order]][:40]
        if pool.size == 0:
            pool = order[kept[order]][-40:]
        t = int(rng.choice(pool))
        race[r, t] = 1e-30
        probes[r] = kept[t]
        q = osm.target_probs(x[r], 1.0, k, float(np.float32(top_p)))
        want[r] = t if kept[t] else int(np.argmax(q))
    assert probes.any()
    one = np.arange(B + 1, dtype=np.int32)
    p = dev(ok.bf16_bits(x)).view(torch.bfloat16) if dtype == "bf16" else dev(x)
    got = tv.accept_sampled(dev(np.full(B, -1, np.int32)), dev(np.zeros(B, np.int32)), p, dev(one), dev(np.zeros(B, np.float32)),
                            dev(race), top_k=dev(np.full(B, k, np.int32)), top_p=dev(np.full(B, top_p, np.float32)), max_nodes=1)
    assert np.array_equal(host(got[3]), want)


@pytest.mark.parametrize("V,dtype,kw", [(835584, "bf16", dict(T=[1.0], p=[0.9])), (417792, "f32", dict(T=[0.7], k=[300], p=[0.95])),
                                        (1 << 20, "bf16", {}), (1 << 20, "f32", {})])
def test_the_largest_vocabularies(tv, V, dtype, kw):
    """All that a row's slices have room for in shared memory, and all that is allowed where nothing is truncated."""
    c = Case(80, [4, 3], V, "star", dtype=dtype, q=None, **kw)
    c.check(c.run(tv, max_nodes=4), most=0.5)
    with pytest.raises(tv.TVError) as e:                 # a slice more
        wide = torch.zeros((7, V + 64), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
        tv.accept_sampled(dev(c.parent), dev(c.tok), wide, dev(c.off), dev(c.u), torch.ones((2, V + 64), device="cuda"),
                          temperature=dev(c.T), top_k=dev(c.k), top_p=dev(c.p), max_nodes=4)
    assert e.value.status == -2


@pytest.mark.parametrize("kind,q", [("star", None), ("chain", "drawn"), ("random", None)])
def test_the_largest_trees(tv, kind, q):
    """1024 nodes in a request, next to one of a single node; in the star all children are refused one after another."""
    c = Case(81, [1024, 1, 700], 3000, kind, dtype="f32", q=q, spread=0.5)
    rng = np.random.default_rng(81)
    if kind == "star":
        for a, n in ((c.off[0], 1024), (c.off[2], 700)):
            c.tok[a + 1:a + n] = rng.permutation(3000)[:n - 1]
            c.u[a + 1:a + n] = np.float32(0.99)
    if kind == "chain":                                  # the draft is the target's own
        x = c.logits.astype(np.float64)
        e = np.exp(x - x.max(1, keepdims=True))
        c.q = (e / e.sum(1, keepdims=True)).astype(np.float32)
        c.u = (c.u * 0.999).astype(np.float32)
    got = c.run(tv, max_nodes=1024)
    c.check(got, most=0.4)
    if kind == "chain":
        assert host(got[0])[0] == 1023 and host(got[2])[0, -1] == 1023
    if kind == "star":
        assert (host(got[0]) == 0).all()


def test_the_largest_batch(tv):
    """65535 requests of 0 to 2 nodes: as in batches of 4096."""
    B, V = 65535, 9
    rng = np.random.default_rng(82)
    counts = rng.integers(0, 3, B)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1])
    first = np.zeros(n, bool)
    first[off[:-1][counts > 0]] = True
    parent = np.where(first, -1, 0).astype(np.int32)
    tok, u = rng.integers(0, V, n).astype(np.int32), rng.random(n).astype(np.float32)
    x, race = rng.standard_normal((n, V)).astype(np.float32), rng.exponential(size=(B, V)).astype(np.float32)
    T, k = rng.uniform(0.2, 2, B).astype(np.float32), rng.integers(0, 6, B).astype(np.int32)
    p = rng.uniform(0.5, 1.1, B).astype(np.float32)

    def run(b0, b1):
        a, b = off[b0], off[b1]
        return tv.accept_sampled(dev(parent[a:b]), dev(tok[a:b]), dev(x[a:b]), dev(off[b0:b1 + 1] - a), dev(u[a:b]),
                                 dev(race[b0:b1]), temperature=dev(T[b0:b1]), top_k=dev(k[b0:b1]), top_p=dev(p[b0:b1]),
                                 max_nodes=2)
    whole = run(0, B)
    parts = [run(b0, min(b0 + 4096, B)) for b0 in range(0, B, 4096)]
    for t, w in zip(zip(*parts), whole):
        assert torch.equal(torch.cat(t), w)
    want = osm.verify(parent, tok, x, off[:301], u, race, 1, None, None, T, k, p)
    sure = want[4] > 2e-5
    for g, w in zip(whole, want[:4]):
        assert np.array_equal(host(g)[:300][sure], w[sure])
