"""GPU parity of accept_sampled against oracle/sampled.py (fp64).

Decisions whose two sides lie within 1e-5 of each other (relative) may go
either way: an fp32 probability is off by a few 2^-24 for its exponent's
argument, times at most 30 for the argument's size, and as much again for the
normaliser, about 4e-6.  The oracle gives each request's smallest distance;
requests below the bound are left out, and the tests' inputs have few."""
import numpy as np
import pytest
import torch

import synth
from gpu_util import dev, host
from oracle import sampled as osm
from oracle.kv4 import bf16_bits

pytestmark = pytest.mark.gpu
MARGIN = 1e-5


def trees(rng, counts, kind):
    parent = []
    for n in counts:
        for i in range(n):
            parent.append(-1 if i == 0 else i - 1 if kind == "chain" else 0 if kind == "star" else int(rng.integers(0, i)))
    return np.array(parent, np.int32), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


class Case:
    def __init__(self, seed, counts, V, kind="random", dtype="bf16", q="mixed", T=None, k=None, p=None, spread=2.0):
        rng = np.random.default_rng(seed)
        self.parent, self.off = trees(rng, counts, kind)
        n, B = int(self.off[-1]), len(counts)
        x = (rng.standard_normal((n, V)) * spread).astype(np.float32)
        self.logits = synth.bf16_bits(x) if dtype == "bf16" else x
        draft = x + rng.standard_normal(x.shape).astype(np.float32)
        e = np.exp(draft - draft.max(1, keepdims=True))
        self.q = (e / e.sum(1, keepdims=True)).astype(np.float32) if q else None
        self.drawn = rng.integers(0, 2, n).astype(np.uint8) if q == "mixed" else None
        src = np.clip(self.parent, 0, None) + np.repeat(self.off[:-1], counts)
        fav = np.argsort(-draft, 1)[:, :3]
        self.tok = fav[src, rng.integers(0, min(3, V), n)].astype(np.int32)
        if q:
            mine = np.array([rng.choice(V, p=e[s] / e[s].sum()) for s in src], np.int32)
            self.tok = np.where(np.ones(n, bool) if self.drawn is None else self.drawn > 0, mine, self.tok).astype(np.int32)
        self.u, self.race = rng.random(n).astype(np.float32), rng.exponential(size=(B, V)).astype(np.float32)
        per = lambda v, t: None if v is None else np.array([v[i % len(v)] for i in range(B)], t)  # noqa: E731
        self.T, self.k, self.p = per(T, np.float32), per(k, np.int32), per(p, np.float32)
        self.depth = max(1, max(counts) - 1)

    def p_tensor(self):
        t = dev(self.logits)
        return t.view(torch.bfloat16) if t.dtype == torch.int16 else t

    def run(self, tv, **kw):
        args = dict(q_prob=dev(self.q), drawn=dev(self.drawn), temperature=dev(self.T), top_k=dev(self.k), top_p=dev(self.p),
                    max_depth=self.depth) | kw
        p = args.pop("p_logits", None)
        return tv.accept_sampled(dev(self.parent), dev(self.tok), self.p_tensor() if p is None else p, dev(self.off),
                                 dev(self.u), dev(self.race), **args)

    def check(self, got, most=0.05):
        want = osm.verify(self.parent, self.tok, self.logits, self.off, self.u, self.race, self.depth, self.q, self.drawn,
                          self.T, self.k, self.p)
        sure = want[4] > MARGIN
        assert (~sure).mean() <= most
        for g, w in zip(got, want[:4]):
            assert np.array_equal(host(g)[sure], w[sure])
        return want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,V,kw", [
    ([1], 1, dict(q=None)),
    ([1, 5, 9], 7, dict()),
    ([60], 1000, dict(q=None)),
    ([16] * 24, 1001, dict(kind="chain", q="drawn", T=[0.8], p=[0.95])),
    ([16] * 24, 4096, dict(kind="chain", q="drawn")),
    ([30, 0, 17, 3] * 5, 2500, dict(T=[1.0, 0.6, 0.0, 1.4], k=[50, 0, 3, 1], p=[0.9, 0.5, 0.3, 1.0])),
    ([12] * 20, 333, dict(kind="star", q="drawn", T=[1.3])),
    ([12] * 20, 333, dict(kind="star", k=[5, 20])),
    ([40] * 12, 20011, dict(q=None, k=[0, 1000, 1, 30000], p=[0.99, 0.0, 1.0])),
    ([20] * 10, 9000, dict(spread=0.05, p=[0.7])),
    ([20] * 10, 9000, dict(spread=30.0, T=[0.1, 10.0], p=[0.7], k=[0, 700])),
])
def test_matches(tv, counts, V, kw, dtype):
    c = Case(len(counts) * 1000 + V, counts, V, dtype=dtype, **kw)
    got = c.run(tv)
    c.check(got)
    for a, b in zip(got, c.run(tv)):
        assert torch.equal(a, b)


def test_real_vocabulary(tv):
    c = Case(1, [16, 7, 16, 12], synth.QWEN3_VOCAB, "chain", q="drawn", T=[0.8, 1.0], p=[0.95, 1.0], k=[0, 50], spread=3.0)
    c.check(c.run(tv))


def test_one_row_workspace_strides_and_streams(tv):
    c = Case(2, [9, 8, 7], 1000, T=[0.7], p=[0.9])
    n = int(c.off[-1])
    wide = torch.full((n, 1500), 99.0, dtype=torch.bfloat16, device="cuda")
    for start in (0, 8, 3):                                  # vector loads, and rows at odd addresses
        p = wide[:, start:start + 1000]
        p.copy_(c.p_tensor())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = c.run(tv, p_logits=p, ws=tv.accept_sampled_workspace(3, n, 1000))
        s.synchronize()
        c.check(got)
    with pytest.raises(tv.TVError) as e:
        c.run(tv, ws=torch.empty(20 * n - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_and_odd_logits(tv, dtype):
    """-inf, the type's lowest, NaN and +inf among the logits; a row with nothing but -inf and NaN."""
    inf, low = float("inf"), float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min)
    for T, k, p in ((1.0, 0, 1.0), (0.5, 3, 1.0), (1.0, 0, 0.6), (2.0, 300, 0.99), (0.0, 0, 1.0)):
        c = Case(3, [6] * 12, 700, dtype="f32", q=None, T=[T], k=[k], p=[p])
        rng = np.random.default_rng(4)
        x = c.logits
        x[rng.random(x.shape) < 0.4] = -inf
        x[rng.random(x.shape) < 0.1] = low
        x[rng.random(x.shape) < 0.1] = np.nan
        x[c.off[1]] = -inf                                   # request 1's root: nothing can be drawn
        x[c.off[2]], x[c.off[2], 5] = np.nan, -inf
        x[c.off[3], [7, 300, 699]] = inf                     # three tokens share everything
        x[c.off[4]] = low                                    # a uniform row
        x[c.off[5]] = -inf
        x[c.off[5], 698] = -2.0                              # one token left
        if dtype == "bf16":
            c.logits = bf16_bits(x)
        got = c.run(tv)
        want = c.check(got, most=0.25)
        assert host(got[3])[1] == -1 and host(got[3])[2] == -1 and want[3][1] == -1


def test_tokens_outside_the_vocabulary_are_refused(tv):
    """Also by a greedy row that has no token to choose."""
    for q in (None, "drawn"):
        c = Case(11, [5] * 4, 50, "star", dtype="f32", q=q, T=[0.0, 1.0])
        c.tok[:] = np.tile([-1, -1, 50, -2, 2 ** 31 - 1], 4)
        c.logits[c.off[0]], c.logits[c.off[1]] = -np.inf, -np.inf
        want = c.check(c.run(tv), most=0.5)
        assert (want[0] == 0).all() and (want[3][:2] == -1).all()


def test_ties_and_repeated_tokens(tv):
    """Equal logits stay together in a truncation; a retrieved token that comes twice is refused the second time; a
    request at temperature 0 takes the lowest index of the highest logits."""
    V = 64
    c = Case(5, [9] * 16, V, "star", dtype="f32", q=None, k=[4], T=[1.0, 0.0])
    c.logits[:] = np.round(c.logits)
    c.tok[:] = c.tok % 3
    c.check(c.run(tv))
    c.u[:] = 0.999999
    want = c.check(c.run(tv), most=1.0)
    assert (want[0][::2] == 0).sum() > 0


def test_draft_equal_to_target_is_accepted(tv):
    c = Case(6, [16] * 8, 500, "chain", dtype="f32", q="drawn")
    x = c.logits.astype(np.float64)
    e = np.exp(x - x.max(1, keepdims=True))
    c.q = (e / e.sum(1, keepdims=True)).astype(np.float32)
    c.u = (c.u * 0.999).astype(np.float32)
    acc = host(c.run(tv)[0])
    assert (acc == 15).all()


def test_a_residual_of_nothing_gives_the_target_again(tv):
    """q above p everywhere it matters: every draw is refused, and nothing is left."""
    c = Case(7, [4] * 6, 40, "star", dtype="f32", q="drawn")
    c.q[:] = 1.0
    c.u[:] = 0.9999
    c.check(c.run(tv))


def test_lossless_on_the_gpu(tv):
    """20000 requests of one retrieved and two drawn children: 5 standard deviations of a frequency are at most
    5 sqrt(0.25 / 20000) = 0.0177."""
    B, V = 20000, 6
    rng = np.random.default_rng(8)
    row = np.array([1.0, 0.2, -0.5, 0.7, -2.0, 0.1], np.float32)
    q = np.array([0.1, 0.4, 0.2, 0.1, 0.1, 0.1])
    tok = np.stack([np.zeros(B), np.full(B, 3), *rng.choice(V, (2, B), p=q)], 1).astype(np.int32)
    par = np.tile(np.array([-1, 0, 0, 0], np.int32), B)
    acc, best, _, bonus = (host(t) for t in tv.accept_sampled(
        dev(par), dev(tok.ravel()), dev(np.tile(row, (4 * B, 1))), dev(np.arange(B + 1, dtype=np.int32) * 4),
        dev(rng.random(4 * B).astype(np.float32)), dev(rng.exponential(size=(B, V)).astype(np.float32)),
        q_prob=dev(np.tile(q.astype(np.float32), (4 * B, 1))), drawn=dev(np.tile(np.array([0, 0, 1, 1], np.uint8), B)),
        temperature=dev(np.full(B, 0.8, np.float32)), top_k=dev(np.full(B, 5, np.int32)),
        top_p=dev(np.full(B, 0.97, np.float32)), max_nodes=4, max_depth=1))
    first = np.where(acc > 0, tok[np.arange(B), np.maximum(best, 0)], bonus)
    want = osm.target_probs(row, 0.8, 5, 0.97)
    assert np.abs(np.bincount(first, minlength=V) / B - want).max() < 0.0177


@pytest.mark.parametrize("B", [4, 20])        # (20 x 16 rows: those out of reach are left out)
def test_captured_and_replayed(tv, B):
    c = Case(9 + B, [16] * B, 2000, "chain", q="drawn", T=[0.8], p=[0.9])
    n = int(c.off[-1])
    args = [dev(c.parent), dev(c.tok), c.p_tensor(), dev(c.off), dev(c.u), dev(c.race)]
    kw = dict(q_prob=dev(c.q), temperature=dev(c.T), top_p=dev(c.p), max_nodes=16, max_depth=c.depth)
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = (torch.empty(B, **i32), torch.empty(B, **i32), torch.empty((B, c.depth + 1), **i32), torch.empty(B, **i32))
    ws = tv.accept_sampled_workspace(B, n, 2000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tv.accept_sampled(*args, ws=ws, outputs=outs, **kw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tv.accept_sampled(*args, ws=ws, outputs=outs, **kw)
        for seed in (1, 2):
            c.u = np.random.default_rng(seed).random(n).astype(np.float32)
            args[4].copy_(torch.from_numpy(c.u))
            g.replay()
            s.synchronize()
            c.check(outs, most=0.1)


def test_forests_whose_rows_are_left_out(tv):
    """Enough rows that unreachable ones are skipped: wide and deep trees, more than 32 children, repeated tokens, retrieved
    and drawn nodes, greedy requests among them; the outputs do not depend on what was skipped."""
    for kind, counts, q in (("random", [64] * 24, "mixed"), ("star", [70] * 20, None), ("chain", [128] * 12, "drawn"),
                            ("random", [200, 1, 0, 90] * 6, None)):
        c = Case(len(counts) + counts[0], counts, 500, kind, dtype="f32", q=q, T=[0.7, 1.0, 0.0], k=[0, 40], p=[0.9, 1.0])
        c.tok[::3] = c.tok[::3] % 7
        got = c.run(tv, ws=torch.full((20 * int(c.off[-1]) + 256,), 255, dtype=torch.uint8, device="cuda"))
        c.check(got, most=0.1)


def test_two_streams_at_once(tv):
    cs = [Case(30 + i, [16] * 16, 3000, "chain", q="drawn", T=[0.9], p=[0.95]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            outs.append([c.run(tv) for _ in range(3)])
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        for got in o:
            c.check(got, most=0.1)
