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
