"""CPU checks of eviction and of sampled verification: the oracles against their
definitions, and what the entry points refuse before any launch."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT
from oracle import kv4_evict as oe
from oracle import sampled as osm

LIB = os.path.join(ROOT, "speculative_decoding_tree_02_gb300", "libtreeverify.so")


# ------------------------------------------------------------------- eviction
def test_mass_of_full_attention_sums_to_the_rows():
    rng = np.random.default_rng(0)
    L, Hkv, g, d, n = 23, 2, 3, 16, 5
    K = rng.standard_normal((L, Hkv, d)).astype(np.float32)
    q = rng.standard_normal((n, Hkv * g, d)).astype(np.float32)
    s = np.einsum("nhgd,lhd->nhgl", q.reshape(n, Hkv, g, d).astype(np.float64), K.astype(np.float64)) / np.sqrt(d)
    lse = np.log(np.exp(s).sum(-1)).reshape(n, -1).astype(np.float32)
    m, tol = oe.attn_mass(q, lse, [K], [L], [0, n], n, None, L)
    assert np.allclose(m.sum(-1), n * g, atol=1e-5)
    m2, _ = oe.attn_mass(q, lse, [K], [L], [0, n], n, m.astype(np.float32), L, decay=0.5)
    assert np.allclose(m2, 1.5 * m, rtol=1e-6) and (tol > 0).all()


def test_mass_masks():
    rng = np.random.default_rng(1)
    K = rng.standard_normal((9, 1, 16)).astype(np.float32)
    q = rng.standard_normal((4, 1, 16)).astype(np.float32)
    lse = np.array([[0.0], [-np.inf], [0.3], [0.1]], np.float32)
    m, _ = oe.attn_mass(q, lse, [K], [9], [0, 4], 4, None, 12, old_len=[5], causal=True, vis=[7, 9, 2, -3])
    w = lambda i, n: np.where(np.arange(9) < n, np.exp(K[:, 0].astype(np.float64) @ q[i, 0] / 4 - lse[i, 0]), 0)  # noqa: E731
    assert np.allclose(m[0, 0, :9], w(0, 6) + w(2, 2)) and np.isnan(m[0, 0, 9:]).all()


@pytest.mark.parametrize("n,budget,sink,recent", [(10, 4, 1, 1), (10, 10, 2, 3), (10, 20, 4, 4), (7, 3, 2, 5), (7, 3, 9, 9),
                                                  (5, 0, 1, 1), (0, 4, 1, 1), (12, 5, 0, 0)])
def test_select_keeps_sinks_recent_and_the_highest(n, budget, sink, recent):
    rng = np.random.default_rng(n + budget)
    x = rng.integers(0, 4, (1, 1, 16)).astype(np.float32)
    x[0, 0, 3] = np.nan
    idx, kept, new_len = oe.evict_select(x, [n], [budget], sink, recent, 32)
    m = min(n, budget)
    t = idx[0, 0, :m]
    assert new_len[0] == m and (idx[0, 0, m:] == -1).all() and (np.diff(t) > 0).all()
    a = min(sink, m)
    z = min(recent, m - a)
    assert set(range(a)) <= set(t.tolist()) and set(range(n - z, n)) <= set(t.tolist())
    rest = [i for i in t if a <= i < n - z]
    out = [i for i in range(a, n - z) if i not in rest]
    rank = lambda i: (-np.inf if np.isnan(x[0, 0, i]) else x[0, 0, i], -i)  # noqa: E731
    assert not rest or not out or min(map(rank, rest)) > max(map(rank, out))


# ------------------------------------------------------------------- sampling
def test_target_probs_truncation():
    x = np.log(np.array([0.4, 0.3, 0.1, 0.1, 0.06, 0.04]))
    assert np.allclose(osm.target_probs(x), [0.4, 0.3, 0.1, 0.1, 0.06, 0.04])
    assert np.allclose(osm.target_probs(x, top_k=2), np.array([4, 3, 0, 0, 0, 0]) / 7)
    assert np.allclose(osm.target_probs(x, top_k=3), np.array([4, 3, 1, 1, 0, 0]) / 9)      # a class stays whole
    assert np.allclose(osm.target_probs(x, top_p=0.6), np.array([4, 3, 0, 0, 0, 0]) / 7)
    assert np.allclose(osm.target_probs(x, top_p=0.0), [1, 0, 0, 0, 0, 0])
    assert np.allclose(osm.target_probs(x, top_k=2, top_p=0.5), [1, 0, 0, 0, 0, 0])         # 4/7 reaches a half
    assert np.allclose(osm.target_probs(x, temperature=0.0), [1, 0, 0, 0, 0, 0])
    assert osm.target_probs(np.array([-np.inf, np.nan])).sum() == 0
    assert np.allclose(osm.target_probs(np.array([np.inf, 1.0, np.inf])), [0.5, 0, 0.5])


@pytest.mark.parametrize("drawn_mix", ["drawn", "proposed", "mixed"])
def test_the_rule_is_lossless(drawn_mix):
    """The first emitted token (accepted child or bonus) is distributed as the target says.  30000 trials: 5 standard
    deviations of a frequency are at most 5 sqrt(0.25 / 30000) = 0.0145."""
    rng = np.random.default_rng({"drawn": 1, "proposed": 2, "mixed": 3}[drawn_mix])
    V, trials = 5, 30000
    logits = np.array([[1.0, 0.2, -0.5, 0.7, -2.0]], np.float32)
    want = osm.target_probs(logits[0], 0.8, 4, 0.95)
    q1 = np.array([0.1, 0.5, 0.2, 0.1, 0.1])
    drawn = {"drawn": [1, 1, 1], "proposed": [0, 0, 0], "mixed": [0, 1, 1]}[drawn_mix]
    parent = np.array([-1, 0, 0, 0])
    count = np.zeros(V)
    toks = np.where(np.array(drawn), rng.choice(V, (trials, 3), p=q1), np.array([3, 1, 1]))
    u, race = rng.random((trials, 4)), rng.exponential(size=(trials, 1, V))
    rows = np.repeat(logits, 4, 0)
    q = np.repeat(q1[None].astype(np.float32), 4, 0)
    for t in range(trials):
        acc, best, _, bonus, _ = osm.verify(parent, np.concatenate([[0], toks[t]]), rows, [0, 4], u[t], race[t], 3, q,
                                            np.array([0] + drawn), [0.8], [4], [0.95])
        count[toks[t, best[0] - 1] if acc[0] else bonus[0]] += 1
    assert np.abs(count / trials - want).max() < 0.0145


# ------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls here pass placeholder addresses")
    if not os.path.exists(LIB):
        subprocess.run([sys.executable, "-m", "speculative_decoding_tree_02_gb300.build"], cwd=ROOT, check=True)
    import speculative_decoding_tree_02_gb300 as tv
    return tv.load_library()


B_ = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)
MASS = dict(q=B_, ldq=128, lse=B_, dtype=1, cache=B_, n_pages=4, page=16, table=B_, table_ld=4, cache_len=B_, row_off=B_,
            path=None, path_ld=0, vis=None, old=B_, causal=1, B=1, max_rows=4, rows=4, max_len=64, Hq=2, Hkv=1, d=64,
            scale=0.125, decay=1.0, s_in=B_, in_ld=64, s_out=B_, out_ld=64, err=None, stream=None)
SELECT = dict(score=B_, ld=64, cache_len=B_, budget=B_, sink=1, recent=1, B=1, H=1, max_len=64, idx=B_, idx_ld=32, out=ODD,
              out_ld=32, new_len=ODD, err=None, stream=None)
COMPACT = dict(cache=B_, n_pages=4, page=16, table=B_, table_ld=4, cache_len=B_, idx=B_, idx_ld=32, new_len=B_, B=1,
               max_keep=32, dst=None, dst_ld=0, H=1, d=64, err=None, stream=None)
SAMPLED = dict(parent=B_, tok=B_, p=B_, dtype=1, V=100, ld=100, q=B_, ldq=100, drawn=None, node_off=B_, B=1, max_nodes=4,
               rows=4, max_depth=3, T=None, k=None, tp=None, u=B_, race=B_, ldr=100, acc=B_, best=B_, path=B_, bonus=B_,
               ws=B_, ws_bytes=80, stream=None)
FLOATS = {"scale", "decay"}


def call(lib, fn, base, **change):
    args = [ctypes.c_float(v) if k in FLOATS else v for k, v in {**base, **change}.items()]
    return getattr(lib, fn)(*args)


@pytest.mark.parametrize("want,change", [
    (-1, dict(dtype=2)), (-1, dict(B=-1)), (-1, dict(max_rows=-1)), (-1, dict(Hq=3, Hkv=2)), (-1, dict(page=0)),
    (-2, dict(page=24)), (-2, dict(d=96, ldq=192)), (-2, dict(B=70000)), (-1, dict(scale=0.0)), (-1, dict(scale=float("nan"))),
    (-1, dict(decay=1.5)), (-1, dict(decay=-0.1)), (-1, dict(decay=float("nan"))), (-1, dict(out_ld=63)), (-1, dict(in_ld=63)),
    (-1, dict(in_ld=64, out_ld=128)), (-1, dict(cache_len=None)), (-1, dict(row_off=None)), (-1, dict(s_out=None)),
    (-1, dict(old=None)), (-1, dict(path=B_, path_ld=0)), (-1, dict(table=None)), (-1, dict(cache=None)), (-1, dict(q=None)),
    (-1, dict(lse=None)), (-1, dict(ldq=120)), (-1, dict(ldq=132)), (-1, dict(q=ODD)), (-1, dict(cache=ODD)),
    (-2, dict(max_rows=1 << 30, Hq=64, Hkv=1, ldq=4096)), (-2, dict(Hq=65, Hkv=1, ldq=65 * 64)), (-2, dict(table_ld=1 << 28)), (0, dict(B=0)), (0, dict(max_len=0))])
def test_attn_mass_refusals(lib, want, change):
    assert call(lib, "kv4_attn_mass", MASS, **change) == want


@pytest.mark.parametrize("want,change", [
    (-1, dict(B=-1)), (-1, dict(H=0)), (-1, dict(sink=-1)), (-1, dict(recent=-1)), (-1, dict(ld=63)), (-1, dict(out_ld=31)),
    (-2, dict(B=70000)), (-2, dict(max_len=500000, ld=500000)), (-1, dict(cache_len=None)), (-1, dict(budget=None)),
    (-1, dict(new_len=None)), (-1, dict(new_len=B_)), (-1, dict(budget=ODD)), (-1, dict(score=None)), (-1, dict(idx=None)), (-1, dict(out=B_)),
    (0, dict(B=0))])
def test_evict_select_refusals(lib, want, change):
    assert call(lib, "kv4_evict_select", SELECT, **change) == want


@pytest.mark.parametrize("want,change", [
    (-1, dict(B=-1)), (-1, dict(max_keep=-1)), (-1, dict(H=0)), (-1, dict(page=0)), (-2, dict(page=8)), (-2, dict(d=32)),
    (-2, dict(B=70000)), (-2, dict(table_ld=1 << 28)), (-2, dict(dst=B_, dst_ld=1 << 28)), (-1, dict(max_keep=33)),
    (-1, dict(cache=None)), (-1, dict(cache=ODD)), (-1, dict(table=None)), (-1, dict(idx=None)), (-1, dict(new_len=None)),
    (-1, dict(cache_len=None)), (0, dict(B=0)), (0, dict(max_keep=0))])
def test_compact_refusals(lib, want, change):
    assert call(lib, "kv4_compact", COMPACT, **change) == want


@pytest.mark.parametrize("want,change", [
    (-1, dict(dtype=3)), (-1, dict(B=-1)), (-1, dict(V=0)), (-1, dict(ld=99)), (-1, dict(ldr=99)), (-1, dict(ldq=99)),
    (-1, dict(q=None, drawn=B_)), (-2, dict(max_nodes=1025)), (-2, dict(V=840000, ld=840000, ldq=840000, ldr=840000, k=B_)),
    (-2, dict(V=420000, ld=420000, ldq=420000, ldr=420000, tp=B_, dtype=0)), (-2, dict(V=(1 << 20) + 1, ld=1 << 21, ldq=1 << 21, ldr=1 << 21)),
    (-2, dict(B=70000)), (-1, dict(node_off=None)), (-1, dict(acc=None)), (-1, dict(parent=None)), (-1, dict(p=None)),
    (-1, dict(u=None)), (-1, dict(race=None)), (-4, dict(ws=None)), (-4, dict(ws_bytes=79)), (-4, dict(ws=ODD)),
    (0, dict(B=0))])
def test_sampled_refusals(lib, want, change):
    assert call(lib, "accept_sampled", SAMPLED, **change) == want


def test_binding_refuses_host_and_mistyped_tensors(lib):
    import speculative_decoding_tree_02_gb300 as tv
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        tv.kv4_evict_select(torch.zeros(1, 2, 8), z(1), z(1), 8, max_keep=4)
    with pytest.raises(TypeError):
        tv.kv4_evict_select(torch.zeros(1, 2, 8, dtype=torch.float64), z(1), z(1), 8, max_keep=4)
    with pytest.raises(ValueError):
        tv.kv4_evict_select(torch.zeros(1, 2, 8), z(1), z(1), 8)
    cache = torch.zeros(2, 1, 16 * 68, dtype=torch.uint8)
    with pytest.raises(ValueError):
        tv.kv4_compact(cache, 16, z(1, 2), z(1), z(1, 2, 4), z(1), 4)                 # idx for two heads, cache of one
    with pytest.raises(ValueError):
        tv.kv4_attn_mass(torch.zeros(3, 2, 128), torch.zeros(3, 2), cache, 16, z(1, 2), z(1), z(2), 3, max_len=8)
    with pytest.raises(ValueError):
        tv.kv4_attn_mass(torch.zeros(3, 2, 64), torch.zeros(3, 2), cache, 16, z(1, 2), z(1), z(2), 3)
    with pytest.raises(ValueError):
        tv.accept_sampled(z(2), z(2), torch.zeros(2, 10), z(2), torch.zeros(2), torch.ones(1, 9))
    with pytest.raises(TypeError):
        tv.accept_sampled(z(2), z(2), torch.zeros(2, 10, dtype=torch.float16), z(2), torch.zeros(2), torch.ones(1, 10))
