"""GPU tests of kv4_attn_mass, kv4_evict_select and kv4_compact at the edges of what their contracts allow."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from oracle import kv4_evict as oe
from test_gpu_evict import Mass
from test_gpu_kv4 import prefixes, random_pool, tables

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("g,path", [(1, False), (3, True)])
def test_mass_of_more_than_two_to_the_24_rows(tv, g, path):
    """Rows numbered 2^24 and above: a handful weighs something, all others have lse = inf."""
    n, d, L, old = (1 << 24) + 77, 64, 200, 100
    rng = np.random.default_rng(g)
    table, n_pages = tables(rng, [L], 64)
    pool = random_pool(rng, n_pages, 1, 64, d)
    live = np.array([0, 3, 60, (1 << 24) - 1, 1 << 24, (1 << 24) + 5, n - 1])       # numbers in the request's list
    rows = n - 1 - live if path else live                                           # places in q
    hq = torch.from_numpy(rng.standard_normal((live.size, g, d)).astype(np.float32)).to(torch.bfloat16)
    hl = (3 + rng.random((live.size, g))).astype(np.float32)
    q = torch.zeros((n, g, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, g), float("inf"), device="cuda")
    q[dev(rows)], lse[dev(rows)] = hq.cuda(), dev(hl)
    i32 = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    src = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")[None] if path else None
    out, err = tv.kv4_attn_mass(q, lse, dev(pool[0]), 64, dev(table), i32(L), i32(0, n), n, old_len=i32(old), path=src,
                                causal=True, max_len=L)
    assert int(err) == 0
    # row by row: what each live row sees, as a request of its own
    keys = [k for k, _ in prefixes(pool, table, [L], 64)]
    want, tol = np.zeros((1, L)), np.zeros((1, L))
    for j, x, l in zip(live, hq.float().numpy(), hl):
        w, t = oe.attn_mass(x[None], l[None], keys, [L], [0, 1], 1, None, L, vis=[min(L, old + int(j) + 1)])
        want, tol = want + w[0], tol + t[0]
    # (sums of n g numbers, zeros but for the live ones, whose additions are what rounds: 2^-24 each)
    tol = tol + live.size * g * 2.0 ** -24 * want
    off = np.abs(host(out)[0] - want) > tol
    assert off.sum() == 0


@pytest.mark.parametrize("rows", [4, 60])            # 16 and 240 per KV head: both bf16 kernels
@pytest.mark.parametrize("bf16", [True, False])
def test_mass_tells_of_a_path_beyond_max_rows(tv, rows, bf16):
    """Accepted rows behind the first max_rows are left out, and *err says so; a path that ends there is whole."""
    m = Mass(11, [90, 70], [rows, rows], 8, 2, 64, 16, bf16, path=True)
    out, err = m.run(tv)
    m.check(out)
    assert int(err) == 0 and m.path[0, rows] == -1
    m.max_rows = rows - 1
    out, err = m.run(tv)
    assert int(err) == 1
    m.check(out)
    m.path[:, rows - 1] = -1                             # the same rows without the entry that was left out
    again, err = m.run(tv)
    assert int(err) == 0 and torch.equal(out, again)
    m.path = m.path[:, :rows - 1].copy()                 # no column behind max_rows
    again, err = m.run(tv)
    assert int(err) == 0 and torch.equal(out, again)


def test_empty_batches(tv):
    """No request: all four operators return empty outputs and no error."""
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = tv.kv4_new_cache(3, 16, 2, 64)
    q, lse = torch.zeros(0, 4, 64, device="cuda"), torch.zeros(0, 4, device="cuda")
    score = torch.zeros(0, 2, 40, device="cuda")
    for kw in (dict(score=score), dict(max_len=40), dict(score=score, score_out=torch.zeros(0, 2, 48, device="cuda"))):
        out, err = tv.kv4_attn_mass(q, lse, cache, 16, z(0, 3), z(0), z(1), 4, old_len=z(0), **kw)
        assert out.shape[0] == 0 and int(err) == 0
    idx, kept, new_len, err = tv.kv4_evict_select(score, z(0), z(0), 40, max_keep=8)
    assert idx.shape == (0, 2, 8) and kept.shape == (0, 2, 8) and new_len.numel() == 0 and int(err) == 0
    assert int(tv.kv4_compact(cache, 16, z(0, 3), z(0), idx, new_len, 8)) == 0
    outs = tv.accept_sampled(z(0), z(0), torch.zeros(0, 50, device="cuda"), z(1), torch.zeros(0, device="cuda"),
                             torch.zeros(0, 50, device="cuda"), max_nodes=4)
    assert [t.numel() for t in outs] == [0, 0, 0, 0]


def test_requests_without_tokens(tv):
    """Two requests that hold nothing, with and without room for scores."""
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for room in (0, 7):
        idx, kept, new_len, err = tv.kv4_evict_select(torch.zeros(2, 3, room, device="cuda"), z(2), z(2) + 5, room, 1, 1, max_keep=4)
        assert bool((idx == -1).all()) and new_len.tolist() == [0, 0] and int(err) == 0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("d,P", [(64, 16), (128, 64)])
@pytest.mark.parametrize("rows,g,path", [(120, 4, False), (50, 4, True), (520, 1, False), (90, 7, True)])
def test_mass_of_many_rows_with_nan(tv, rows, g, path, d, P, bf16):
    """More than 192 rows per KV head, split over the CTAs of a cluster: NaN keys, lse and rows reach only what sees them."""
    H, L = 2, 700
    m = Mass(rows + d, [L], [rows], g * H, H, d, P, bf16, path=path, causal=False, vis=True)
    src = m.path[0, :rows] if path else np.arange(rows)
    m.vis[:] = m.rng.integers(0, 600, m.vis.size)
    a, b, c, e = (int(src[i]) for i in (rows // 5, rows // 3, rows // 2, rows - 1))
    m.vis[[a, b, c, e]] = [L, 60, 0, 130]
    m.lse[[a, b, c, e]] = 2.0
    m.lse[c] = NAN                                       # sees nothing
    page, slot = m.table[0, 650 // P], 650 % P           # a key whose scale is NaN, seen by row a alone
    cache, kn, ks, vn, vs = m.pool
    cache[page, 1, P * d + 2 * slot:P * d + 2 * slot + 2] = [0xC0, 0x7F]
    ks[page, 1, slot] = NAN
    out, err = m.run(tv)
    m.check(out)
    assert int(err) == 0 and bool(out[0, 1, 650].isnan()) and int(out.isnan().sum()) == 1
    m.lse[b, g] = NAN                                    # of KV head 1
    out, err = m.run(tv)
    m.check(out)
    assert int(err) == 0 and int(out.isnan().sum()) == 61 and bool(out[0, 1, :60].isnan().all())
    m.q[e, 0], m.hq[e, 0] = NAN, NAN                     # a row of KV head 0
    out, _ = m.run(tv)
    m.check(out)
    assert int(out[0, 0].isnan().sum()) == 130
    m.lse[e, 0] = -INF                                   # which now saw nothing, it is said
    out, _ = m.run(tv)
    m.check(out)
    assert not bool(out[0, 0].isnan().any())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,g", [(120, 4), (600, 1), (60, 6)])
def test_mass_of_many_rows_with_bad_pages_and_rows(tv, rows, g, bf16):
    """More than 192 rows per KV head: bad page entries, rows outside the tensor, lengths and rows beyond their bounds."""
    H, lens = 2, [600, 333]
    m = Mass(rows, lens, [rows, rows - 7], g * H, H, 64, 32, bf16, causal=False)
    m.table[0, 3], m.table[0, 17], m.table[1, 0] = -1, 10 ** 6, m.pool[0].shape[0]
    m.page_ok = [~np.isin(np.arange(600) // 32, [3, 17]), np.arange(333) // 32 != 0]
    out, err = m.run(tv)
    m.check(out)
    assert int(err) == 1
    # rows outside the tensor, at both ends and in the middle of a path
    m = Mass(rows + 1, lens, [rows, rows - 7], g * H, H, 64, 32, bf16, path=True, causal=True)
    n = m.lse.shape[0]
    m.path[0, [0, rows // 2, rows - 1]] = [n, 2 ** 31 - 1, n + 5]
    out, err = m.run(tv)
    m.check(out)
    assert int(err) == 1
    # an offset that begins before the tensor
    m = Mass(rows + 2, lens, [rows, rows - 7], g * H, H, 64, 32, bf16, causal=False)
    m.off = m.off - 3
    out, err = m.run(tv)
    m.check(out)
    assert int(err) == 1
    # rows past max_rows, tokens past max_len
    m = Mass(rows + 3, lens, [rows, rows - 7], g * H, H, 64, 32, bf16, causal=False)
    m.max_rows = rows - 9
    out, err = m.run(tv)
    assert int(err) == 1
    m.check(out)
    before = torch.full((2, H, m.cols), 9.0, device="cuda")
    out, err = m.run(tv, max_len=301, score_out=before.clone())
    assert int(err) == 1 and bool((out[:, :, 301:] == 9).all())


@pytest.mark.parametrize("pages,cols", [(3, 0), (0, 2)])
def test_move_without_pages_or_columns(tv, pages, cols):
    """Requests that hold nothing, over a table of no columns or a cache of no pages; a token to be kept is an error."""
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.full((pages, 2, 16 * 68), 7, dtype=torch.uint8, device="cuda")
    for dst in (None, z(2, 3)):
        assert int(tv.kv4_compact(cache, 16, z(2, cols), z(2), z(2, 2, 4), z(2), 4, dst_table=dst)) == 0
        assert int(tv.kv4_compact(cache, 16, z(2, cols), z(2) + 5, z(2, 2, 4), z(2) + 1, 4, dst_table=dst)) == 1
    assert bool((cache == 7).all())


def test_the_largest_batches(tv):
    """65535 requests through the weights, the choice and the move: as the same requests in batches of 8192."""
    B, H, P, d = 65535, 1, 16, 64
    rng = np.random.default_rng(90)
    lens = rng.integers(0, 17, B).astype(np.int32)
    cache = torch.from_numpy(rng.integers(0, 256, (B, H, P * (d + 4)), dtype=np.uint8)).cuda()
    scales = torch.rand((B, H, 2 * P), device="cuda") * 0.2 + 0.2
    cache[:, :, P * d:] = scales.to(torch.bfloat16).view(torch.uint8)
    table = np.stack([rng.permutation(B)], 1).astype(np.int32)
    budget = rng.integers(0, 12, B).astype(np.int32)
    lse = (3 + rng.random((B, 2))).astype(np.float32)
    for bf16 in (True, False):
        q = torch.from_numpy(rng.standard_normal((B, 2, d)).astype(np.float32)).cuda().to(torch.bfloat16 if bf16 else torch.float32)

        def run(b0, b1, pool):
            n = b1 - b0
            off = dev(np.arange(n + 1, dtype=np.int32))
            s, e = tv.kv4_attn_mass(q[b0:b1], dev(lse[b0:b1]), pool, P, dev(table[b0:b1]), dev(lens[b0:b1]), off, 1, max_len=16)
            idx, kept, new, _ = tv.kv4_evict_select(s, dev(lens[b0:b1]), dev(budget[b0:b1]), 16, 1, 1, max_keep=12, err=e)
            tv.kv4_compact(pool, P, dev(table[b0:b1]), dev(lens[b0:b1]), idx, new, 12, err=e)
            assert int(e) == 0
            return s, idx, torch.where(idx >= 0, kept, torch.zeros_like(kept)), new
        a, b = cache.clone(), cache.clone()
        whole = run(0, B, a)
        parts = [run(b0, min(b0 + 8192, B), b) for b0 in range(0, B, 8192)]
        for t, w in zip(zip(*parts), whole):
            assert torch.equal(torch.cat(t), w)
        assert torch.equal(a, b) and bool((whole[0] > 0).any())
        assert np.array_equal(host(whole[3]), np.minimum(lens, budget))
