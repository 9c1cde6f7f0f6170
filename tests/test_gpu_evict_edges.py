"""GPU tests of kv4_attn_mass, kv4_evict_select and kv4_compact at the edges of what their contracts allow."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from oracle import kv4_evict as oe
from test_gpu_evict import Mass
from test_gpu_kv4 import prefixes, random_pool, tables

pytestmark = pytest.mark.gpu


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
