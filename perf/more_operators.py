"""Cases of the operators around one sampled serving step over the paged 4-bit cache.

Four operators: ``kv4_attn_mass`` adds up the attention weight that cached
tokens receive, ``kv4_evict_select`` chooses by it which tokens a request keeps,
``kv4_compact`` moves the kept tokens together, and ``accept_sampled`` verifies
drafted tokens against the target's probabilities (temperature, top-k, top-p)
from given random numbers.

``run`` computes a case in plain torch operations (32 bits, 64 where values lie
next to a border; rounded once at the end) or, when ``own`` is true, through
the library's entry points.

Cache format.  ``cache`` is uint8 [n_pages, Hkv, P * (d + 4)], P tokens per
page.  One (page, head) block holds
  K codes   [d/32][P][16 bytes]  chunk c of token t: its dims 32c .. 32c+31
  V codes   [P/16][d][8 bytes]   dim by dim, the 16 tokens of a group
  K scales  bf16 [P], V scales bf16 [P]
Eight codes make a little-endian 32-bit word: item e (a dim of a key, a token
of a value) sits in nibble e//2 + 4*(e%2).  A code is n + 8 with n in -7..7
and stands for scale * n.
"""
import math
import random

import torch

own = False

DEV = "cuda"
NIB = [0, 4, 1, 5, 2, 6, 3, 7]     # nibble of item e


# --------------------------------------------------------------------- cases
def _mass(name, B, rows, mode, Hq, Hkv, d, lmin, lmax, page, decay=1.0, dtype="bf16"):
    return dict(name=name, op="mass", B=B, rows=rows, mode=mode, Hq=Hq, Hkv=Hkv, d=d, lmin=lmin, lmax=lmax, page=page,
                decay=decay, dtype=dtype)


def _accept(name, B, nmin, nmax, tree, V, q, temp, top_k, top_p, dtype="bf16"):
    return dict(name=name, op="accept", B=B, nmin=nmin, nmax=nmax, tree=tree, V=V, q=q, temp=temp, top_k=top_k,
                top_p=top_p, dtype=dtype)


def listed():
    return [
        # weights of one request's decoding step: a single token's rows, where latency counts
        _mass("mass one token", 1, 1, "token", 32, 8, 128, 2048, 2048, 64),
        # weights of a batch's decoding step over ragged prefixes, older steps counting less
        _mass("mass tokens batch", 64, 1, "token", 32, 8, 128, 512, 4096, 64, 0.95),
        # the accepted paths of a verified batch of block drafts (1 + 15 nodes), after they were appended
        _mass("mass paths batch", 64, 16, "path", 32, 8, 128, 512, 4096, 64),
        # prompts in chunks: 1024 new tokens of each of eight requests weigh all tokens before them
        _mass("mass prompt chunk", 8, 1024, "prompt", 32, 8, 128, 1024, 4096, 64),
        # the small fp32 geometry (4 heads of 64 on one KV head): 60 rows over 128 tokens
        _mass("mass tiny f32", 1, 60, "prompt", 4, 1, 64, 128, 128, 16, dtype="f32"),
        # a batch over its budget chooses what it keeps
        dict(name="select batch", op="select", B=64, Hkv=8, lmin=512, lmax=4096, bmin=1024, bmax=2048, sink=4,
             recent=128),
        # one long request comes down to an eighth
        dict(name="select long", op="select", B=1, Hkv=8, lmin=131072, lmax=131072, bmin=16384, bmax=16384, sink=4,
             recent=1024),
        # a batch's kept tokens move to pages of its own (its old ones are shared), and are read back
        dict(name="compact batch", op="compact", B=32, Hkv=8, d=128, lmin=512, lmax=4096, kmin=512, kmax=1024, page=64,
             dtype="bf16"),
        # one long request's kept tokens
        dict(name="compact long", op="compact", B=1, Hkv=8, d=128, lmin=65536, lmax=65536, kmin=8192, kmax=8192,
             page=128, dtype="bf16"),
        # block drafts of a batch (a root and 15 drawn tokens each), sampled at temperature 0.8 in a nucleus
        _accept("accept chains", 64, 16, 16, "chain", 151936, True, 0.8, 0, 0.95),
        # one request's hybrid tree: retrieved nodes come without a distribution, the nodes of the draft with one
        _accept("accept hybrid tree", 1, 61, 61, "random", 151936, True, 1.0, 50, 0.9),
        # the small fp32 geometry: retrieved nodes only, no truncation
        _accept("accept tiny f32", 1, 60, 60, "random", 1000, False, 1.0, 0, 1.0, "f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["mass", "mass", "mass", "select", "compact", "accept", "accept"])
    Hkv, g = rng.choice([(8, 4), (8, 4), (1, 4), (2, 8), (4, 1), (4, 7), (2, 16)])
    d = rng.choice([128, 128, 64])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    B = _log(rng, 1, 64)
    if op == "accept":
        V = _log(rng, 1000, 151936)
        nmax = _log(rng, 1, min(113, 1024 * 151936 // (B * V)))
        return dict(op=op, B=B, nmin=rng.randint(1, nmax), nmax=nmax, tree=rng.choice(["chain", "random"]), V=V,
                    q=rng.random() < 0.6, temp=rng.choice([0.0, 1.0, round(rng.uniform(0.3, 1.5), 2)]),
                    top_k=rng.choice([0, 0, _log(rng, 1, 1000)]),
                    top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 2)]), dtype=dtype)
    if op == "select":
        lmax = _log(rng, 1, min(131072, (1 << 18) // B))
        bmax = _log(rng, 1, max(1, lmax + lmax // 4))
        return dict(op=op, B=B, Hkv=Hkv, lmin=rng.randint(0, lmax), lmax=lmax, bmin=rng.randint(1, bmax), bmax=bmax,
                    sink=rng.choice([0, 4, 17]), recent=rng.choice([0, 33, _log(rng, 1, lmax)]))
    if op == "compact":
        lmax = _log(rng, 1, min(65536, (1 << 17) // B))
        kmax = _log(rng, 1, max(1, min(lmax, 32768 // B)))
        return dict(op=op, B=B, Hkv=Hkv, d=d, lmin=rng.randint(0 if B > 3 else 1, lmax), lmax=lmax,
                    kmin=rng.randint(0 if B > 3 else 1, kmax), kmax=kmax, page=page, dtype=dtype)
    mode = rng.choice(["token", "path", "prompt"])
    lmax = _log(rng, 1, min(8192, 131072 // B))
    rows = 1 if mode == "token" else _log(rng, 1, min(lmax, 64 if mode == "path" else 1024))
    if dtype == "f32":
        # the fp32 geometry is a small one
        B, lmax, rows = min(B, 4), min(lmax, 1024), min(rows, 64, lmax, 1024)
    B = max(1, min(B, 1_000_000_000 // (rows * Hkv * g * lmax)))
    lmin = rng.randint(min(rows, lmax), lmax)
    case = _mass("", B, rows, mode, Hkv * g, Hkv, d, lmin, lmax, page, rng.choice([1.0, 0.9]), dtype)
    del case["name"]
    return case


# -------------------------------------------------------------------- inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed & 0x7FFFFFFF)


def _spread(lo, hi, B):
    """B lengths in [lo, hi], ragged and in no order: part of the case, the same for every seed."""
    return [lo + int((i * 0.6180339887498949 + 0.5) % 1.0 * (hi - lo + 1)) for i in range(B)]


def _ints(values):
    return torch.tensor(values, device=DEV, dtype=torch.int32)


def _offsets(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return _ints(off)


def _table(gen, lens, page, spare=0):
    """Block table of requests with ``lens`` tokens over randomly ordered pages (-1 where there is none), the number of
    pages, and ``spare`` pages that no request holds."""
    used = [(n + page - 1) // page for n in lens]
    cols = max(1, max(used))
    n_pages = max(1, sum(used)) + spare
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    have = torch.arange(cols, device=DEV)[None, :] < _ints(used)[:, None]
    table = torch.full((len(lens), cols), -1, dtype=torch.int32, device=DEV)
    table[have] = perm[:sum(used)]
    return table, n_pages, perm[n_pages - spare:]


def _pack(x, page, values):
    """[pages, Hkv, page, d] fp32 rows -> (codes uint8, scales bf16) as a block holds them."""
    s = (x.abs().amax(-1) / 7 * 1.004).to(torch.bfloat16)
    n = torch.round(x / s.float()[..., None]).clamp(-7, 7)
    code = (n + 8).to(torch.uint8)
    pages, H, P, d = x.shape
    if values:
        it = code.view(pages, H, P // 16, 16, d).transpose(3, 4).reshape(pages, H, -1, 8)     # [.., group, d, 16]
    else:
        it = code.view(pages, H, P, d // 32, 32).transpose(2, 3).reshape(pages, H, -1, 8)     # [.., chunk, P, 32]
    nib = it[..., [0, 2, 4, 6, 1, 3, 5, 7]].reshape(pages, H, -1, 4, 2)                       # item of nibble m
    return (nib[..., 0] | (nib[..., 1] << 4)).reshape(pages, H, -1), s


def _new_cache(gen, n_pages, case):
    """A pool whose every slot holds a quantised row (recycled pages: slots past a request's end are stale)."""
    H, P, d = case["Hkv"], case["page"], case["d"]
    cache = torch.empty((n_pages, H, P * (d + 4)), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (H * P * d))
    for p0 in range(0, n_pages, step):
        n = min(step, n_pages - p0)
        parts = [_pack(torch.randn((n, H, P, d), generator=gen, device=DEV), P, v) for v in (False, True)]
        cache[p0:p0 + n] = torch.cat([parts[0][0], parts[1][0]] + [c[1].view(torch.uint8).reshape(n, H, -1)
                                                                  for c in parts], 2)
    return cache


def _scores(gen, *shape):
    """What accumulated weights look like: heavy tails, and tokens that no row has looked at."""
    x = torch.exp(3 * torch.randn(shape, generator=gen, device=DEV) - 4)
    return torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.1, torch.zeros_like(x), x)


def _mass_counts(case):
    """Per request: tokens cached before the rows' own, rows taken, rows held."""
    total = _spread(case["lmin"], case["lmax"], case["B"])
    if case["mode"] == "path":
        cnt = _spread(1, case["rows"], case["B"])
    else:
        cnt = [case["rows"]] * case["B"]
    cnt = [min(c, t) for c, t in zip(cnt, total)]
    held = [case["rows"]] * case["B"] if case["mode"] == "path" else cnt
    return total, cnt, held


def _prepare_mass(case, gen, st):
    B, H, Hq, d, P = (case[k] for k in ("B", "Hkv", "Hq", "d", "page"))
    total, cnt, held = _mass_counts(case)
    table, n_pages, _ = _table(gen, total, P)
    n = sum(held)
    off = _offsets(held)
    # the rows as a fused projection's output holds them, q beside k and v
    qkv = torch.randn((n, Hq + 2 * H, d), generator=gen, device=DEV).to(_dt(case))
    st.update(cache=_new_cache(gen, n_pages, case), table=table, q=qkv[:, :Hq], cache_len=_ints(total), row_off=off,
              old_len=_ints([t - c for t, c in zip(total, cnt)]), path=None, max_rows=max(cnt), counts=cnt, held=held,
              totals=total, score=_scores(gen, B, H, max(total) + 64))
    st["score_out"] = torch.zeros_like(st["score"])
    if case["mode"] == "path":
        # increasing node indices of the accepted path, the root first
        path = torch.full((B, case["rows"]), -1, dtype=torch.int32)
        host = torch.Generator().manual_seed(case["rows"])
        for r, c in enumerate(cnt):
            pick = torch.cat([torch.zeros(1, dtype=torch.int64),
                              1 + torch.randperm(held[r] - 1, generator=host)[:c - 1].sort().values])
            path[r, :c] = pick[:c].to(torch.int32)
        st["path"] = path.to(DEV)
    # the attention's log-sum-exp of every row that counts
    lse = torch.zeros((n, Hq), device=DEV)
    K = _keys(st["cache"], P, d)
    for r, (rows, see) in enumerate(_rows_of(st)):
        s = _row_scores(st, K, r, rows)
        lse[rows] = torch.logsumexp(torch.where(see[None, :, None, :], s, torch.full_like(s, -math.inf)),
                                    3).permute(1, 0, 2).reshape(-1, Hq)
    st["lse"] = lse


def _prepare_accept(case, gen, st):
    V, B = case["V"], case["B"]
    cnt = _spread(case["nmin"], case["nmax"], B)
    n = sum(cnt)
    # next-token logits: a broad bulk and a few tens of tokens that stand out
    x = torch.randn((n, V), generator=gen, device=DEV) * 1.5
    peaks = torch.randint(0, V, (n, 40), generator=gen, device=DEV)
    x.scatter_add_(1, peaks, 5 + 9 * torch.rand((n, 40), generator=gen, device=DEV))
    st["p"] = x.to(_dt(case))
    st["q"] = None
    temp = case["temp"]
    # the drafter's distribution: the target's, blurred, at the request's temperature
    guess = x
    del x
    step = max(1, (1 << 27) // V)
    tok_rows = torch.empty((n, 4), dtype=torch.int64, device=DEV)
    if case["q"]:
        st["q"] = torch.empty((n, V), device=DEV)
    for i in range(0, n, step):
        z = guess[i:i + step] + 0.6 * torch.randn(guess[i:i + step].shape, generator=gen, device=DEV)
        z = torch.softmax(z / (temp if temp > 0 else 1.0), 1)
        tok_rows[i:i + step] = torch.topk(z, 4, 1).indices
        if st["q"] is not None:
            st["q"][i:i + step] = z
    del guess
    # the trees' shapes are part of the case, the same for every seed
    shape = random.Random(n)
    parent, host_drawn = [], []
    for c in cnt:
        for i in range(c):
            parent.append(-1 if i == 0 else i - 1 if case["tree"] == "chain" else int(shape.random() ** 1.5 * i))
            host_drawn.append(1 if case["tree"] == "chain" or i % 3 else 0)
    st["parent"] = _ints(parent)
    st["drawn"] = None if case["tree"] == "chain" or st["q"] is None else torch.tensor(host_drawn, dtype=torch.uint8,
                                                                                      device=DEV)
    # a node's token: drawn from its parent's row of q, or one of the drafter's favourites there
    first = _offsets(cnt).tolist()
    src = torch.tensor([first[r] + max(parent[first[r] + i], 0) for r in range(B) for i in range(cnt[r])], device=DEV)
    like = tok_rows[src, torch.randint(0, 4, (n,), generator=gen, device=DEV)]
    if st["q"] is not None:
        pick = torch.empty(n, dtype=torch.int64, device=DEV)
        for i in range(0, n, step):
            pick[i:i + step] = torch.multinomial(st["q"][src[i:i + step]], 1, generator=gen)[:, 0]
        like = pick if st["drawn"] is None else torch.where(st["drawn"].bool(), pick, like)
    kids = {}
    depth = [0] * n
    for r in range(B):
        for i in range(1, cnt[r]):
            p = first[r] + parent[first[r] + i]
            kids[p] = kids.get(p, 0) + 1
            depth[first[r] + i] = depth[p] + 1
    st.update(tok=like.to(torch.int32), node_off=_ints(first), counts=cnt, most_kids=max(kids.values(), default=0),
              max_depth=max(depth), u=torch.rand((n,), generator=gen, device=DEV),
              race=torch.empty((B, V), device=DEV).exponential_(generator=gen),
              temp=torch.full((B,), temp, device=DEV), top_k=torch.full((B,), case["top_k"], dtype=torch.int32, device=DEV),
              top_p=torch.full((B,), case["top_p"], device=DEV), ws=None)
    i32 = dict(dtype=torch.int32, device=DEV)
    st["outputs"] = (torch.empty(B, **i32), torch.empty(B, **i32), torch.empty((B, st["max_depth"] + 1), **i32),
                     torch.empty(B, **i32))


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case=case)
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "accept":
        _prepare_accept(case, gen, st)
    elif case["op"] == "mass":
        _prepare_mass(case, gen, st)
    else:
        B, H = case["B"], case["Hkv"]
        lens = _spread(case["lmin"], case["lmax"], B)
        st["cache_len"] = _ints(lens)
        if case["op"] == "select":
            budget = _spread(case["bmin"], case["bmax"], B)
            keep = max(1, max(min(a, b) for a, b in zip(lens, budget)))
            st.update(score=_scores(gen, B, H, max(1, case["lmax"])), budget=_ints(budget), max_len=max(lens),
                      idx=torch.empty((B, H, keep), **i32), score_out=torch.zeros((B, H, keep), device=DEV),
                      new_len=torch.empty(B, **i32))
        else:
            kept = [min(a, b) for a, b in zip(lens, _spread(case["kmin"], case["kmax"], B))]
            pages = [(k + case["page"] - 1) // case["page"] for k in kept]
            table, n_pages, free = _table(gen, lens, case["page"], sum(pages))
            dst = torch.full((B, max(1, max(pages))), -1, **i32)
            dst[torch.arange(dst.shape[1], device=DEV)[None, :] < _ints(pages)[:, None]] = free
            # kept tokens: the highest of random weights, in order
            w = torch.rand((B, H, max(1, max(lens))), generator=gen, device=DEV)
            t = torch.arange(w.shape[2], device=DEV)
            w = torch.where(t < st["cache_len"][:, None, None], w, torch.full_like(w, -1.0))
            rank = w.argsort(2, descending=True).argsort(2)
            new_len = _ints(kept)
            at = torch.where(rank < new_len[:, None, None], t, torch.full_like(t, 1 << 30)).sort(2).values
            at = at[:, :, :max(1, max(kept))]
            n = sum(kept)
            st.update(cache=_new_cache(gen, n_pages, case), table=table, dst=dst, new_len=new_len, counts=kept,
                      idx=torch.where(at < (1 << 30), at, torch.full_like(at, -1)).to(torch.int32).contiguous(),
                      max_keep=max(kept), out_off=_offsets(kept),
                      outputs=tuple(torch.empty((n, H, case["d"]), dtype=_dt(case), device=DEV) for _ in range(2)))
    st["err"] = torch.zeros(1, **i32)
    return st


# ---------------------------------------------------------------- plain form
def _unpack(cache, page, d, values):
    """K or V fp32 [pages, Hkv, page, d] of the whole pool."""
    pages, H, _ = cache.shape
    c = cache[:, :, page * d // 2 * values: page * d // 2 * (1 + values)]
    nib = torch.stack([c & 15, c >> 4], -1).view(pages, H, -1, 8)[..., NIB]
    if values:
        n = nib.view(pages, H, page // 16, d, 16).transpose(3, 4).reshape(pages, H, page, d)
    else:
        n = nib.view(pages, H, d // 32, page, 32).transpose(2, 3).reshape(pages, H, page, d)
    o = page * d + 2 * page * values
    s = cache[:, :, o:o + 2 * page].contiguous().view(torch.bfloat16).float()
    return (n.float() - 8.0) * s[..., None]


def _keys(cache, page, d):
    return _unpack(cache, page, d, False)


def _rows_of(st):
    """Per request the indices of the rows that count and what each sees [rows, tokens]."""
    off = 0
    for r, (n, c, held) in enumerate(zip(st["totals"], st["counts"], st["held"])):
        j = torch.arange(c, device=DEV)
        rows = off + (j if st["path"] is None else st["path"][r, :c].long())
        yield rows, torch.arange(n, device=DEV)[None, :] < (n - c + j + 1)[:, None]
        off += held


def _row_scores(st, K, r, rows):
    """scale * q.k [Hkv, rows, group, tokens] of request r's rows, fp32."""
    case = st["case"]
    H, d, P, n = case["Hkv"], case["d"], case["page"], st["totals"][r]
    k = K[st["table"][r, :(n + P - 1) // P].long()].permute(1, 0, 2, 3).reshape(H, -1, d)[:, :n]
    q = st["q"][rows].float().view(len(rows), H, -1, d).permute(1, 0, 2, 3)
    return (q.reshape(H, -1, d) @ k.transpose(1, 2)).view(H, len(rows), -1, n) * (1.0 / math.sqrt(d))


def _plain_mass(st):
    case = st["case"]
    H = case["Hkv"]
    K = _keys(st["cache"], case["page"], case["d"])
    out = st["score_out"].clone()
    for r, (rows, see) in enumerate(_rows_of(st)):
        n, c = st["totals"][r], st["counts"][r]
        s = _row_scores(st, K, r, rows) - st["lse"][rows].view(len(rows), H, -1).permute(1, 0, 2)[..., None]
        w = torch.where(see[None, :, None, :], torch.exp(s), torch.zeros_like(s)).sum((1, 2))
        before = torch.where(torch.arange(n, device=DEV) < n - c, st["score"][r, :, :n], torch.zeros_like(w))
        out[r, :, :n] = case["decay"] * before + w
    return out


def _order_key(x):
    """int64 in the order of fp32 ``x`` (zeros alike, NaN below all)."""
    b = (x + 0.0).view(torch.int32).long()
    k = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    return torch.where(torch.isnan(x), torch.full_like(k, -(1 << 40)), k)


def _plain_select(st):
    case = st["case"]
    ln, x = st["cache_len"].long(), st["score"]
    keep = st["idx"].shape[2]
    n = torch.minimum(ln, st["budget"].long())
    ms = n.clamp(max=case["sink"])
    mr = (n - ms).clamp(max=case["recent"])
    t = torch.arange(x.shape[2], device=DEV)
    c = lambda v: v[:, None, None]  # noqa: E731
    mid = (t >= c(ms)) & (t < c(ln - mr))
    key = torch.where(mid, _order_key(x), torch.full((), -(1 << 41), device=DEV))
    rank = key.sort(dim=2, descending=True, stable=True).indices.argsort(2)
    kept = (t < c(ms)) | ((t >= c(ln - mr)) & (t < c(ln))) | (mid & (rank < c(n - ms - mr)))
    at = torch.where(kept, t, torch.full_like(t, 1 << 40)).sort(2).values[:, :, :keep]
    some = at < (1 << 40)
    s = torch.gather(x, 2, at.clamp(max=x.shape[2] - 1))
    return (torch.where(some, at, torch.full_like(at, -1)).to(torch.int32), torch.where(some, s, st["score_out"]),
            n.to(torch.int32))


def _plain_compact(st):
    case = st["case"]
    dt, P = _dt(case), case["page"]
    vals = []
    for v in (False, True):
        X = _unpack(st["cache"], P, case["d"], v)
        parts = []
        for r, k in enumerate(st["counts"]):
            t = st["idx"][r, :, :k].long()                                             # [H, k]
            page = st["table"][r].long()[t // P]
            h = torch.arange(case["Hkv"], device=DEV)[:, None]
            parts.append(X[page, h, t % P].transpose(0, 1))
        vals.append(torch.cat(parts).to(dt))
    return vals[0], vals[1]


def _plain_probs(st, rows):
    """The target's distribution of each request's row, fp64 [B, V]."""
    l = st["p"][rows].float().double()
    V = l.shape[1]
    T = st["temp"].double()[:, None]
    best = torch.zeros_like(l).scatter_(1, l.argmax(1, keepdim=True), 1.0)
    s, _ = l.sort(1, descending=True)
    k = st["top_k"].long()
    k = torch.where(k > 0, k.clamp(max=V), torch.full_like(k, V))
    kth = s.gather(1, (k - 1)[:, None])
    warm = torch.where(T > 0, T, torch.ones_like(T))
    w = torch.exp((s - s[:, :1]) / warm) * (s >= kth)
    above = w.cumsum(1) - w
    count = (above < st["top_p"].double()[:, None] * w.sum(1, keepdim=True)).sum(1, keepdim=True).clamp(min=1)
    floor = torch.where(st["top_p"][:, None] < 1, torch.maximum(kth, s.gather(1, count - 1)), kth)
    p = torch.exp((l - s[:, :1]) / warm) * (l >= floor)
    p = p / p.sum(1, keepdim=True)
    return torch.where(T > 0, p, best)


def _plain_accept(st):
    B = st["case"]["B"]
    b = torch.arange(B, device=DEV)
    first = st["node_off"][:-1].long()
    cnt = (st["node_off"][1:] - st["node_off"][:-1]).long()
    N = max(st["counts"])
    i = torch.arange(N, device=DEV)
    at = (first[:, None] + i).clamp(max=st["parent"].numel() - 1)
    parent = torch.where(i < cnt[:, None], st["parent"].long()[at], torch.full_like(at, -2))
    cur = torch.zeros(B, dtype=torch.int64, device=DEV)
    depth, live = cur.clone(), cur == 0
    path = torch.full((B, st["max_depth"] + 1), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = 0
    last = torch.zeros((B, st["race"].shape[1]), dtype=torch.float64, device=DEV)
    for _ in range(st["max_depth"] + 1):
        row = first + cur
        p = _plain_probs(st, row)
        q = st["q"][row].double() if st["q"] is not None else None
        kid = (parent == cur[:, None]) & (i > 0)
        nth = kid.cumsum(1)
        nxt = torch.full_like(cur, -1)
        now = p
        for c in range(st["most_kids"]):
            has = kid & (nth == c + 1)
            ask = live & has.any(1) & (nxt < 0)
            ch = has.int().argmax(1)
            x = st["tok"].long()[first + ch]
            px = now[b, x]
            drawn = torch.full_like(ask, q is not None)
            if st["drawn"] is not None:
                drawn = st["drawn"][first + ch].bool()
            qx = torch.where(drawn, q[b, x], torch.ones_like(px)) if q is not None else torch.ones_like(px)
            ok = st["u"].double()[first + ch] * qx < px
            nxt = torch.where(ask & ok, ch, nxt)
            rest = now.clone()
            rest[b, x] = 0.0
            if q is not None:
                rest = torch.where(drawn[:, None], (now - q).clamp(min=0), rest)
            z = rest.sum(1, keepdim=True)
            rest = torch.where(z > 0, rest / z, p)
            greedy = st["temp"][:, None] <= 0
            now = torch.where((ask & ~ok)[:, None] & ~greedy, rest, now)
        stop = live & (nxt < 0)
        last = torch.where(stop[:, None], now, last)
        live = live & ~stop
        cur = torch.where(live, nxt, cur)
        depth = depth + live
        path = torch.where(live[:, None] & (torch.arange(path.shape[1], device=DEV) == depth[:, None]), cur[:, None], path)
    bonus = (last / st["race"].double()).argmax(1)
    return tuple(t.to(torch.int32) for t in (depth, cur, path, bonus))


# ----------------------------------------------------------------------- run
def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"mass": _plain_mass, "select": _plain_select, "compact": _plain_compact, "accept": _plain_accept}[op](st)
    import speculative_decoding_tree_02_gb300 as tv
    if op == "mass":
        out, _ = tv.kv4_attn_mass(st["q"], st["lse"], st["cache"], case["page"], st["table"], st["cache_len"],
                                  st["row_off"], st["max_rows"], score=st["score"], old_len=st["old_len"],
                                  path=st["path"], causal=True, decay=case["decay"], score_out=st["score_out"],
                                  err=st["err"])
        return out
    if op == "select":
        idx, score, new_len, _ = tv.kv4_evict_select(st["score"], st["cache_len"], st["budget"], st["max_len"],
                                                     n_sink=case["sink"], n_recent=case["recent"], idx=st["idx"],
                                                     score_out=st["score_out"], new_len=st["new_len"], err=st["err"])
        return idx, score, new_len
    if op == "compact":
        tv.kv4_compact(st["cache"], case["page"], st["table"], st["cache_len"], st["idx"], st["new_len"], st["max_keep"],
                       dst_table=st["dst"], err=st["err"])
        # the moved tokens as the values that the cache now holds for them
        k, v, _ = tv.kv4_gather(st["cache"], case["page"], st["dst"], st["out_off"], st["max_keep"],
                                outputs=st["outputs"], err=st["err"])
        return k, v
    if st["ws"] is None:     # a serving loop keeps its workspace
        st["ws"] = tv.accept_sampled_workspace(case["B"], st["p"].shape[0], case["V"], st["p"].device)
    return tv.accept_sampled(st["parent"], st["tok"], st["p"], st["node_off"], st["u"], st["race"], q_prob=st["q"],
                             drawn=st["drawn"], temperature=st["temp"], top_k=st["top_k"], top_p=st["top_p"],
                             max_nodes=max(st["counts"]), max_depth=st["max_depth"], ws=st["ws"], outputs=st["outputs"])


# ---------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass."""
    B = case["B"]
    if case["op"] == "accept":
        e = 2 if case["dtype"] == "bf16" else 4
        # the rows that the walk reaches: about two accepted tokens in a chain or a tree, and the last row
        rows = sum(min(3, c) for c in _spread(case["nmin"], case["nmax"], B))
        V = case["V"]
        return {"bytes": rows * V * e + B * V * (4 + (4 if case["q"] else 0)), "flops": 4 * rows * V}
    H = case["Hkv"]
    lens = _spread(case["lmin"], case["lmax"], B)
    if case["op"] == "select":
        kept = sum(min(a, b) for a, b in zip(lens, _spread(case["bmin"], case["bmax"], B)))
        return {"bytes": max(1, H * (4 * sum(lens) + 8 * kept)), "flops": H * sum(lens)}
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "compact":
        n = max(1, sum(min(a, b) for a, b in zip(lens, _spread(case["kmin"], case["kmax"], B))))
        # codes and scales out and in, the list; the values read back
        return {"bytes": n * H * (2 * (d + 4) + 4) + n * H * (d + 4 + 2 * d * e), "flops": 2 * n * H * d}
    total, cnt, _ = _mass_counts(case)
    see = sum(c * (n - c) + c * (c + 1) // 2 for n, c in zip(total, cnt))      # (row, token) pairs
    Hq = case["Hq"]
    return {"bytes": sum(total) * H * (d // 2 + 2 + 8) + sum(cnt) * Hq * (d * e + 4), "flops": 2 * d * Hq * see}


# --------------------------------------------------------------------- exact
def _code64(cache, page, d, pages, t, values):
    """K or V [n, Hkv, d] in fp64 of tokens ``t`` [n, Hkv] of a request on ``pages``, decoded item by item."""
    n, H = t.shape
    head = torch.arange(H, device=DEV).expand(n, H)
    blk = cache[pages.long()[t // page], head]                                       # [n, H, bytes]
    slot = (t % page)[..., None]
    dim = torch.arange(d, device=DEV)
    item = slot % 8 if values else dim % 8
    nib = (item // 2 + 4 * (item % 2)).expand(n, H, d)
    if values:
        at = page * d // 2 + (slot // 16 * d + dim) * 8 + slot % 16 // 8 * 4 + nib // 2
    else:
        at = dim // 32 * page * 16 + slot * 16 + dim % 32 // 8 * 4 + nib // 2
    code = (blk.gather(2, at).long() >> (4 * (nib % 2))) & 15
    o = page * d + 2 * page * values + 2 * slot
    lo, hi = (blk.gather(2, o + i).int() for i in (0, 1))
    return (code - 8).double() * ((lo << 16) | (hi << 24)).view(torch.float32).double()


def _exact_mass(case, st):
    H, g = case["Hkv"], case["Hq"] // case["Hkv"]
    out = st["score_out"].double()
    old, row_off = st["old_len"].tolist(), st["row_off"].tolist()
    for r, n in enumerate(st["cache_len"].tolist()):
        t = torch.arange(n, device=DEV)
        k = _code64(st["cache"], case["page"], case["d"], st["table"][r], t[:, None].expand(n, H), False)
        if st["path"] is None:
            rows = torch.arange(row_off[r], row_off[r + 1], device=DEV)
        else:
            mine = st["path"][r][st["path"][r] >= 0].long()
            rows = row_off[r] + mine
        last = old[r] + torch.arange(len(rows), device=DEV)          # the row's own token, the last that it sees
        for h in range(H):
            w = torch.zeros(n, dtype=torch.float64, device=DEV)
            for i in range(h * g, (h + 1) * g):
                a = (st["q"][rows, i].double() @ k[:, h].T) / math.sqrt(case["d"])
                a = a - st["lse"][rows, i].double()[:, None]
                w += torch.exp(a.masked_fill(t[None, :] > last[:, None], -math.inf)).sum(0)
            keep = st["score"][r, h, :n].double() * case["decay"]
            keep[old[r]:] = 0
            out[r, h, :n] = keep + w
    return out


def _exact_select(case, st):
    idx = torch.full_like(st["idx"], -1)
    out = st["score_out"].double()
    lens, budget = st["cache_len"].tolist(), st["budget"].tolist()
    n_kept = []
    for r, (n, b) in enumerate(zip(lens, budget)):
        keep = min(n, b)
        n_kept.append(keep)
        a = min(case["sink"], keep)
        z = min(case["recent"], keep - a)
        for h in range(case["Hkv"]):
            x = st["score"][r, h, :n].double()
            mid = torch.argsort(-x[a:n - z], stable=True)[:keep - a - z] + a
            some = torch.cat([torch.arange(a, device=DEV), mid, torch.arange(n - z, n, device=DEV)]).sort().values
            idx[r, h, :keep] = some.to(torch.int32)
            out[r, h, :keep] = x[some]
    return idx, out, _ints(n_kept)


def _exact_row(l, T, k, top_p):
    """The target's distribution over one row of logits."""
    l = l.double()
    if T <= 0:
        p = torch.zeros_like(l)
        p[(l == l.max()).nonzero()[0]] = 1.0
        return p
    value, group = torch.unique(l, return_inverse=True)              # ascending classes of equal logits
    size = torch.bincount(group).double()
    if 0 < k < l.numel():
        above = size.flip(0).cumsum(0).flip(0) - size                # tokens with a higher logit
        size = torch.where(above < k, size, torch.zeros_like(size))
    mass = size * torch.exp((value - value[-1]) / T)
    if top_p < 1:
        above = mass.flip(0).cumsum(0).flip(0) - mass
        on = above < top_p * mass.sum()
        on[-1] = True
        mass = torch.where(on, mass, torch.zeros_like(mass))
    return (mass / mass.sum() / size.clamp(min=1))[group]


def _exact_accept(case, st):
    off, parent, tok = (st[k].tolist() for k in ("node_off", "parent", "tok"))
    u = st["u"].double().tolist()
    drawn = [int(st["q"] is not None)] * len(tok) if st["drawn"] is None else st["drawn"].tolist()
    top_p = float(st["top_p"][0])                                    # as the type holds them
    temp = float(st["temp"][0])
    out = [[], [], [], []]
    for r in range(case["B"]):
        a, n = off[r], off[r + 1] - off[r]
        walk = [0]
        while True:
            cur = walk[-1]
            p = _exact_row(st["p"][a + cur], temp, case["top_k"], top_p)
            left, on = p.clone(), None
            for c in (i for i in range(1, n) if parent[a + i] == cur):
                x = tok[a + c]
                if u[a + c] * (float(st["q"][a + cur, x]) if drawn[a + c] else 1.0) < float(left[x]):
                    on = c
                    break
                if temp <= 0:
                    continue
                if drawn[a + c]:
                    left = torch.relu(left - st["q"][a + cur].double())
                else:
                    left[x] = 0
                left = left / left.sum() if float(left.sum()) > 0 else p.clone()
            if on is None:
                break
            walk.append(on)
        out[0].append(len(walk) - 1)
        out[1].append(walk[-1])
        out[2].append(walk + [-1] * (st["max_depth"] + 1 - len(walk)))
        out[3].append(int((left / st["race"][r].double()).argmax()))
    return tuple(_ints(o) for o in out)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "mass":
        return _exact_mass(case, st)
    if case["op"] == "select":
        return _exact_select(case, st)
    if case["op"] == "accept":
        return _exact_accept(case, st)
    outs = []
    for v in (False, True):
        parts = [_code64(st["cache"], case["page"], case["d"], st["table"][r], st["idx"][r, :, :k].long().T, v)
                 for r, k in enumerate(st["counts"])]
        outs.append(torch.cat(parts))
    return tuple(outs)
