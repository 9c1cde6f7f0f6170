"""Cases of the 4-bit paged KV cache operators.

Four operators of one serving path: ``tv_rope`` rotates the candidate nodes'
query and key rows at their positions, ``kv4_append`` rotates, quantises and
appends rows to the paged cache, ``kv4_gather`` reads cached rows back, and
``tree_verify_attn_kv4`` verifies draft trees against the cache.

``run`` computes a case in plain torch operations (fp32, rounded once at the
end) or, when ``own`` is true, through the library's entry points.

Cache format.  ``cache`` is uint8 [n_pages, Hkv, P * (d + 4)], P tokens per
page.  One (page, head) block holds
  K codes   [d/32][P][16 bytes]  chunk c of token t: its dims 32c .. 32c+31
  V codes   [P/16][d][8 bytes]   dim by dim, the 16 tokens of a group
  K scales  bf16 [P], V scales bf16 [P]
Eight codes make a little-endian 32-bit word: item e (a dim of a key, a token
of a value) sits in nibble e//2 + 4*(e%2).  A code is n + 8 with n in -7..7
and stands for scale * n; a row (token, head) has one scale
  s = max(a/7 rounded up to bf16, 2^-100), a = max|x| over the row, fp32.
and n = x / s rounded to the nearest, ties to even.
"""
import math

import torch

own = False

DEV = "cuda"
NIB = [0, 4, 1, 5, 2, 6, 3, 7]     # nibble of item e
SCALE_MIN = 2.0 ** -100


# --------------------------------------------------------------------- cases
def _attn(name, B, nodes, Hq, Hkv, d, lmin, lmax, page, tree="chain", vis=False, dtype="bf16"):
    return dict(name=name, op="attn", B=B, nodes=nodes, Hq=Hq, Hkv=Hkv, d=d, lmin=lmin, lmax=lmax, page=page,
                tree=tree, vis=vis, dtype=dtype)


def listed():
    return [
        # the small fp32 geometry (4 heads of 64 on one KV head): a 60-node tree over 128 tokens
        _attn("attn tiny tree f32", 1, 60, 4, 1, 64, 128, 128, 16, "random", dtype="f32"),
        # plain decoding of one request: a single token, where latency counts
        _attn("attn one token", 1, 1, 32, 8, 128, 2048, 2048, 64),
        # plain decoding of a batch: single tokens over ragged prefixes
        _attn("attn tokens batch", 64, 1, 32, 8, 128, 512, 4096, 64),
        # block drafts verified in a batch: chains of 1 + 15 tokens over ragged prefixes
        _attn("attn chains batch", 64, 16, 32, 8, 128, 512, 4096, 64),
        # block-size sweep: seven chains under one root, 113 nodes, long prefixes, small pages
        _attn("attn sweep long", 8, 113, 32, 8, 128, 8192, 8192, 16, "sweep"),
        # proposal tree: 64 branches of 16 along one trunk, each node sees its own part of the trunk
        _attn("attn proposal tree", 1, 1024, 32, 8, 128, 4096, 4096, 128, "branches", vis=True),
        # the accepted paths of a verified batch go into the cache, then back as rows
        dict(name="append paths", op="append", B=64, nmin=1, nmax=16, lmin=512, lmax=4096, Hkv=8, d=128, page=64,
             rot=128, inter=False, path=True, dtype="bf16"),
        # prompts of a batch go into the cache, then back as rows (a prompt in chunks reads them)
        dict(name="append prompts", op="append", B=8, nmin=512, nmax=4096, lmin=0, lmax=100, Hkv=8, d=128, page=64,
             rot=128, inter=False, path=False, dtype="bf16"),
        # one request's prefix back as rows for the contiguous attention
        dict(name="gather one", op="gather", B=1, lmin=2048, lmax=2048, Hkv=8, d=128, page=64, dtype="bf16"),
        # a whole batch's prefixes
        dict(name="gather batch", op="gather", B=64, lmin=512, lmax=4096, Hkv=8, d=128, page=64, dtype="bf16"),
        # rotation of a verification step's candidate rows
        dict(name="rope nodes", op="rope", n=1024, pmax=4112, Hq=32, Hkv=8, d=128, rot=128, inter=False, dtype="bf16"),
        # rotation of a prompt
        dict(name="rope prompt", op="rope", n=16411, pmax=131072, Hq=32, Hkv=8, d=128, rot=64, inter=True,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "gather", "rope"])
    Hkv, g = rng.choice([(8, 4), (8, 4), (1, 4), (2, 8), (4, 1), (4, 7), (2, 16)])
    d = rng.choice([128, 128, 64])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    rot = rng.choice([d, d, d // 2])
    if op == "rope":
        return dict(op=op, n=_log(rng, 1, 16384), pmax=_log(rng, 64, 131072), Hq=Hkv * g, Hkv=Hkv, d=d, rot=rot,
                    inter=rng.random() < 0.5, dtype=dtype)
    B = _log(rng, 1, 64)
    lmax = _log(rng, 1, min(8192, 131072 // B))
    lmin = rng.randint(0 if B > 3 else 1, lmax)
    if op == "gather":
        return dict(op=op, B=B, lmin=lmin, lmax=lmax, Hkv=Hkv, d=d, page=page, dtype=dtype)
    if op == "append":
        path = rng.random() < 0.5
        nmax = _log(rng, 1, 64) if path else _log(rng, 1, min(4096, 32768 // B))
        return dict(op=op, B=B, nmin=rng.randint(0 if B > 3 else 1, nmax), nmax=nmax, lmin=lmin, lmax=lmax, Hkv=Hkv,
                    d=d, page=page, rot=rot, inter=rng.random() < 0.5, path=path, dtype=dtype)
    tree = rng.choice(["chain", "random", "branches", "sweep"])
    nodes = 113 if tree == "sweep" else _log(rng, 1, 128)
    if dtype == "f32":
        # the fp32 geometry is a small one
        B, nodes, lmax = min(B, 4), min(nodes, 64), min(lmax, 1024)
        tree = "random" if tree == "sweep" else tree
        lmin = min(lmin, lmax)
    B = max(1, min(B, 200_000_000 // (nodes * Hkv * g * lmax)))
    case = _attn("", B, nodes, Hkv * g, Hkv, d, lmin, lmax, page, tree, rng.random() < 0.3, dtype)
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


def _lengths(lo, hi, B):
    return torch.tensor(_spread(lo, hi, B), device=DEV, dtype=torch.int64)


def _offsets(counts):
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _table(gen, lens, page):
    """Block table of requests with ``lens`` tokens over randomly ordered pages; -1 where there is none."""
    used = (lens + page - 1) // page
    cols = max(1, int(used.max()))
    n_pages = max(1, int(used.sum()))
    perm = torch.randperm(n_pages, generator=gen, device=DEV)
    have = torch.arange(cols, device=DEV)[None, :] < used[:, None]
    table = torch.full((lens.numel(), cols), -1, dtype=torch.int32, device=DEV)
    table[have] = perm[: int(used.sum())].to(torch.int32)
    return table, n_pages


def _rope_table(max_pos, rot):
    """cos | sin of pos * 10000^(-2i/rot), fp32 [max_pos, rot], angles in fp64."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _parents(case, gen):
    n, tree = case["nodes"], case["tree"]
    if tree == "chain":
        return [i - 1 for i in range(n)]
    if tree == "sweep":          # a root and seven chains of 13 .. 19
        par = [-1]
        for b in range(13, 20):
            par += [0] + list(range(len(par), len(par) + b - 1))
        return par
    if tree == "branches":       # branches of 16, each with its own root
        return [-1 if i % 16 == 0 else i - 1 for i in range(n)]
    u = torch.rand(n, generator=gen, device=DEV).tolist()
    return [-1] + [int(u[i] * i) for i in range(1, n)]


def _ancestors(par, words):
    rows = []
    for i, p in enumerate(par):
        rows.append((rows[p] if p >= 0 else 0) | (1 << i))
    sign = lambda w: w - (1 << 64) if w >> 63 else w  # noqa: E731
    return torch.tensor([[sign(r >> (64 * w) & (2 ** 64 - 1)) for w in range(words)] for r in rows], dtype=torch.int64)


def _pack(x, page, values):
    """[pages, Hkv, page, d] fp32 rows -> (codes uint8, scales bf16) as a block holds them."""
    s = _scale(x)
    n = torch.round(x / s[..., None]).clamp(-7, 7)
    code = (n + 8).to(torch.uint8)
    pages, H, P, d = x.shape
    if values:
        it = code.view(pages, H, P // 16, 16, d).transpose(3, 4)                   # [.., group, d, 16]
        it = it.reshape(pages, H, -1, 8)
    else:
        it = code.view(pages, H, P, d // 32, 32).transpose(2, 3).reshape(pages, H, -1, 8)   # [.., chunk, P, 32]
    order = [0, 2, 4, 6, 1, 3, 5, 7]                                               # item of nibble m
    nib = it[..., order].reshape(pages, H, -1, 4, 2)
    byte = nib[..., 0] | (nib[..., 1] << 4)
    return byte.reshape(pages, H, -1), s.to(torch.bfloat16)


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


def prepare(case, seed):
    gen = _gen(seed)
    dt, op = _dt(case), case["op"]
    st = dict(case=case)
    rand = lambda *shape: torch.randn(shape, generator=gen, device=DEV).to(dt)  # noqa: E731
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    if op == "rope":
        n, Hq, Hkv, d = case["n"], case["Hq"], case["Hkv"], case["d"]
        qkv = rand(n, Hq + 2 * Hkv, d)          # one projection's output: q, k and v side by side
        st.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], rope=_rope_table(case["pmax"], case["rot"]),
                  pos=torch.randint(0, case["pmax"], (n,), generator=gen, device=DEV, dtype=torch.int32),
                  outputs=(torch.empty((n, Hq, d), dtype=dt, device=DEV),
                           torch.empty((n, Hkv, d), dtype=dt, device=DEV)))
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return st
    B, H, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    lens = _lengths(case["lmin"], case["lmax"], B)
    if op == "append":
        if case["path"]:
            # chains of nmax nodes of which cnt were accepted (the root always is)
            rows = torch.full((B,), case["nmax"], dtype=torch.int64, device=DEV)
            cnt = _lengths(max(1, case["nmin"]), case["nmax"], B)
            j = torch.arange(case["nmax"], device=DEV)[None, :]
            st["path"] = i32(torch.where(j < cnt[:, None], j.expand(B, -1), -1)).contiguous()
        else:
            rows = cnt = _lengths(case["nmin"], case["nmax"], B)
            st["path"] = None
        n = int(rows.sum())
        table, n_pages = _table(gen, lens + cnt, page)
        st.update(k=rand(n, H, d), v=rand(n, H, d), cache=_new_cache(gen, n_pages, case), table=table,
                  cache_len=i32(lens), row_off=_offsets(rows), out_off=_offsets(cnt), max_new=int(cnt.max()),
                  rope=_rope_table(int((lens + cnt).max()) + 1, case["rot"]),
                  new_len=torch.empty(B, dtype=torch.int32, device=DEV))
        m = int(cnt.sum())
    elif op == "gather":
        table, n_pages = _table(gen, lens, page)
        st.update(cache=_new_cache(gen, n_pages, case), table=table, out_off=_offsets(lens),
                  max_rows=int(lens.max()))
        m = int(lens.sum())
    else:
        N, Hq = case["nodes"], case["Hq"]
        table, n_pages = _table(gen, lens, page)
        par = _parents(case, gen)
        words = (N + 63) // 64
        st.update(cache=_new_cache(gen, n_pages, case), table=table, cache_len=i32(lens), q=rand(B * N, Hq, d),
                  k_tree=rand(B * N, H, d), v_tree=rand(B * N, H, d),
                  anc=_ancestors(par, words).to(DEV).repeat(B, 1),
                  node_off=(torch.arange(B + 1, device=DEV) * N).to(torch.int32), vis=None,
                  out=torch.empty((B * N, Hq, d), dtype=dt, device=DEV),
                  lse=torch.empty((B * N, Hq), dtype=torch.float32, device=DEV))
        if case["vis"]:
            # sorted anchors in the prefix, one for each branch of 16 nodes
            nb = (N + 15) // 16
            a = torch.sort(torch.rand((B, nb), generator=gen, device=DEV), 1).values
            v = (a * (lens[:, None] + 1)).long().clamp(max=lens[:, None])
            st["vis"] = i32(v.repeat_interleave(16, 1)[:, :N].reshape(-1)).contiguous()
        st["ws"] = None
        m = 0
    if m or op != "attn":
        st["outputs"] = tuple(torch.empty((m, H, d), dtype=dt, device=DEV) for _ in range(2))
    st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return st


# ---------------------------------------------------------------- plain form
def _scale(x):
    """Scale of each row of fp32 ``x`` [.., d]: max|x| / 7 rounded up to bf16, at least 2^-100."""
    a = x.abs().amax(-1)
    a = a / torch.full_like(a, 7.0)          # a true division (a scalar divisor becomes a reciprocal product)
    up = ((a.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)
    return torch.where(torch.isfinite(a), up, torch.full_like(a, math.nan)).clamp(min=SCALE_MIN)


def _unpack(cache, page, d):
    """(K, V) fp32 [pages, Hkv, page, d] of the whole pool."""
    pages, H, _ = cache.shape
    out = []
    for values in (False, True):
        c = cache[:, :, page * d // 2 * values: page * d // 2 * (1 + values)]
        nib = torch.stack([c & 15, c >> 4], -1).view(pages, H, -1, 8)[..., NIB]
        if values:
            n = nib.view(pages, H, page // 16, d, 16).transpose(3, 4).reshape(pages, H, page, d)
        else:
            n = nib.view(pages, H, d // 32, page, 32).transpose(2, 3).reshape(pages, H, page, d)
        o = page * d + 2 * page * values
        s = cache[:, :, o:o + 2 * page].contiguous().view(torch.bfloat16).float()
        out.append((n.float() - 8.0) * s[..., None])
    return out


def _rotate(x, pos, table, inter):
    rot = table.shape[1]
    cs = table[pos.long()][:, None, :]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    y1, y2 = a * c - b * s, b * c + a * s
    y = torch.stack([y1, y2], -1).flatten(-2) if inter else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _row_of(off, total):
    """Request and index within it of each of ``total`` rows."""
    i = torch.arange(total, device=off.device)
    r = torch.searchsorted(off[1:].long(), i, right=True)
    return r, i - off.long()[r]


def _plain_append(st):
    case = st["case"]
    total = st["outputs"][0].shape[0]
    r, j = _row_of(st["out_off"], total)
    src = st["row_off"].long()[r] + (j if st["path"] is None else st["path"].long()[r, j])
    pos = st["cache_len"].long()[r] + j
    k = _rotate(st["k"][src], pos, st["rope"], case["inter"])
    v = st["v"][src].float()
    vals = []
    for x in (k, v):
        s = _scale(x)[..., None]
        vals.append((torch.round(x / s).clamp(-7, 7) * s).to(_dt(case)))
    return vals[0], vals[1], (st["cache_len"] + (st["out_off"][1:] - st["out_off"][:-1])).to(torch.int32)


def _plain_gather(st):
    case = st["case"]
    K, V = _unpack(st["cache"], case["page"], case["d"])
    r, j = _row_of(st["out_off"], st["outputs"][0].shape[0])
    page = st["table"].long()[r, j // case["page"]]
    slot = j % case["page"]
    return K[page, :, slot].to(_dt(case)), V[page, :, slot].to(_dt(case))


def _plain_attn(st):
    case = st["case"]
    B, N, Hq, H, d, P = (case[k] for k in ("B", "nodes", "Hq", "Hkv", "d", "page"))
    g = Hq // H
    lens = st["cache_len"].long()
    K, V = _unpack(st["cache"], P, d)
    cols = st["table"].shape[1]
    pages = st["table"].long().clamp(min=0)
    K = K[pages].permute(0, 2, 1, 3, 4).reshape(B, H, cols * P, d)
    V = V[pages].permute(0, 2, 1, 3, 4).reshape(B, H, cols * P, d)
    kt = st["k_tree"].float().view(B, N, H, d).transpose(1, 2)
    vt = st["v_tree"].float().view(B, N, H, d).transpose(1, 2)
    q = st["q"].float().view(B, N, H, g, d).permute(0, 2, 1, 3, 4).reshape(B, H, N * g, d)
    t = torch.arange(cols * P, device=q.device)
    vis = lens[:, None].expand(B, N) if st["vis"] is None else torch.minimum(st["vis"].long().view(B, N).clamp(min=0),
                                                                             lens[:, None])
    see = t[None, None, :] < vis[:, :, None]                                        # [B, N, L]
    i = torch.arange(N, device=q.device)
    anc = (st["anc"].view(B, N, -1)[:, :, i // 64] >> (i % 64)[None, None, :]) & 1   # [B, N, N]
    see = torch.cat([see, anc.bool()], 2).repeat_interleave(g, 1)[:, None]
    s = torch.cat([q @ K.transpose(2, 3), q @ kt.transpose(2, 3)], 3) * (1.0 / math.sqrt(d))
    s = torch.where(see, s, torch.full((), -math.inf, device=q.device))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    L = cols * P
    o = e[..., :L] @ V + e[..., L:] @ vt
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l))[..., 0]
    back = lambda x: x.reshape(B, H, N, g, -1).permute(0, 2, 1, 3, 4).reshape(B * N, Hq, -1)  # noqa: E731
    return back(o).to(_dt(case)), back(lse[..., None])[..., 0].contiguous()


# ----------------------------------------------------------------------- run
def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        if op == "rope":
            return tuple(_rotate(x, st["pos"], st["rope"], case["inter"]).to(_dt(case)) for x in (st["q"], st["k"]))
        return {"append": _plain_append, "gather": _plain_gather, "attn": _plain_attn}[op](st)
    import speculative_decoding_tree_02_gb300 as tv
    if op == "rope":
        q, k, _ = tv.tv_rope(st["q"], st["k"], st["pos"], st["rope"], interleaved=case["inter"],
                             outputs=st["outputs"], err=st["err"])
        return q, k
    if op == "append":
        new_len, _ = tv.kv4_append(st["k"], st["v"], st["cache"], case["page"], st["table"], st["cache_len"],
                                   st["row_off"], st["max_new"], path=st["path"], rope=st["rope"],
                                   interleaved=case["inter"], new_len=st["new_len"], err=st["err"])
        # the appended rows as the values that the cache now holds for them
        k, v, _ = tv.kv4_gather(st["cache"], case["page"], st["table"], st["out_off"], st["max_new"],
                                start=st["cache_len"], outputs=st["outputs"], err=st["err"])
        return k, v, new_len
    if op == "gather":
        k, v, _ = tv.kv4_gather(st["cache"], case["page"], st["table"], st["out_off"], st["max_rows"],
                                outputs=st["outputs"], err=st["err"])
        return k, v
    if st["ws"] is None:     # a serving loop keeps its workspace
        st["ws"] = tv.tree_verify_attn_kv4_workspace(case["B"], case["nodes"], case["Hq"], case["Hkv"], case["d"],
                                                     st["q"].dtype, st["q"].device)
    out, lse, _ = tv.tree_verify_attn_kv4(st["q"], st["cache"], case["page"], st["table"], st["cache_len"],
                                          st["k_tree"], st["v_tree"], st["node_off"], st["anc"], case["nodes"],
                                          vis_prefix=st["vis"], out=st["out"], lse=st["lse"], ws=st["ws"],
                                          err=st["err"])
    return out, lse


# ---------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass."""
    e = 2 if case["dtype"] == "bf16" else 4
    d, H = case["d"], case["Hkv"]
    if case["op"] == "rope":
        n = case["n"]
        return {"bytes": n * (2 * (case["Hq"] + H) * d * e + 4) + min(n, case["pmax"]) * case["rot"] * 4,
                "flops": 3 * n * (case["Hq"] + H) * case["rot"]}
    B = case["B"]
    ln = sum(_spread(case["lmin"], case["lmax"], B)) / B
    row = H * (d + 4)                       # one token's codes and scales, all KV heads
    if case["op"] == "append":
        n = max(1, sum(_spread(max(1, case["nmin"]) if case["path"] else case["nmin"], case["nmax"], B)))
        # rows in, table rows, cache out; the values read back
        return {"bytes": n * (2 * H * d * e + case["rot"] * 4 + row) + n * 2 * H * d * e, "flops": n * 8 * H * d}
    if case["op"] == "gather":
        n = max(B * ln, 1)
        return {"bytes": n * (row + 2 * H * d * e), "flops": n * 2 * H * d}
    N, Hq = case["nodes"], case["Hq"]
    see = ln / 2 if case["vis"] else ln     # mean visible prefix of a node
    depth = {"chain": (N + 1) / 2, "branches": min(N + 1, 17) / 2, "sweep": 9.5}.get(case["tree"], math.log(N) + 1)
    return {"bytes": B * ln * row + B * N * (2 * Hq * d * e + 2 * H * d * e + Hq * 4),
            "flops": 4 * d * Hq * B * N * (see + depth)}


# --------------------------------------------------------------------- exact
def _codes64(cache, page, d, r_pages, count):
    """K and V [count, Hkv, d] in fp64 of the first ``count`` tokens on ``r_pages``, decoded item by item."""
    H = cache.shape[1]
    t = torch.arange(count, device=cache.device)
    blk = cache[r_pages.long()[t // page]]                                          # [count, H, bytes]
    slot = t % page
    dim = torch.arange(d, device=cache.device)
    nibble = lambda e: e // 2 + 4 * (e % 2)  # noqa: E731
    mk = nibble(dim % 8)
    kb = (dim // 32)[None, :] * page * 16 + slot[:, None] * 16 + (dim % 32 // 8)[None, :] * 4 + (mk // 2)[None, :]
    mv = nibble(slot % 8)
    vb = page * d // 2 + (slot // 16)[:, None] * d * 8 + dim[None, :] * 8 + (slot % 16 // 8 * 4 + mv // 2)[:, None]
    take = lambda b: torch.gather(blk, 2, b[:, None, :].expand(count, H, d)).long()  # noqa: E731
    k = (take(kb) >> (4 * (mk % 2))[None, None, :]) & 15
    v = (take(vb) >> (4 * (mv % 2))[:, None, None]) & 15

    def scale(o):
        b = o + 2 * slot
        lo, hi = (torch.gather(blk, 2, (b + i)[:, None, None].expand(count, H, 1)).int() for i in (0, 1))
        return ((lo << 16) | (hi << 24)).view(torch.float32).double()
    return (k - 8).double() * scale(page * d), (v - 8).double() * scale(page * d + 2 * page)


def _rotate64(x, pos, table, inter):
    half = table.shape[1] // 2
    y = x.double().clone()
    c, s = table[pos.long(), :half].double()[:, None], table[pos.long(), half:].double()[:, None]
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    y[..., a] = x[..., a].double() * c - x[..., b].double() * s
    y[..., b] = x[..., b].double() * c + x[..., a].double() * s
    return y


def _quant64(x):
    a = x.abs().amax(-1, keepdim=True) / 7
    m, e = torch.frexp(a)                       # a = m * 2^e with m in [1/2, 1): bf16 keeps 8 bits of m
    s = torch.ldexp(torch.ceil(m * 256) / 256, e).clamp(min=SCALE_MIN)
    return torch.round(x / s) * s


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(_rotate64(x, st["pos"], st["rope"], case["inter"]) for x in (st["q"], st["k"]))
    off = st["out_off"].tolist() if "out_off" in st else None
    if case["op"] == "append":
        ks, vs = [], []
        for r, (n0, l0) in enumerate(zip(st["row_off"].tolist()[:-1], st["cache_len"].tolist())):
            j = torch.arange(off[r + 1] - off[r], device=DEV)
            src = n0 + (j if st["path"] is None else st["path"][r, :j.numel()].long())
            ks.append(_quant64(_rotate64(st["k"][src], l0 + j, st["rope"], case["inter"])))
            vs.append(_quant64(st["v"][src].double()))
        return torch.cat(ks), torch.cat(vs), None
    lens = st["cache_len"].tolist() if "cache_len" in st else [b - a for a, b in zip(off, off[1:])]
    if case["op"] == "gather":
        parts = [_codes64(st["cache"], case["page"], case["d"], st["table"][r], n) for r, n in enumerate(lens)]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    N, Hq, H, d = case["nodes"], case["Hq"], case["Hkv"], case["d"]
    out = torch.zeros((case["B"] * N, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((case["B"] * N, Hq), -math.inf, dtype=torch.float64, device=DEV)
    bit = torch.arange(N, device=DEV)
    for r, n in enumerate(lens):
        kp, vp = _codes64(st["cache"], case["page"], d, st["table"][r], n)
        rows = slice(r * N, (r + 1) * N)
        k = torch.cat([kp, st["k_tree"][rows].double()])
        v = torch.cat([vp, st["v_tree"][rows].double()])
        seen = torch.full((N,), n, device=DEV) if st["vis"] is None else st["vis"][rows].long().clamp(0, n)
        anc = (st["anc"][rows][:, bit // 64] >> (bit % 64)) & 1
        see = torch.cat([torch.arange(n, device=DEV)[None, :] < seen[:, None], anc.bool()], 1)
        some = see.any(1)
        for h in range(H):
            heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
            s = torch.einsum("nhd,td->nht", st["q"][rows, heads].double(), k[:, h]) / math.sqrt(d)
            s = s.masked_fill(~see[:, None, :], -math.inf)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(some[:, None], z, torch.zeros_like(z))[..., None])
            out[rows, heads] = torch.einsum("nht,td->nhd", p, v[:, h])
            lse[rows, heads] = z
    return out, lse
