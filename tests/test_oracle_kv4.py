"""Pins of the 4-bit cache oracle (no GPU): the quantiser against its
definition, the block layout by round trips, rotation by its group property,
attention against the tree-attention oracle; and the host checks of the
library's calls and of the binding."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import synth
from conftest import ROOT
from oracle import attention as oatt
from oracle import kv4 as ok

LIB = os.path.join(ROOT, "speculative_decoding_tree_02_gb300", "libtreeverify.so")


def rows(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape).astype(np.float32)


def test_quantise_is_within_half_a_step_and_the_scale_is_a_bf16_upper_bound():
    x = rows(0, 200, 64) * np.float32(10.0) ** np.random.default_rng(1).integers(-6, 6, (200, 1)).astype(np.float32)
    n, s = ok.quantise(x)
    assert np.array_equal(s, ok.f32(ok.bf16_bits(s)))
    a = np.abs(x).max(-1).astype(np.float64)
    assert (7.0 * s >= a * (1 - 2.0 ** -23)).all() and (7.0 * s <= a * (1 + 2.0 ** -7) * (1 + 2.0 ** -22)).all()
    assert np.abs(n).max() == 7 and np.abs(n).min() == 0
    err = np.abs(ok.values(n, s).astype(np.float64) - x)
    assert (err <= s[:, None] * 0.5 * (1 + 2.0 ** -20)).all()


def test_quantise_ties_go_to_even_and_edge_rows():
    x = np.array([[7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 6.5]], np.float32)
    n, s = ok.quantise(x)
    assert s[0] == 1.0 and n[0].tolist() == [7, 0, 2, 2, 0, -2, -2, 6]
    n, s = ok.quantise(np.zeros((1, 8), np.float32))
    assert s[0] == ok.SCALE_MIN and not n.any()
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 8), np.float32)
        x[0, 3] = bad
        n, s = ok.quantise(x)
        assert np.isnan(s[0]) and np.isnan(ok.values(n, s)).all()


@pytest.mark.parametrize("P,d", [(16, 64), (32, 128), (64, 64), (128, 128)])
def test_block_round_trip_touches_every_nibble_once(P, d):
    rng = np.random.default_rng(P + d)
    kn, vn = rng.integers(-7, 8, (2, P, d))
    ks, vs = ok.f32(ok.bf16_bits(rng.uniform(0.1, 2, (2, P)).astype(np.float32)))
    block = rng.integers(0, 256, P * (d + 4)).astype(np.uint8)
    for t in rng.permutation(P):
        ok.write_row(block, P, d, t, kn[t], ks[t], vn[t], vs[t])
    for got, want in zip(ok.read_block(block, P, d), (kn, ks, vn, vs)):
        assert np.array_equal(got, want)


def test_the_case_file_packs_the_same_blocks():
    """perf/operators.py states the layout a third time (torch, whole pools at once)."""
    import importlib.util
    import torch
    spec = importlib.util.spec_from_file_location("perf_operators", os.path.join(ROOT, "perf", "operators.py"))
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    P, d = 32, 64
    x = torch.randn((2, 1, P, d), generator=torch.Generator().manual_seed(0))
    (kc, ks), (vc, vs) = (ops._pack(x * (1 + i), P, bool(i)) for i in (0, 1))
    cache = torch.cat([kc, vc, ks.view(torch.uint8).reshape(2, 1, -1), vs.view(torch.uint8).reshape(2, 1, -1)], 2)
    want = np.zeros((2, 1, P * (d + 4)), np.uint8)
    kq, vq = ok.quantise(x.numpy()), ok.quantise((2 * x).numpy())
    for pg in range(2):
        for t in range(P):
            ok.write_row(want[pg, 0], P, d, t, kq[0][pg, 0, t], kq[1][pg, 0, t], vq[0][pg, 0, t], vq[1][pg, 0, t])
    assert np.array_equal(cache.numpy(), want)
    K, V = ops._unpack(cache, P, d)
    assert np.array_equal(K.numpy(), ok.values(*kq)) and np.array_equal(V.numpy(), ok.values(*vq))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_positions(interleaved):
    table = ok.rope_table(64, 32)
    x, y = rows(2, 1, 2, 48), rows(3, 1, 2, 48)

    def dot(p, q):
        a = ok.rotate(x, [p], table, interleaved).astype(np.float64)
        b = ok.rotate(y, [q], table, interleaved).astype(np.float64)
        return (a * b).sum(-1)
    np.testing.assert_allclose(dot(5, 2), dot(40, 37), atol=1e-4)
    r = ok.rotate(x, [11], table, interleaved)
    np.testing.assert_allclose((r ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-5)
    assert np.array_equal(r[..., 32:], x[..., 32:])
    assert np.array_equal(ok.rotate(x, [0], table, interleaved), x)


def test_append_by_path_equals_append_of_the_picked_rows():
    P, H, d = 16, 2, 64
    k, v = rows(4, 12, H, d), rows(5, 12, H, d)
    table = np.array([[2, 0], [1, 3]], np.int32)
    caches = [np.zeros((4, H, P * (d + 4)), np.uint8) for _ in range(2)]
    path = np.array([[0, 2, 5, -1], [1, 3, 4, 5]], np.int32)
    n1 = ok.append(caches[0], P, table, [14, 3], k, v, [0, 6, 12], path)
    pick = np.array([0, 2, 5, 7, 9, 10, 11])
    n2 = ok.append(caches[1], P, table, [14, 3], k[pick], v[pick], [0, 3, 7])
    assert n1.tolist() == n2.tolist() == [17, 7]
    assert np.array_equal(caches[0], caches[1])
    K, V = ok.gather(caches[0], P, table, [14, 3], [3, 4])[0]
    assert np.array_equal(K, ok.values(*ok.quantise(k[[0, 2, 5]]))) and np.array_equal(
        V, ok.values(*ok.quantise(v[[0, 2, 5]])))


def test_attention_equals_the_tree_attention_oracle_on_the_cached_values():
    d = synth.tiny_tree(N=20, P=40)
    n0 = d["parent"].size
    table = np.array([[1, 0, 2]], np.int32)
    cache = np.zeros((3, 1, 16 * (64 + 4)), np.uint8)
    ok.append(cache, 16, table, [0], d["k_pre"], d["v_pre"], [0, 40])
    pre = ok.gather(cache, 16, table, [0], [40])
    see = np.zeros((n0, n0), bool)
    for i in range(n0):
        see[i, i] = True
        if d["parent"][i] >= 0:
            see[i] |= see[d["parent"][i]]
    vis = np.random.default_rng(0).integers(0, 41, n0)
    o, l, _, _ = ok.attention(d["q"], pre, d["k_tree"], d["v_tree"], d["node_off"], see, vis)
    ro, rl = oatt.tree_attention(d["q"], pre[0][0], pre[0][1], np.array([0, 40]), d["k_tree"], d["v_tree"],
                                 d["node_off"], d["parent"], vis)
    np.testing.assert_allclose(o, ro, atol=1e-12)
    np.testing.assert_allclose(l, rl, atol=1e-12)


# --------------------------------------------------------------- host checks
EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -4


@pytest.fixture(scope="module")
def tv():
    if not os.path.exists(LIB):
        subprocess.run([sys.executable, "-m", "speculative_decoding_tree_02_gb300.build"], cwd=ROOT, check=True)
    import speculative_decoding_tree_02_gb300 as m
    m.load_library()
    return m


def rope_call(lib, b, **kw):
    a = dict(q=b, ldq=512, k=b, ldk=128, dt=1, n=4, Hq=4, Hkv=1, d=128, pos=b, table=b, max_pos=8, rot=128, inter=0,
             qo=b, ko=b, err=None) | kw
    return lib.tv_rope(*a.values(), None)


def append_call(lib, b, **kw):
    a = dict(k=b, ldk=256, v=b, ldv=256, dt=1, rows=4, row_off=b, path=None, path_ld=0, B=1, max_new=4, pos=None,
             table=b, max_pos=8, rot=128, inter=0, cache=b, n_pages=2, page=16, bt=b, bt_ld=2,
             clen=b, H=2, d=128, new_len=None, err=None) | kw
    return lib.kv4_append(*a.values(), None)


def gather_call(lib, b, **kw):
    a = dict(cache=b, n_pages=2, page=16, bt=b, bt_ld=2, start=None, out_off=b, B=1, max_rows=4, rows=4, H=2, d=128,
             dt=1, k=b, v=b, err=None) | kw
    return lib.kv4_gather(*a.values(), None)


def attn_call(lib, b, **kw):
    a = dict(q=b, ldq=512, cache=b, n_pages=2, page=16, bt=b, bt_ld=2, clen=b, k=b, ldk=256, v=b, ldv=256, node_off=b,
             node_cnt=None, anc=b, words=1, vis=None, B=1, nodes=4, total=4, Hq=4, Hkv=2, d=128, dt=1,
             scale=0.1, out=b, lse=None, ws=b, ws_bytes=1 << 40, err=None) | kw
    return lib.tree_verify_attn_kv4(*a.values(), None)


REFUSALS = [
    (rope_call, EINVAL, dict(dt=2)), (rope_call, EINVAL, dict(n=-1)), (rope_call, EINVAL, dict(ldq=511)),
    (rope_call, EINVAL, dict(ldq=516)), (rope_call, EINVAL, dict(ldk=64)), (rope_call, EINVAL, dict(rot=144)),
    (rope_call, EINVAL, dict(table=None)), (rope_call, EINVAL, dict(ko=None)), (rope_call, EINVAL, dict(pos=None)),
    (rope_call, EUNSUPPORTED, dict(rot=24)), (rope_call, EUNSUPPORTED, dict(d=72, rot=16)),
    (rope_call, EUNSUPPORTED, dict(d=1024, ldq=8192, ldk=8192)), (rope_call, EINVAL, dict(q="odd")),
    (rope_call, 0, dict(n=0)),
    (append_call, EINVAL, dict(dt=7)), (append_call, EINVAL, dict(ldk=128)), (append_call, EINVAL, dict(ldv=260)),
    (append_call, EINVAL, dict(max_new=-1)), (append_call, EINVAL, dict(path="b", path_ld=0)),
    (append_call, EINVAL, dict(table=None)), (append_call, EINVAL, dict(new_len="clen")),
    (append_call, EINVAL, dict(cache=None)), (append_call, EINVAL, dict(cache="odd")),
    (append_call, EINVAL, dict(bt_ld=1 << 28)), (append_call, EUNSUPPORTED, dict(page=24)),
    (append_call, EUNSUPPORTED, dict(page=256)), (append_call, EUNSUPPORTED, dict(d=96, rot=0)),
    (append_call, EUNSUPPORTED, dict(B=65536)), (append_call, 0, dict(B=0)),
    (gather_call, EINVAL, dict(dt=9)), (gather_call, EINVAL, dict(rows=-1)), (gather_call, EINVAL, dict(out_off=None)),
    (gather_call, EINVAL, dict(v=None)), (gather_call, EUNSUPPORTED, dict(page=8)),
    (gather_call, EUNSUPPORTED, dict(d=32)), (gather_call, 0, dict(rows=0)), (gather_call, 0, dict(max_rows=0)),
    (attn_call, EINVAL, dict(Hq=5)), (attn_call, EINVAL, dict(scale=0.0)), (attn_call, EINVAL, dict(scale=float("nan"))),
    (attn_call, EINVAL, dict(scale=float("inf"))), (attn_call, EINVAL, dict(words=0)),
    (attn_call, EINVAL, dict(nodes=65)), (attn_call, EINVAL, dict(anc=None)), (attn_call, EINVAL, dict(ldq=256)),
    (attn_call, EINVAL, dict(ldk=255)), (attn_call, EINVAL, dict(ldk=1 << 31)), (attn_call, EINVAL, dict(ldv=1 << 40)),
    (attn_call, EINVAL, dict(dt=2)), (attn_call, EUNSUPPORTED, dict(bt_ld=1 << 28)),
    (attn_call, EUNSUPPORTED, dict(B=40000)), (attn_call, EINVAL, dict(q="odd")), (attn_call, EINVAL, dict(bt=None)),
    (attn_call, EUNSUPPORTED, dict(page=48)), (attn_call, EUNSUPPORTED, dict(d=96)),
    (attn_call, EUNSUPPORTED, dict(nodes=1025, words=17)), (attn_call, EUNSUPPORTED, dict(Hq=130, Hkv=2, ldq=1 << 16)),
    (attn_call, EWORKSPACE, dict(ws=None)), (attn_call, EWORKSPACE, dict(ws_bytes=16)),
    (attn_call, EWORKSPACE, dict(ws="odd")), (attn_call, 0, dict(B=0)), (attn_call, 0, dict(total=0)),
]


@pytest.mark.parametrize("call,want,kw", REFUSALS)
def test_calls_are_refused_before_any_launch(tv, call, want, kw):
    """Placeholder addresses stand in for the arrays; every call here returns before a launch."""
    b = 1 << 12
    sub = {"odd": b + 2, "b": b, "clen": b}
    kw = {k: sub[v] if isinstance(v, str) else v for k, v in kw.items()}
    assert call(tv.load_library(), b, **kw) == want


@pytest.mark.parametrize("kw", [dict(max_new=0), dict(rows=0), dict(rows=0, max_new=0), dict()])
def test_append_wants_its_block_table_whatever_the_rows(tv, kw):
    assert append_call(tv.load_library(), 1 << 12, **kw, bt=None) == EINVAL


def test_cache_size_counts_blocks_and_refuses_other_shapes(tv):
    lib = tv.load_library()
    assert lib.kv4_cache_size(3, 64, 8, 128) == 3 * 8 * 64 * 132
    for bad in ((3, 60, 8, 128), (3, 64, 8, 96), (0, 64, 8, 128), (3, 64, 0, 128)):
        assert lib.kv4_cache_size(*bad) == 0


@pytest.mark.parametrize("kw", [
    dict(bt_ld=(1 << 27) - 1), dict(bt_ld=(1 << 24) - 1, page=128, dt=0), dict(bt_ld=(1 << 27) - 4095),   # tokens
    dict(bt_ld=1 << 26, Hq=128, Hkv=128, ldq=1 << 14, ldk=1 << 14, ldv=1 << 14),              # tiles of a request
    dict(bt_ld=1 << 22, Hq=128, Hkv=128, ldq=1 << 14, ldk=1 << 14, ldv=1 << 14, B=400, nodes=1024, words=16)])   # in all
def test_attention_refuses_what_its_counters_cannot_hold(tv, kw):
    """A prefix of 2^31 - 16 tokens: the tile after the last begins past 2^31."""
    assert attn_call(tv.load_library(), 1 << 12, **kw) == EUNSUPPORTED


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (7, 1), (32, 8), (64, 2), (64, 1), (9, 9), (40, 2)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_covers_smaller_calls(tv, Hq, Hkv, d, dtype):
    """A server keeps one workspace for its most requests and largest trees."""
    size = tv.load_library().tree_verify_attn_kv4_workspace_size
    last = 0
    for nodes in (1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 33, 64, 65, 113, 128, 129, 500, 1024):
        by_b = [size(B, nodes, Hq, Hkv, d, dtype) for B in (1, 2, 3, 16, 17, 64, 100, 1000)]
        assert by_b == sorted(by_b) and by_b[0] > 0
        assert size(64, nodes, Hq, Hkv, d, dtype) >= last
        last = size(64, nodes, Hq, Hkv, d, dtype)


def test_binding_refuses_wrong_tensors(tv):
    import torch
    cache = torch.zeros((2, 1, 16 * 68), dtype=torch.uint8)
    row = torch.zeros((4, 1, 64))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok_args = dict(k=row, v=row, cache=cache, page_size=16, block_table=i32(1, 2), cache_len=i32(1), row_off=i32(2),
                   max_new=4, err=i32(1))
    for bad, exc in ((dict(v=row.double()), TypeError), (dict(v=row[:, :, :32]), ValueError),
                     (dict(row_off=i32(3)), ValueError), (dict(cache_len=torch.zeros(1)), TypeError),
                     (dict(cache=cache[:, :, :-4]), ValueError), (dict(page_size=15), ValueError),
                     (dict(k=torch.zeros((4, 64, 1)).transpose(1, 2)[..., ::1].half()), TypeError),
                     (dict(path=i32(2, 4)), ValueError), (dict(block_table=i32(2)), ValueError),
                     ({}, ValueError)):          # the last: host tensors
        with pytest.raises(exc):
            tv.kv4_append(**{**ok_args, **bad})
    with pytest.raises(ValueError):
        tv.kv4_new_cache(4, 24, 8, 128, device="cpu")
    assert tv.kv4_new_cache(4, 32, 2, 64, device="cpu").shape == (4, 2, 32 * 68)
    with pytest.raises(ValueError):              # heads of a row not packed
        tv.tv_rope(torch.zeros((3, 4, 96))[:, :, :64], None, i32(3), torch.zeros((8, 64)), err=i32(1))
    with pytest.raises(ValueError):
        tv.kv4_gather(cache, 16, i32(1, 2), i32(2), 4)
    q = torch.zeros((4, 2, 64))
    with pytest.raises(ValueError):              # the cache holds heads of another size
        tv.tree_verify_attn_kv4(torch.zeros((4, 2, 128)), cache, 16, i32(1, 2), i32(1), row, row, i32(2),
                                torch.zeros((4, 1), dtype=torch.int64), 4)
    with pytest.raises(ValueError):              # host tensors
        tv.tree_verify_attn_kv4(q, cache, 16, i32(1, 2), i32(1), row, row, i32(2),
                                torch.zeros((4, 1), dtype=torch.int64), 4, err=i32(1), ws=torch.zeros(1 << 20,
                                                                                                 dtype=torch.uint8))


def test_no_warp_of_a_team_leaves_its_loop_at_a_wait():
    """The barriers of the tcgen05 kernel count all threads of a team, so a wait that expires must not take its warp
    out of the loop: it is noted, and the team's vote before PV sends all of it out.  (Read from the source: a wait
    that expires is not provoked on a GPU.)"""
    import re
    src = open(os.path.join(os.path.dirname(LIB), "csrc", "attn_kv4_tc.cu")).read()
    body = src[src.index("attn_kernel(const __grid_constant__"):]
    waits = re.findall(r"^.*wait\w*\(.*abort_flag.*$", body, re.M)
    assert len(waits) == 4 and all(re.match(r"\s*(if \(it > 0\) )?team_wait\([^;]*\);(\s*//.*)?$", w) for w in waits)
    assert "void team_wait(" in src                           # nothing to branch on
    assert "slow = any_of<256>(tbar, *abort_flag != 0 ||" in body and "if (__builtin_expect(aborted, 0)) break;" in body
