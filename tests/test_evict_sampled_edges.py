"""CPU checks of what the entry points of eviction and sampled verification answer before any launch, at the edges."""
import pytest

from test_oracle_evict_sampled import COMPACT, MASS, SAMPLED, SELECT, call, lib  # noqa: F401

NOTHING = {k: None for k in ("q", "lse", "cache", "table", "cache_len", "row_off", "old", "s_in", "s_out")}


@pytest.mark.parametrize("fn,base,change", [
    ("kv4_attn_mass", MASS, dict(B=0, rows=0, in_ld=0, **NOTHING)),               # no scores before: two absent arrays
    ("kv4_attn_mass", MASS, dict(B=0, rows=0, in_ld=80, out_ld=64, **NOTHING)),   # empty scores of two widths
    ("kv4_attn_mass", MASS, dict(max_len=0, in_ld=0, s_in=None, s_out=None)),
    ("kv4_evict_select", SELECT, dict(B=0, score=None, cache_len=None, budget=None, idx=None, out=None, new_len=None)),
    ("kv4_compact", COMPACT, dict(B=0, cache=None, table=None, cache_len=None, idx=None, new_len=None)),
    ("accept_sampled", SAMPLED, dict(B=0, rows=0, parent=None, tok=None, p=None, q=None, ldq=0, node_off=None, u=None, race=None,
                                     acc=None, best=None, path=None, bonus=None, ws=None, ws_bytes=0)),
])
def test_an_empty_batch_is_no_error(lib, fn, base, change):  # noqa: F811
    assert call(lib, fn, base, **change) == 0


def test_one_array_of_two_widths_is_refused(lib):  # noqa: F811
    assert call(lib, "kv4_attn_mass", MASS, in_ld=80, out_ld=64) == -1
    assert call(lib, "kv4_evict_select", SELECT, out=SELECT["score"], ld=64, out_ld=80) == -1


def test_choice_without_scores_of_no_tokens(lib):  # noqa: F811
    """No token, no scores and none wanted: nothing to refuse (without a device the launch is what fails)."""
    assert call(lib, "kv4_evict_select", SELECT, max_len=0, score=None, ld=0, out=None, out_ld=32) != -1


def test_binding_refuses_tables_without_columns(lib):  # noqa: F811
    """An empty tensor has no address, and none means something else: all rows, in place, no scores."""
    import torch

    import speculative_decoding_tree_02_gb300 as tv
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    cache, q = torch.zeros(2, 1, 16 * 68, dtype=torch.uint8), torch.zeros(3, 2, 64)
    score = torch.zeros(1, 1, 32)
    mass = (q, torch.zeros(3, 2), cache, 16, z(1, 2), z(1), z(2), 3)
    with pytest.raises(ValueError, match="path has no columns"):
        tv.kv4_attn_mass(*mass, score=score, path=z(1, 0))
    with pytest.raises(ValueError, match="path has no columns"):
        tv.kv4_append(q[:, :1], q[:, :1], cache, 16, z(1, 2), z(1), z(2), 3, path=z(1, 0))
    with pytest.raises(ValueError, match="dst_table has no columns"):
        tv.kv4_compact(cache, 16, z(1, 2), z(1), z(1, 1, 4), z(1), 4, dst_table=z(1, 0))
    with pytest.raises(ValueError, match="score has no columns"):
        tv.kv4_attn_mass(*mass, score=score[:, :, :0], max_len=8, score_out=score)
    with pytest.raises(ValueError, match="score_out has no columns"):
        tv.kv4_evict_select(score, z(1), z(1), 32, max_keep=4, score_out=score[:, :, :0])
    with pytest.raises(ValueError, match="takes device tensors"):                       # (the calls themselves are in order)
        tv.kv4_attn_mass(*mass, score=score, path=z(1, 2))
    with pytest.raises(ValueError, match="takes device tensors"):
        tv.kv4_compact(cache, 16, z(1, 2), z(1), z(1, 1, 4), z(1), 4, dst_table=z(1, 1))
    with pytest.raises(ValueError, match="takes device tensors"):
        tv.kv4_evict_select(score, z(1), z(1), 32, max_keep=4, score_out=score)


@pytest.mark.parametrize("change", [dict(table=None, table_ld=0), dict(cache=None, n_pages=0)])
def test_move_without_pages_or_columns(lib, change):  # noqa: F811
    """A table of no columns, a cache of no pages: nothing to refuse (without a device the launch is what fails)."""
    assert call(lib, "kv4_compact", COMPACT, **change) != -1
