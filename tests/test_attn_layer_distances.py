"""Host-side checks of the distances between an attention call's rows: which views of
shared rows are taken and which are refused, before any device call (no device
needed).  Helpers stand in test_attn_layer_refusals.py."""
import ctypes as C

import pytest

import attention_decode_megakernel_b200 as mk
from test_attn_layer_refusals import (L, P, _cache, _packed_call, _paged_call,  # noqa: F401
                                      _rope_call)


def test_shared_rows_that_no_tensor_map_walks(L):
    """A distance of 0 between several tokens or heads, where the rows go through
    tensor maps: queries of many rows, tokens of packed keys and values."""
    for bad in (dict(q_ts=0), dict(q_hs=0), dict(q_ts=0, q_hs=0), dict(k_ts=0), dict(v_ts=0),
                dict(k_ts=0, k_hs=0), dict(hq=2, q_hs=0), dict(hk=1, hq=2, q_hs=0)):
        assert _packed_call(L, **bad) == mk.MK_ERR_UNSUPPORTED, bad
    many = dict(rows=18, batch=2)  # units of 2 x 9 rows
    for bad in (dict(q_ts=0), dict(q_hs=0), dict(q_ts=0, q_hs=0)):
        assert _paged_call(L, _cache(), **bad, **many) == mk.MK_ERR_UNSUPPORTED, bad
    # nothing to do is nothing to refuse
    assert _packed_call(L, q_ts=0, k_ts=0, rows=0) == mk.MK_OK
    assert _paged_call(L, _cache(), q_hs=0, rows=0) == mk.MK_OK


def test_outputs_whose_rows_overlap(L):
    """What a call writes has a place of its own for every token and head: a distance
    below head_dim (0: an expanded tensor) is refused."""
    for bad in (dict(o_ts=0), dict(o_hs=0), dict(o_ts=56), dict(o_hs=32)):
        assert _paged_call(L, _cache(), **bad) == mk.MK_ERR_ARG, bad
        assert _packed_call(L, **bad) == mk.MK_ERR_ARG, bad
    for bad in (dict(qo_ts=0), dict(qo_hs=0), dict(ko_ts=0), dict(ko_hs=0), dict(qo_hs=48),
                dict(ko_ts=56), dict(q_hs=0, qo_hs=0)):
        assert _rope_call(L, **bad) == mk.MK_ERR_ARG, bad
    cache = _cache()
    for k_ts, k_hs, v_ts, v_hs in ((0, 64, 128, 64), (128, 0, 128, 64), (128, 64, 0, 64),
                                   (128, 64, 128, 0), (128, 56, 128, 64), (128, 64, 32, 64)):
        assert L.mk_kv_read(C.addressof(cache), P, 3, P, k_ts, k_hs, P, v_ts, v_hs, 0,
                            None) == mk.MK_ERR_ARG


def test_a_distance_that_nothing_walks(L):
    """One token or one head: its distance may be anything, 0 too.  (Empty calls stand
    in for launches.)"""
    assert _paged_call(L, _cache(), o_ts=0, q_ts=0, rows=0) == mk.MK_OK
    assert _rope_call(L, qo_ts=0, ko_ts=0, tokens=0) == mk.MK_OK


def test_more_rows_than_the_entries_count(L, monkeypatch):
    """Expanded tensors may have more rows than the C entries' 32 bits count: refused, not
    cut to what is left of the number."""
    torch = pytest.importorskip("torch")
    from test_attn_layer_workspace import _on_device
    made = []
    for call in (mk._norm_rope_call, mk._kv_write_call, mk._kv_read_call, mk._paged_call,
                 mk._packed_call):
        monkeypatch.setattr(call, "quick", lambda *a: False)
        monkeypatch.setattr(call, "slow", lambda *a: made.append(a))
    i32 = dict(dtype=torch.int32)
    cache = mk.KvCache(_on_device(2, 2, 16, 64), _on_device(2, 2, 16, 64))
    ws, cu = _on_device(4096, dtype=torch.uint8), _on_device(2, **i32)
    monkeypatch.setattr(mk, "_vector", lambda t, *a: t.data_ptr())
    for n in (2 ** 31, 2 ** 32 + 3):
        q, k = (_on_device(1, h, 64).expand(n, -1, -1) for h in (4, 2))
        wide = _on_device(3, 1, 64).expand(-1, n, -1)
        pos, slots = _on_device(1, **i32).expand(n), _on_device(1, dtype=torch.int64).expand(n)
        table = _on_device(1, 1, **i32).expand(1, n)
        few, few_k = _on_device(3, 4, 64), _on_device(3, 2, 64)
        for bad in (lambda: mk.qk_norm_rope(mk.Rope(64, 1e4), q, k, pos),
                    lambda: mk.qk_norm_rope(mk.Rope(64, 1e4), wide, None, pos[:3]),
                    lambda: mk.kv_write(cache, k, k, slots),
                    lambda: mk.kv_read(cache, slots, k, k),
                    lambda: mk.attn_paged(q, cache, table[:, :2], cu[:1], cu, q, workspace=ws),
                    lambda: mk.attn_paged(few, cache, table, cu[:1], cu, few, workspace=ws),
                    lambda: mk.attn_paged(few, cache, table[0, :, None], cu[:1], cu, few,
                                          workspace=ws),
                    lambda: mk.attn_packed(q, k, k, cu, q, workspace=ws),
                    lambda: mk.attn_packed(few, few_k, few_k,
                                           _on_device(1, **i32).expand(n + 1), few, workspace=ws)):
            with pytest.raises(ValueError):
                bad()
    assert not made


def test_more_sequences_than_the_kernels_count(L):
    for batch in (2 ** 30 + 1, 2 ** 31 - 1):
        assert _paged_call(L, _cache(), batch=batch) == mk.MK_ERR_UNSUPPORTED
        assert _packed_call(L, batch=batch) == mk.MK_ERR_UNSUPPORTED
