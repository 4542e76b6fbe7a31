"""Host-side checks of the distances between an attention call's rows: which views of
shared rows are taken and which are refused, before any device call (no device
needed).  Helpers stand in test_attn_layer_refusals.py."""
import ctypes as C

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
