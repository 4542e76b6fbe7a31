"""Host-side checks of the distances between an attention call's rows: which views of
shared rows are taken and which are refused, before any device call (no device
needed).  Helpers stand in test_attn_layer_refusals.py."""
import pytest

import attention_decode_megakernel_b200 as mk
from test_attn_layer_refusals import L, _cache, _packed_call, _paged_call  # noqa: F401


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
