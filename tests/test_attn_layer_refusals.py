"""Host-side behaviour of the attention layer's operators: frequencies of
mk_rope_init against the formulas, and every refusal of the C entries, which
come before any device call (no device needed)."""
import ctypes as C
import math

import pytest

import attention_decode_megakernel_b200 as mk
from attention_decode_megakernel_b200 import build
import attention_ref as ref


@pytest.fixture(scope="module")
def L():
    build.build()
    return mk.lib()


@pytest.mark.parametrize("rot,theta", [(16, 1e4), (64, 1e7), (128, 5e5), (256, 1e7)])
@pytest.mark.parametrize("scaling,given", [
    ("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=2.5)),
    ("yarn", dict(factor=4.0, original_ctx=32768, low=1.0, high=32.0)),
    ("yarn", dict(factor=40.0, original_ctx=64, low=1.0, high=32.0)),
    ("banded", dict(factor=8.0, original_ctx=8192, low=1.0, high=4.0)),
])
def test_rope_frequencies(L, rot, theta, scaling, given):
    r = mk.Rope(rot, theta, interleaved=True, scaling=scaling, **given)
    turns, length = ref.rope_turns(rot, theta, scaling, **given)
    assert r.c.rot_dim == rot and r.c.interleaved == 1
    assert abs(r.c.magnitude - length) <= 2.0 ** -24 * length
    for i in range(128):
        want = turns[i] if i < rot // 2 else 0.0
        # a power, a division and a product or two in 64 bits; the exponent of the
        # power is up to ln(1e9) = 21, which multiplies its own rounding; cut to 2^-64
        assert abs(r.c.turns[i] * 2.0 ** -64 - want) <= 64 * 2.0 ** -53 * abs(want) + 2.0 ** -64


def test_rope_ends_of_the_scalings(L):
    """The fastest pair keeps its frequency, the slowest is divided by the factor."""
    plain = mk.Rope(64, 1e7).c
    for scaling in ("yarn", "banded"):
        r = mk.Rope(64, 1e7, scaling=scaling, factor=4.0, original_ctx=8192, low=1.0, high=4.0).c
        assert r.turns[0] == plain.turns[0]
        assert abs(r.turns[31] - plain.turns[31] / 4) <= 1e-14 * plain.turns[31] + 1
    assert mk.Rope(64, 1e7, scaling="yarn", factor=1.0, original_ctx=8192).c.magnitude == 1.0


def test_rope_refusals(L):
    def init(rot=64, theta=1e4, scaling=0, factor=1.0, ctx=1.0, low=1.0, high=2.0, r=mk.mk_rope()):
        return L.mk_rope_init(C.byref(r) if r is not None else None, rot, 0, theta, scaling, factor,
                              ctx, low, high)
    assert init() == mk.MK_OK
    assert init(r=None) == mk.MK_ERR_ARG
    for rot, rc in ((0, mk.MK_ERR_ARG), (-16, mk.MK_ERR_ARG), (8, mk.MK_ERR_UNSUPPORTED),
                    (24, mk.MK_ERR_UNSUPPORTED), (272, mk.MK_ERR_UNSUPPORTED)):
        assert init(rot=rot) == rc, rot
    for theta in (1.0, 0.0, -5.0, math.nan, math.inf):
        assert init(theta=theta) == mk.MK_ERR_ARG, theta
    for scaling in (-1, 5):
        assert init(scaling=scaling) == mk.MK_ERR_ARG
    for factor in (0.5, 0.0, math.nan, math.inf):
        for scaling in (1, 2, 3, 4):
            assert init(scaling=scaling, factor=factor) == mk.MK_ERR_ARG
    for scaling in (3, 4):
        for bad in (dict(ctx=0.0), dict(ctx=math.nan), dict(low=0.0), dict(low=2.0),
                    dict(high=math.inf)):
            assert init(scaling=scaling, factor=2.0, **bad) == mk.MK_ERR_ARG, bad
        assert init(scaling=scaling, factor=2.0, ctx=64.0) == mk.MK_OK
    with pytest.raises(ValueError):
        mk.Rope(64, 1e4, scaling="other")
    with pytest.raises(mk.MkError):
        mk.Rope(20, 1e4)


# Stand-ins for device addresses: never read, since every call below is refused
# (or empty) before a launch.
P = 1 << 20


def _rope_call(L, **k):
    a = dict(rope=mk.Rope(64, 1e4).c, q=P, q_ts=512, q_hs=64, k=P, k_ts=512, k_hs=64, qg=P, kg=P,
             pos=P, qo=P, qo_ts=512, qo_hs=64, ko=P, ko_ts=512, ko_hs=64, tokens=4, hq=4, hk=2,
             hd=64, eps=1e-6, dtype=0)
    a.update(k)
    return L.mk_qk_norm_rope(
        C.addressof(a["rope"]) if a["rope"] is not None else None, a["q"], a["q_ts"], a["q_hs"],
        a["k"], a["k_ts"], a["k_hs"], a["qg"], a["kg"], a["pos"], a["qo"], a["qo_ts"], a["qo_hs"],
        a["ko"], a["ko_ts"], a["ko_hs"], a["tokens"], a["hq"], a["hk"], a["hd"], a["eps"],
        a["dtype"], None)


def test_norm_rope_refusals(L):
    assert _rope_call(L, tokens=0) == mk.MK_OK
    assert _rope_call(L, tokens=0, q=None, pos=None, qo=None) == mk.MK_OK
    for bad in (dict(rope=None), dict(rope=mk.mk_rope()), dict(rope=mk.Rope(128, 1e4).c),
                dict(q=None), dict(q=P + 8), dict(k=None), dict(k=P + 2), dict(qo=None),
                dict(ko=None), dict(pos=None), dict(pos=P + 2), dict(qg=P + 2), dict(kg=P + 8),
                dict(q_ts=511), dict(q_hs=60), dict(k_ts=-512), dict(qo_ts=4), dict(ko_hs=1),
                dict(tokens=-1), dict(hq=0), dict(hk=-1), dict(eps=-1.0), dict(eps=math.nan),
                dict(dtype=3), dict(dtype=-1), dict(dtype=4)):
        assert _rope_call(L, **bad) == mk.MK_ERR_ARG, bad
    for hd in (0, 32, 96, 512):
        assert _rope_call(L, hd=hd) == mk.MK_ERR_UNSUPPORTED, hd
    assert _rope_call(L, tokens=0, hk=0, k=None, ko=None) == mk.MK_OK


def _cache(**k):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, page_stride=16 * 64 * 2, head_stride=16 * 64,
             pos_stride=64, n_pages=8, page_size=16, kv_heads=2, head_dim=64, dtype=3)
    a.update(k)
    return mk.mk_kv_cache(*(a[n] for n, _ in mk.mk_kv_cache._fields_))


BAD_CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=P + 8), 1), (dict(v=P + 4), 1),
    (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(k_scale=P + 2), 1),
    (dict(k_scale=P + 4), 1), (dict(v_scale=P + 8), 1),
    (dict(page_stride=-2048), 1), (dict(page_stride=2047), 1), (dict(head_stride=1000), 1),
    (dict(pos_stride=72), 1), (dict(pos_stride=32), 1), (dict(head_stride=0), 1),
    (dict(page_stride=0), 1), (dict(n_pages=0), 1), (dict(kv_heads=0), 1), (dict(page_size=0), 1),
    (dict(dtype=2), 1), (dict(dtype=4), 1), (dict(dtype=-1), 1),
    (dict(page_size=8), 7), (dict(page_size=48), 7), (dict(page_size=512), 7),
    (dict(head_dim=96), 7), (dict(head_dim=0), 7),
]


def _write_call(L, cache, **k):
    a = dict(k=P, k_ts=128, k_hs=64, v=P, v_ts=128, v_hs=64, slots=P, tokens=3, dtype=0)
    a.update(k)
    c = C.addressof(cache) if cache is not None else None
    rows = (a["k"], a["k_ts"], a["k_hs"], a["v"], a["v_ts"], a["v_hs"])
    w = L.mk_kv_write(c, *rows, a["slots"], a["tokens"], a["dtype"], None)
    r = L.mk_kv_read(c, a["slots"], a["tokens"], *rows, a["dtype"], None)
    assert w == r
    return w


def test_kv_refusals(L):
    assert _write_call(L, _cache(), tokens=0) == mk.MK_OK
    assert _write_call(L, _cache(), tokens=0, k=None, v=None, slots=None) == mk.MK_OK
    assert _write_call(L, None) == mk.MK_ERR_ARG
    for bad, rc in BAD_CACHES:
        assert _write_call(L, _cache(**bad)) == rc, bad
    for bad in (dict(k=None), dict(v=None), dict(k=P + 8), dict(slots=None), dict(slots=P + 4),
                dict(tokens=-1), dict(k_ts=127), dict(v_hs=4), dict(v_ts=-128), dict(dtype=3),
                dict(dtype=9)):
        assert _write_call(L, _cache(), **bad) == mk.MK_ERR_ARG, bad


def _paged_call(L, cache, **k):
    a = dict(q=P, q_ts=256, q_hs=64, table=P, stride=4, lens=P, cu=P, out=P, o_ts=256, o_hs=64,
             lse=None, rows=3, batch=2, hq=4, scale=0.125, dtype=0, ws=P,
             ws_bytes=L.mk_attn_ws_bytes(64))
    a.update(k)
    return L.mk_attn_paged(C.addressof(cache) if cache is not None else None, a["q"], a["q_ts"],
                           a["q_hs"], a["table"], a["stride"], a["lens"], a["cu"], a["out"],
                           a["o_ts"], a["o_hs"], a["lse"], a["rows"], a["batch"], a["hq"],
                           a["scale"], a["dtype"], a["ws"], a["ws_bytes"], None)


def _packed_call(L, **k):
    a = dict(q=P, q_ts=256, q_hs=64, k=P, k_ts=128, k_hs=64, v=P, v_ts=128, v_hs=64, cu=P, out=P,
             o_ts=256, o_hs=64, lse=None, rows=3, batch=2, hq=4, hk=2, hd=64, scale=0.125, dtype=0,
             ws=P, ws_bytes=L.mk_attn_ws_bytes(64))
    a.update(k)
    return L.mk_attn_packed(a["q"], a["q_ts"], a["q_hs"], a["k"], a["k_ts"], a["k_hs"], a["v"],
                            a["v_ts"], a["v_hs"], a["cu"], a["out"], a["o_ts"], a["o_hs"],
                            a["lse"], a["rows"], a["batch"], a["hq"], a["hk"], a["hd"],
                            a["scale"], a["dtype"], a["ws"], a["ws_bytes"], None)


BAD_ATTN = [dict(q=None), dict(q=P + 8), dict(q_ts=255), dict(q_hs=-64), dict(out=None),
            dict(out=P + 2), dict(o_ts=4), dict(cu=None), dict(cu=P + 2), dict(lse=P + 2),
            dict(rows=-1), dict(batch=-1), dict(hq=0), dict(hq=3), dict(scale=0.0),
            dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(dtype=2),
            dict(dtype=3), dict(ws=None), dict(ws=P + 128), dict(ws_bytes=1000)]


def test_attn_refusals(L):
    for hd in (64, 128, 256):
        assert L.mk_attn_ws_bytes(hd) > 0
    for hd in (0, 32, 80, 512):
        assert L.mk_attn_ws_bytes(hd) == 0
    assert _paged_call(L, _cache(), rows=0) == mk.MK_OK
    assert _paged_call(L, _cache(), batch=0) == mk.MK_OK
    assert _packed_call(L, rows=0) == mk.MK_OK
    assert _packed_call(L, batch=0) == mk.MK_OK
    assert _paged_call(L, None) == mk.MK_ERR_ARG
    for bad, rc in BAD_CACHES:
        assert _paged_call(L, _cache(**bad)) == rc, bad
    for bad in BAD_ATTN:
        assert _paged_call(L, _cache(), **bad) == mk.MK_ERR_ARG, bad
        assert _packed_call(L, **bad) == mk.MK_ERR_ARG, bad
    for bad in (dict(table=None), dict(table=P + 2), dict(stride=0), dict(stride=-1),
                dict(lens=None), dict(lens=P + 1)):
        assert _paged_call(L, _cache(), **bad) == mk.MK_ERR_ARG, bad
    # a 16-bit cache must have the rows' type
    assert _paged_call(L, _cache(dtype=1)) == mk.MK_ERR_ARG
    for bad in (dict(k=None), dict(v=P + 4), dict(k_ts=4), dict(v_hs=-64), dict(hk=0)):
        assert _packed_call(L, **bad) == mk.MK_ERR_ARG, bad
    for hd in (0, 96, 512):
        assert _packed_call(L, hd=hd) == mk.MK_ERR_UNSUPPORTED, hd


def test_binding_refusals():
    """Shapes, types and devices that the binding can see are ValueErrors."""
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    q, k = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf)
    pos = torch.zeros(3, dtype=torch.int32)
    rope = mk.Rope(64, 1e4)
    for bad in (lambda: mk.qk_norm_rope(rope, q, k, pos),              # not on a CUDA device
                lambda: mk.qk_norm_rope(rope, q, k, pos.long()),
                lambda: mk.qk_norm_rope(rope, q, k.float(), pos),
                lambda: mk.qk_norm_rope(rope, q.transpose(1, 2), k, pos),
                lambda: mk.qk_norm_rope(rope, q, k[:2], pos),
                lambda: mk.qk_norm_rope(rope, q, k, pos, q_gain=torch.ones(64)),
                lambda: mk.qk_norm_rope(rope, q.double(), None, pos),
                lambda: mk.KvCache(k, k),
                lambda: mk.KvCache(torch.zeros(2, 2, 16, 64, dtype=bf),
                                   torch.zeros(2, 2, 16, 64, dtype=bf), torch.ones(2, 2, 16),
                                   torch.ones(2, 2, 16)),
                lambda: mk.KvCache(torch.zeros(2, 2, 16, 64, dtype=torch.float8_e4m3fn),
                                   torch.zeros(2, 2, 16, 64, dtype=torch.float8_e4m3fn))):
        with pytest.raises(ValueError):
            bad()
    cache = mk.KvCache(torch.zeros(2, 2, 16, 64, dtype=bf), torch.zeros(2, 2, 16, 64, dtype=bf))
    slots, out = torch.zeros(3, dtype=torch.int64), torch.zeros_like(q)
    lens, cu = torch.ones(1, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    table, ws = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8)
    for bad in (lambda: mk.kv_write(cache, k, k, slots),
                lambda: mk.kv_write(cache, k, k, slots.int()),
                lambda: mk.kv_write(cache, q, q, slots),
                lambda: mk.kv_read(cache, slots[:2], k, k),
                lambda: mk.attn_paged(q, cache, table, lens, cu, out, workspace=ws),
                lambda: mk.attn_paged(q, cache, table.long(), lens, cu, out, workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu[:1], out, workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu, out[:2], workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu, out.float(), workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu, out, lse=torch.zeros(3, 2),
                                      workspace=ws),
                lambda: mk.attn_packed(q, k, k[:2], cu, out, workspace=ws),
                lambda: mk.attn_packed(q, k, k, cu.long(), out, workspace=ws)):
        with pytest.raises(ValueError):
            bad()


def test_reference_e4m3_against_torch():
    """The tests' own 8-bit rounding, on every bf16 value up to 448 and on rows."""
    torch = pytest.importorskip("torch")
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    full = torch.full((len(x), 1), 448.0)
    codes, scale = ref.to_e4m3(torch.cat([x[:, None], full], 1))
    assert bool((scale == 1).all())
    assert torch.equal(codes[:, 0].float(), x.to(torch.float8_e4m3fn).float())
    rows = torch.tensor([[448.0, 1.0], [449.0, 1.0], [0.0, 0.0], [1e-30, 0.0], [1.75, -1.0]])
    assert ref.to_e4m3(rows)[1].tolist() == [1.0, 2.0, 2.0 ** -64, 2.0 ** -64, 2.0 ** -8]


def test_binding_takes_no_other_objects():
    """What is no tensor (or a tensor of a subclass) is not handed to the quick way's
    tensor functions; the long way answers for it."""
    torch = pytest.importorskip("torch")
    q, pos = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    rope = mk.Rope(64, 1e4)
    for bad in ([1, 2], "text", 5, None, object(), torch.nn.Parameter(torch.zeros(3, 4, 64)), q):
        assert not mk._norm_rope_call.quick(rope.address, bad, q, pos, None, None, None, None, 1e-6)
        with pytest.raises((ValueError, AttributeError)):
            mk.qk_norm_rope(rope, bad, None, pos)
