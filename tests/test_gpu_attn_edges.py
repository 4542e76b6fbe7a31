"""GPU tests of the attention calls at the corners of what include/mk.h allows:
what lies behind a sequence in its last page, rows that share memory, streams
that are not the current one; against attention in 64 bits (attention_ref.attend,
whose error bounds are derived there) or the same call in its ordinary form."""
import math

import pytest

import attention_ref as ref
from test_gpu_attn import make_paged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def mk():
    import attention_decode_megakernel_b200 as m
    from attention_decode_megakernel_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


@pytest.mark.parametrize("behind", [2.0 ** -140, 2.0 ** -149, -(2.0 ** -140), 0.0, -1.0, math.inf,
                                    -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("t", [1, 3, 40])
def test_scales_behind_a_sequence(mk, behind, dtype, hd, t):
    """The scales that a page of an e4m3 cache holds behind a sequence are never part of
    a result, whatever they are: subnormal, zero, negative, infinite or NaN."""
    gen = torch.Generator(device="cuda").manual_seed(hd + t)
    lens = [1, 2, 15, 17, 31, 77, 129, 300]
    pool, table, rows = make_paged(gen, lens, 2, hd, 32, E4)
    for s in pool[2:]:  # (make_paged leaves NaN wherever no key lies)
        s.copy_(torch.where(torch.isnan(s), torch.full_like(s, behind), s))
    q = torch.randn(t * len(lens), 8, hd, generator=gen, device="cuda").to(dtype)
    out, lse = torch.empty_like(q), torch.empty(len(q), 8, device="cuda")
    cu = torch.arange(len(lens) + 1, **I32) * t
    mk.attn_paged(q, mk.KvCache(*pool), table, torch.tensor(lens, **I32), cu, out, lse=lse)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        at = slice(b * t, (b + 1) * t)
        want = ref.attend(q[at].cpu().double(), rows[b][0], rows[b][1],
                          [max(0, n - t + i + 1) for i in range(t)], hd ** -0.5, dtype, HF,
                          rows[b][2])
        ref.check(out[at], want[0], want[2], "out of sequence %d" % b)
        ref.check(lse[at], want[1], want[3], "lse of sequence %d" % b)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hd,n", [(64, 300), (128, 700), (256, 145)])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
def test_packed_keys_that_share_heads(mk, dtype, hd, n, which):
    """Keys or values expanded over their heads give the bits of their contiguous copies."""
    gen = torch.Generator(device="cuda").manual_seed(hd)
    q, k, v = (torch.randn(n, h, hd, generator=gen, device="cuda").to(dtype) for h in (8, 4, 4))
    if "k" in which:
        k = k[:, 1:2].expand(-1, 4, -1)
    if "v" in which:
        v = v[:, 2:3].expand(-1, 4, -1)
    cu = torch.tensor([0, n // 3, n], **I32)
    got, want = torch.empty_like(q), torch.empty_like(q)
    lse = [torch.empty(n, 8, device="cuda") for _ in "ab"]
    mk.attn_packed(q, k, v, cu, got, lse=lse[0])
    mk.attn_packed(q, k.contiguous(), v.contiguous(), cu, want, lse=lse[1])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(*lse)
    for at in (slice(0, n // 3), slice(n // 3, n)):
        x = ref.attend(q[at].cpu().double(), k[at].cpu().double(), v[at].cpu().double(),
                       list(range(1, at.stop - at.start + 1)), hd ** -0.5, dtype, dtype)
        ref.check(got[at], x[0], x[2], "out")


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("heads", [4, 8])
def test_paged_queries_that_share_rows(mk, kind, hd, heads):
    """Queries expanded over heads, tokens or both: the bits of their contiguous copies
    while a unit has 16 rows or less, a refusal that writes nothing beyond."""
    gen = torch.Generator(device="cuda").manual_seed(hd)
    lens, t = [40, 300], 4
    pool, table, _ = make_paged(gen, lens, 2, hd, 16, kind)
    cache, sl = mk.KvCache(*pool), torch.tensor(lens, **I32)
    base = torch.randn(2 * t, heads, hd, generator=gen, device="cuda").to(BF)
    cu = torch.tensor([0, t, 2 * t], **I32)
    for q in (base[:, 3:4].expand(-1, heads, -1), base[5:6].expand(2 * t, -1, -1),
              base[:1, :1].expand(2 * t, heads, -1)):
        got, want = (torch.full((2 * t, heads, hd), math.nan, dtype=BF, device="cuda")
                     for _ in "ab")
        mk.attn_paged(q, cache, table, sl, cu, got)
        mk.attn_paged(q.contiguous(), cache, table, sl, cu, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want)  # (and so no NaN that was there before)
        got.fill_(7)
        rows = torch.tensor([0, 2 * t], **I32)  # one sequence: units of 16 or 32 rows
        if heads == 4:
            mk.attn_paged(q, cache, table[1:], sl[1:], rows, got)
            mk.attn_paged(q.contiguous(), cache, table[1:], sl[1:], rows, want)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        else:
            with pytest.raises(mk.MkError):
                mk.attn_paged(q, cache, table[1:], sl[1:], rows, got)
            with pytest.raises(mk.MkError):
                mk.attn_packed(q, q[:, :2], q[:, :2], rows, got)
            torch.cuda.synchronize()
            assert bool((got == 7).all())


@pytest.mark.parametrize("n,heads", [(1, 4), (5, 1), (5, 4), (70, 4)])
def test_outputs_in_any_order(mk, n, heads):
    """Outputs laid out [head][token][dim], of one token or of one head: the bits of
    contiguous ones."""
    hd = 64
    gen = torch.Generator(device="cuda").manual_seed(n + heads)
    q, k, v = (torch.randn(n, heads, hd, generator=gen, device="cuda").to(BF) for _ in "qkv")
    cu, pos = torch.tensor([0, n], **I32), torch.arange(n, **I32)
    pool, table, _ = make_paged(gen, [n], heads, hd, 16, BF)
    cache, slots = mk.KvCache(*pool), table[0].long()[pos.long() // 16] * 16 + pos % 16

    def outputs(turned):
        a = [torch.full((heads, n, hd) if turned else (n, heads, hd), 9.0, dtype=BF, device="cuda")
             for _ in range(6)]
        return [x.transpose(0, 1) for x in a] if turned else a

    sides = []
    for turned in (False, True):
        o = outputs(turned)
        mk.qk_norm_rope(mk.Rope(64, 1e4), q, k, pos, o[0], o[1])
        mk.kv_read(cache, slots, o[2], o[3])
        mk.attn_packed(q, k, v, cu, o[4])
        mk.attn_paged(q, cache, table, cu[1:], cu, o[5])
        sides.append(o)
    torch.cuda.synchronize()
    for a, b in zip(*sides):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("t", [1, 40])
def test_own_workspace_on_another_stream(mk, kind, t):
    """Calls on streams that are not the current one, without a workspace, while the current
    one takes and fills memory: the bits of a call alone."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    pool, table, _ = make_paged(gen, [5000, 900], 2, 128, 64, kind)
    cache, lens = mk.KvCache(*pool), torch.tensor([5000, 900], **I32)
    q = torch.randn(2 * t, 8, 128, generator=gen, device="cuda").to(BF)
    k, v = (torch.randn(2 * t, 2, 128, generator=gen, device="cuda").to(BF) for _ in "kv")
    cu = torch.tensor([0, t, 2 * t], **I32)

    def both(a, b, **given):
        mk.attn_paged(q, cache, table, lens, cu, a, **given)
        mk.attn_packed(q, k, v, cu, b, **given)

    want = [torch.empty_like(q) for _ in "ab"]
    both(*want)
    torch.cuda.synchronize()
    size = mk.lib().mk_attn_ws_bytes(128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    handles = [s.cuda_stream for s in streams] + [0]
    got = [[torch.full_like(q, math.nan) for _ in "ab"] for _ in handles]
    torch.cuda.synchronize()
    for _ in range(10):
        for out, h in zip(got, handles):
            both(*out, stream=h)
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for out in got:
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    owners = {s["stream"] for s in torch.cuda.memory_snapshot() if s["total_size"] >= size}
    assert owners >= set(handles[:2])
    # and captured, by the handle of the stream that captures
    out = [torch.full_like(q, math.nan) for _ in "ab"]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(*out, stream=torch.cuda.current_stream().cuda_stream)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refused_calls_write_nothing(mk):
    """Neither way of the binding launches anything for a call that it refuses: every
    buffer that the call could have written keeps its bits."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    hq, hk, hd, n = 8, 2, 64, 10
    x = torch.randn(n, hq + 2 * hk, hd, generator=gen, device="cuda").to(BF)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    pos, slots = torch.arange(n, **I32), torch.arange(n, device="cuda")
    pool = [torch.randn(2, hk, 16, hd, generator=gen, device="cuda").to(BF) for _ in "kv"]
    cache, rope, ws = mk.KvCache(*pool), mk.Rope(64, 1e4), mk.attn_workspace(hd)
    table, lens, cu = (torch.tensor(y, **I32) for y in ([[0, 1]], [n], [0, n]))
    out, lse = torch.full((n, hq, hd), 3.0, dtype=BF, device="cuda"), torch.full((n, hq), 3.0,
                                                                               device="cuda")
    kb, vb = (torch.full((n, hk, hd), 3.0, dtype=BF, device="cuda") for _ in "kv")
    written = [x, *pool, out, lse, kb, vb]
    before = [y.clone() for y in written]
    refused = [
        lambda **s: mk.qk_norm_rope(rope, q, k, pos.long(), **s),
        lambda **s: mk.qk_norm_rope(rope, q, k, pos[:9], **s),
        lambda **s: mk.qk_norm_rope(rope, q, k[:5], pos, out, kb, **s),
        lambda **s: mk.qk_norm_rope(rope, q, k, pos, out, kb[:, :1], **s),
        lambda **s: mk.qk_norm_rope(rope, q, k, pos, out, kb, q_gain=ws[:64], **s),
        lambda **s: mk.qk_norm_rope(rope, q, k, pos, out, kb, eps=-1.0, **s),
        lambda **s: mk.qk_norm_rope(mk.Rope(128, 1e4), q, k, pos, out, kb, **s),
        lambda **s: mk.kv_write(cache, k, v[:, :1], slots, **s),
        lambda **s: mk.kv_write(cache, k, v, slots[:9], **s),
        lambda **s: mk.kv_write(cache, q, q, slots, **s),
        lambda **s: mk.kv_read(cache, slots.int(), kb, vb, **s),
        lambda **s: mk.kv_read(cache, slots, kb, vb[:, :1].expand(-1, hk, -1), **s),
        lambda **s: mk.attn_paged(q, cache, table.t(), lens, cu, out, lse, workspace=ws, **s),
        lambda **s: mk.attn_paged(q, cache, table, lens, cu[:1], out, lse, workspace=ws, **s),
        lambda **s: mk.attn_paged(q, cache, table, lens, cu, out[:9], lse, workspace=ws, **s),
        lambda **s: mk.attn_paged(q, cache, table, lens, cu, out, lse[:, :7], workspace=ws, **s),
        lambda **s: mk.attn_paged(q, cache, table, lens, cu, out, lse, workspace=ws[:4096], **s),
        lambda **s: mk.attn_paged(q, cache, table, lens, cu, out, lse, scale=0.0, workspace=ws, **s),
        lambda **s: mk.attn_packed(q, k, v[:9], cu, out, lse, workspace=ws, **s),
        lambda **s: mk.attn_packed(q, k, v, cu.cpu(), out, lse, workspace=ws, **s),
        lambda **s: mk.attn_packed(q, k, v, cu, out, lse, workspace=ws[:4096], **s),
        lambda **s: mk.attn_packed(q[:, :7], k, v, cu, out[:, :7], lse[:, :7].contiguous(),
                                   workspace=ws, **s)]
    for given in ({}, dict(stream=torch.cuda.current_stream().cuda_stream)):
        for i, call in enumerate(refused):
            with pytest.raises((ValueError, mk.MkError)):
                call(**given)
            torch.cuda.synchronize()
            for a, b in zip(written, before):
                assert torch.equal(a, b), i
    mk.attn_packed(q, k, v, cu, out, lse, workspace=ws)  # what they would have done
    torch.cuda.synchronize()
    assert not bool((out == 3).all()) and not bool((lse == 3).any())
