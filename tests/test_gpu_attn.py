"""GPU tests of mk_attn_paged and mk_attn_packed against attention in 64 bits
(attention_ref.attend, whose error bounds are derived there)."""
import math

import pytest

import attention_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mk():
    import attention_decode_megakernel_b200 as m
    from attention_decode_megakernel_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def make_paged(gen, lens, heads, hd, size, kind, layout="hpd", spread=1.0, spare=2):
    """A cache that holds sequences of `lens` keys in pages in random order, NaN in
    every place behind them; returns (cache tensors, table, K, V in 64 bits)."""
    need = [-(-n // size) for n in lens]
    pages = sum(need) + spare
    raw = torch.uint8 if kind == E4 else kind
    shape = (pages, heads, size, hd) if layout != "phd" else (pages, size, heads, hd)
    k, v = (torch.full(shape, 127 if kind == E4 else math.nan, dtype=raw, device="cuda")
            for _ in "kv")
    if layout == "phd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    scales = [None, None]
    if kind == E4:
        scales = [torch.full((pages, heads, size), math.nan, device="cuda") for _ in "kv"]
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    table = torch.full((len(lens), max(1, max(need))), 1 << 30, dtype=torch.int32)
    rows = []
    for b, n in enumerate(lens):
        kv = []
        for i, pool in enumerate((k, v)):
            x = torch.randn(n, heads, hd, generator=gen, device="cuda") * (spread if i == 0 else 1)
            if kind == E4:
                x *= torch.exp(torch.randn(n, heads, 1, generator=gen, device="cuda") / 2)
                codes, scale = ref.to_e4m3(x.cpu())
                kv.append(codes * scale[..., None])
                if i == 1:
                    kv.append(scale)
                stored = codes.float().to(E4).view(torch.uint8).cuda()
            else:
                stored = x.to(kind)
                kv.append(stored.cpu().double())
            for p in range(need[b]):
                at = slice(p * size, min(n, (p + 1) * size))
                page = order[sum(need[:b]) + p]
                table[b, p] = page
                pool[page, :, :at.stop - at.start] = stored[at].transpose(0, 1)
                if kind == E4:
                    scales[i][page, :, :at.stop - at.start] = scale[at].T.float().cuda()
        rows.append(kv)
    if kind == E4:
        k, v = k.view(E4), v.view(E4)
    return (k, v, scales[0], scales[1]), table.cuda(), rows


def run_paged(mk, gen, new, lens, hq, hk, hd, size, dtype, kind, layout="hpd", pad=2, scale=None,
              spread=1.0, workspace=None):
    """One call, checked row by row; returns what it was called with."""
    pool, table, rows = make_paged(gen, lens, hk, hd, size, kind, layout, spread)
    total = sum(new)
    q = torch.randn(total + pad, hq, hd, generator=gen, device="cuda").to(dtype)
    q[total:] = math.nan
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((total + pad, hq, hd), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((total + pad, hq), 7.0, device="cuda")
    cache = mk.KvCache(*pool)
    args = (q, cache, table, sl, cu, out)
    mk.attn_paged(*args, lse=lse, scale=scale, workspace=workspace)
    torch.cuda.synchronize()
    assert bool((out[total:] == 7).all()) and bool((lse[total:] == 7).all())
    first = 0
    for b, (t, n) in enumerate(zip(new, lens)):
        seen = [max(0, n - t + i + 1) for i in range(t)]
        want = ref.attend(q[first:first + t].cpu().double(), rows[b][0], rows[b][1], seen,
                          hd ** -0.5 if scale is None else scale, dtype,
                          HF if kind == E4 else dtype, rows[b][2] if kind == E4 else None)
        ref.check(out[first:first + t], want[0], want[2], "out of sequence %d" % b)
        ref.check(lse[first:first + t], want[1], want[3], "lse of sequence %d" % b)
        first += t
    return args, lse


KINDS = [(BF, BF), (HF, HF), (BF, E4), (HF, E4)]
LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 500, 1000]


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,size,layout", [(8, 2, 16, "hpd"), (3, 1, 64, "phd"),
                                               (16, 1, 32, "hpd"), (5, 5, 256, "phd")])
def test_paged_single_tokens(mk, dtype, kind, hd, hq, hk, size, layout):
    """Decoding: one new token for each sequence, one sequence without keys."""
    gen = torch.Generator(device="cuda").manual_seed(hd + hq)
    run_paged(mk, gen, [1] * len(LENS), LENS, hq, hk, hd, size, dtype, kind, layout)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,size", [(8, 2, 16), (3, 1, 64), (40, 1, 128), (2, 2, 256)])
def test_paged_chunks(mk, dtype, kind, hd, hq, hk, size):
    """Chunks from nothing to 300 tokens, whole prompts and rows that see no key."""
    gen = torch.Generator(device="cuda").manual_seed(hd * hq)
    new = [5, 0, 8, 1, 33, 130, 300, 7, 64, 3]
    lens = [700, 0, 8, 1, 40, 131, 300, 4, 129, 0]
    run_paged(mk, gen, new, lens, hq, hk, hd, size, dtype, kind, pad=3)


@pytest.mark.parametrize("kind", [BF, E4])
def test_paged_verify_of_drafts(mk, kind):
    gen = torch.Generator(device="cuda").manual_seed(11)
    run_paged(mk, gen, [5, 5, 3, 4], [4096, 700, 3, 2049], 8, 2, 256, 16, BF, kind)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("t", [1, 6, 70])
def test_paged_long_context(mk, dtype, kind, t):
    """One sequence split over all multiprocessors."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    run_paged(mk, gen, [t], [20011], 8, 2, 128, 64, dtype, kind)


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_paged_one_sequence_in_few_and_many_parts(mk, kind, hd):
    """Partial results of 1 to 148 stretches of keys: one warp's and several warps' joins."""
    gen = torch.Generator(device="cuda").manual_seed(hd + 1)
    for n in (129, 513, 700, 1025, 1290, 2000, 4700, 9700):
        run_paged(mk, gen, [1], [n], 2, 1, hd, 32, BF, kind)
    run_paged(mk, gen, [3], [5000], 4, 1, hd, 32, BF, kind)


def test_paged_peaked_scores(mk):
    """Scores of several hundred, the largest in any place: the running maximum."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    for t in (1, 40):
        run_paged(mk, gen, [t, t], [1500, 300], 4, 1, 128, 32, BF, BF, spread=8.0, scale=1.0)
        run_paged(mk, gen, [t, t], [1500, 300], 4, 1, 256, 32, HF, E4, spread=8.0, scale=1.0)


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("t", [1, 50])
def test_paged_rising_scores(mk, kind, t):
    """Keys that grow along the sequence: the maximum rises in every tile."""
    gen = torch.Generator(device="cuda").manual_seed(17)
    n, hd = 900, 128
    pool, table, _ = make_paged(gen, [n], 1, hd, 16, kind)
    k = torch.linspace(0.1, 12, n)[:, None, None] * torch.ones(n, 1, hd)
    v = torch.randn(n, 1, hd)
    cache = mk.KvCache(*pool)
    slots = (table[0].long()[torch.arange(n, device="cuda") // 16] * 16
             + torch.arange(n, device="cuda") % 16)
    mk.kv_write(cache, k.cuda().to(BF), v.cuda().to(BF), slots)
    kb, vb = torch.empty(n, 1, hd, device="cuda"), torch.empty(n, 1, hd, device="cuda")
    mk.kv_read(cache, slots, kb, vb)
    q = (1 + 0.1 * torch.randn(t, 2, hd, generator=gen, device="cuda")).to(BF)
    out, lse = torch.empty_like(q), torch.empty(t, 2, device="cuda")
    cu = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    mk.attn_paged(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), cu, out,
                  lse=lse)
    torch.cuda.synchronize()
    want = ref.attend(q.cpu().double(), kb.cpu().double(), vb.cpu().double(),
                      [n - t + i + 1 for i in range(t)], hd ** -0.5, BF, HF if kind == E4 else BF,
                      pool[3][slots // 16, :, slots % 16].cpu() if kind == E4 else None)
    ref.check(out, want[0], want[2], "out")
    ref.check(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("t", [1, 40])
def test_paged_pages_outside_the_cache(mk, kind, t):
    """A page number outside the cache stands for zeros; seq_lens beyond the table is
    held to it."""
    gen = torch.Generator(device="cuda").manual_seed(19)
    lens = [200, 77]
    pool, table, rows = make_paged(gen, lens, 2, 64, 16, kind)
    table[0, 3], table[0, 7], table[1, 1] = -1, pool[0].shape[0], -(1 << 31)
    for b, p in ((0, 3), (0, 7), (1, 1)):
        for x in rows[b][:2]:
            x[16 * p:16 * p + 16] = 0
    held = table.shape[1] * 16
    assert held == 208
    lens = [10 ** 6, 77]
    table[0, 12] = -5  # the positions 192 .. 207 are zeros too
    for x in (0, 1):
        rows[0][x] = torch.cat([rows[0][x][:192], torch.zeros(16, 2, 64, dtype=torch.float64)])
    if kind == E4:  # rows of zeros count with a scale of one
        for b, p in ((0, 3), (0, 7), (1, 1)):
            rows[b][2][16 * p:16 * p + 16] = 1
        rows[0][2] = torch.cat([rows[0][2][:192], torch.ones(16, 2, dtype=torch.float64)])
    q = torch.randn(2 * t, 4, 64, generator=gen, device="cuda").to(BF)
    out = torch.empty_like(q)
    cu = torch.tensor([0, t, 2 * t], dtype=torch.int32, device="cuda")
    mk.attn_paged(q, mk.KvCache(*pool), table,
                  torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, out)
    torch.cuda.synchronize()
    for b, n in enumerate((held, 77)):
        want = ref.attend(q[b * t:(b + 1) * t].cpu().double(), rows[b][0], rows[b][1],
                          [n - t + i + 1 for i in range(t)], 0.125, BF, HF if kind == E4 else BF,
                          rows[b][2] if kind == E4 else None)
        ref.check(out[b * t:(b + 1) * t], want[0], want[2], "out")


@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("t", [1, 33])
def test_paged_offsets_past_32_bits(mk, kind, t):
    """The last pages of a pool of more than 2^31 values."""
    pages, heads, size, hd = 2100, 16, 256, 256
    gen = torch.Generator(device="cuda").manual_seed(23)
    k = torch.empty((pages, heads, size, hd), dtype=torch.uint8 if kind == E4 else kind,
                    device="cuda")
    v = torch.empty_like(k)
    s = [torch.empty((pages, heads, size), device="cuda") for _ in "kv"] if kind == E4 else [None] * 2
    cache = mk.KvCache(k.view(kind), v.view(kind), *s)
    n = 300
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    at = torch.arange(n, device="cuda")
    slots = table[0].long()[at // size] * size + at % size
    x = torch.randn(2, n, heads, hd, generator=gen, device="cuda").to(BF)
    mk.kv_write(cache, x[0], x[1], slots)
    kb, vb = torch.empty_like(x[0]), torch.empty_like(x[0])
    mk.kv_read(cache, slots, kb, vb)
    q = torch.randn(t, heads, hd, generator=gen, device="cuda").to(BF)
    out = torch.empty_like(q)
    mk.attn_paged(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                  torch.tensor([0, t], dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    want = ref.attend(q.cpu().double(), kb.cpu().double(), vb.cpu().double(),
                      [n - t + i + 1 for i in range(t)], hd ** -0.5, BF, HF if kind == E4 else BF,
                      s[1][slots // size, :, slots % size].cpu() if kind == E4 else None)
    ref.check(out, want[0], want[2], "out")


def run_packed(mk, gen, lens, hq, hk, hd, dtype, pad=2, fused=True, scale=None, spread=1.0):
    total = sum(lens)
    rows = torch.randn(total + pad, hq + 2 * hk, hd, generator=gen, device="cuda")
    rows[:, hq:hq + hk] *= spread
    rows = rows.to(dtype)
    rows[total:] = math.nan  # behind the last sequence
    q, k, v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
    if not fused:  # [head][token][dim]
        q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    out = torch.full((total + pad, hq, hd), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((total + pad, hq), 7.0, device="cuda")
    mk.attn_packed(q, k, v, cu, out, lse=lse, scale=scale)
    torch.cuda.synchronize()
    assert bool((out[total:] == 7).all()) and bool((lse[total:] == 7).all())
    first = 0
    for b, n in enumerate(lens):
        at = slice(first, first + n)
        want = ref.attend(q[at].cpu().double(), k[at].cpu().double(), v[at].cpu().double(),
                          list(range(1, n + 1)), hd ** -0.5 if scale is None else scale, dtype,
                          dtype)
        ref.check(out[at], want[0], want[2], "out of sequence %d" % b)
        ref.check(lse[at], want[1], want[3], "lse of sequence %d" % b)
        first += n
    return (q, k, v, cu, out), lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,fused", [(8, 2, True), (3, 1, False), (40, 1, True), (2, 2, False)])
def test_packed(mk, dtype, hd, hq, hk, fused):
    gen = torch.Generator(device="cuda").manual_seed(hd + 7 * hq)
    run_packed(mk, gen, [1, 0, 2, 17, 31, 32, 33, 127, 128, 129, 300], hq, hk, hd, dtype,
               fused=fused)


@pytest.mark.parametrize("hd,hq,hk", [(64, 4, 1), (128, 4, 2), (256, 8, 2)])
def test_packed_one_long_prompt(mk, hd, hq, hk):
    gen = torch.Generator(device="cuda").manual_seed(hd)
    run_packed(mk, gen, [1531], hq, hk, hd, BF, pad=0)
    run_packed(mk, gen, [1100, 1, 515], hq, hk, hd, HF, spread=6.0, scale=1.0)


def test_packed_nan_of_another_sequence(mk):
    """A sequence full of NaN and infinities spoils no other."""
    gen = torch.Generator(device="cuda").manual_seed(29)
    lens, hq, hk, hd = [70, 40, 90], 4, 2, 64
    rows = torch.randn(200, hq + 2 * hk, hd, generator=gen, device="cuda").to(BF)
    rows[70:110] = math.nan
    rows[75] = math.inf
    q, k, v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
    cu = torch.tensor([0, 70, 110, 200], dtype=torch.int32, device="cuda")
    out = torch.empty(200, hq, hd, dtype=BF, device="cuda")
    mk.attn_packed(q, k, v, cu, out)
    torch.cuda.synchronize()
    for at in (slice(0, 70), slice(110, 200)):
        want = ref.attend(q[at].cpu().double(), k[at].cpu().double(), v[at].cpu().double(),
                          list(range(1, at.stop - at.start + 1)), hd ** -0.5, BF, BF)
        ref.check(out[at], want[0], want[2], "out")


def test_packed_equals_paged(mk):
    """A whole prompt through a paged cache gives what the packed call gives."""
    gen = torch.Generator(device="cuda").manual_seed(31)
    n, hq, hk, hd = 260, 8, 2, 128
    q, k, v = (torch.randn(n, h, hd, generator=gen, device="cuda").to(BF) for h in (hq, hk, hk))
    pool = [torch.empty(17, hk, 16, hd, dtype=BF, device="cuda") for _ in "kv"]
    cache = mk.KvCache(*pool)
    table = torch.randperm(17, generator=gen, device="cuda").to(torch.int32)[None]
    at = torch.arange(n, device="cuda")
    mk.kv_write(cache, k, v, table[0].long()[at // 16] * 16 + at % 16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    mk.attn_packed(q, k, v, cu, a)
    mk.attn_paged(q, cache, table, cu[1:], cu, b)
    torch.cuda.synchronize()
    for got in (a, b):
        want = ref.attend(q.cpu().double(), k.cpu().double(), v.cpu().double(),
                          list(range(1, n + 1)), hd ** -0.5, BF, BF)
        ref.check(got, want[0], want[2], "out")


@pytest.mark.parametrize("t", [1, 20, 200])
@pytest.mark.parametrize("kind", [BF, E4])
def test_same_bits_again_on_a_stream_and_in_a_graph(mk, kind, t):
    gen = torch.Generator(device="cuda").manual_seed(37)
    ws = mk.attn_workspace(256)
    args, lse = run_paged(mk, gen, [t, 1, t], [5000, 800, 401], 8, 2, 256, 16, BF, kind,
                          workspace=ws)
    out = args[5]
    first = (out.clone(), lse.clone())
    ws.fill_(255)  # its content does not matter
    for _ in range(3):
        out.fill_(0)
        mk.attn_paged(*args, lse=lse, workspace=ws)
        assert torch.equal(out[:2 * t + 1], first[0][:2 * t + 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.fill_(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        mk.attn_paged(*args, lse=lse)
    side.synchronize()
    assert torch.equal(out[:2 * t + 1], first[0][:2 * t + 1])
    # two graphs that share a workspace, replayed in turn; the second on shorter lengths
    outs = [torch.zeros_like(out) for _ in "ab"]
    lens = [args[3], args[3].clone()]
    graphs = []
    for o, sl in zip(outs, lens):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mk.attn_paged(args[0], args[1], args[2], sl, args[4], o, workspace=ws)
        graphs.append(g)
    lens[1] -= 300  # lengths are read when the graph runs
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][:2 * t + 1], first[0][:2 * t + 1])
    again = torch.zeros_like(out)
    mk.attn_paged(args[0], args[1], args[2], lens[1], args[4], again, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(outs[1], again) and not torch.equal(outs[0], outs[1])


def test_packed_same_bits_in_a_graph(mk):
    gen = torch.Generator(device="cuda").manual_seed(41)
    args, lse = run_packed(mk, gen, [700, 33, 290], 8, 2, 128, BF, pad=0)
    out = args[4].clone()
    ws = mk.attn_workspace(128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mk.attn_packed(*args, workspace=ws)
    args[4].fill_(0)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[4], out)


def test_calls_side_by_side(mk):
    """Two streams at once, a workspace each."""
    gen = torch.Generator(device="cuda").manual_seed(43)
    calls = [run_paged(mk, gen, [1, 9], [9000, 4000], 8, 2, 128, 64, BF, BF) for _ in range(2)]
    want = [c[0][5].clone() for c in calls]
    ws = [mk.attn_workspace(128) for _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for (args, lse), s, w in zip(calls, streams, ws):
            with torch.cuda.stream(s):
                mk.attn_paged(*args, lse=lse, workspace=w)
    torch.cuda.synchronize()
    for (args, _), x in zip(calls, want):
        assert torch.equal(args[5], x)


def test_many_sequences(mk):
    """A batch of 700 short sequences, some empty."""
    gen = torch.Generator(device="cuda").manual_seed(47)
    lens = [(7 * i) % 90 for i in range(700)]
    run_paged(mk, gen, [1] * 700, lens, 2, 1, 64, 16, BF, BF)
    run_packed(mk, gen, [i % 9 for i in range(700)], 2, 1, 64, BF)


@pytest.mark.parametrize("kind", [BF, E4])
def test_more_sequences_than_a_warp_remembers(mk, kind):
    """2100 sequences, runs of empty ones among them: shares found from two rounds each on."""
    gen = torch.Generator(device="cuda").manual_seed(48)
    new = [0 if 900 < i < 1400 or i % 50 == 7 else 1 + (i % 700 == 0) for i in range(2100)]
    lens = [(7 * i) % 90 if n else 0 for i, n in enumerate(new)]
    run_paged(mk, gen, new, lens, 2, 1, 64, 16, BF, kind)
    run_paged(mk, gen, [9 * n for n in new], [n + 9 for n in lens], 4, 1, 64, 16, BF, kind)


def test_nothing_to_do(mk):
    pool, table, _ = make_paged(torch.Generator(device="cuda").manual_seed(1), [5], 1, 64, 16, BF)
    q = torch.zeros(4, 2, 64, dtype=BF, device="cuda")
    out = torch.full_like(q, 3)
    i32 = dict(dtype=torch.int32, device="cuda")
    mk.attn_paged(q, mk.KvCache(*pool), table, torch.tensor([5], **i32),
                  torch.tensor([0, 0], **i32), out)
    mk.attn_packed(q, q[:, :1], q[:, :1], torch.tensor([0, 0, 0], **i32), out)
    mk.attn_packed(q[:0], q[:0, :1], q[:0, :1], torch.tensor([0, 0], **i32), out[:0])
    mk.attn_paged(q, mk.KvCache(*pool), table[:0], torch.zeros(0, **i32), torch.zeros(1, **i32), out)
    torch.cuda.synchronize()
    assert bool((out == 3).all())
