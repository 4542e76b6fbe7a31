"""GPU tests of mk_kv_write and mk_kv_read: bit for bit against the format's
definition, for every type, page layout and kind of slot."""
import math

import pytest

import attention_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mk():
    import attention_decode_megakernel_b200 as m
    from attention_decode_megakernel_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def make_pool(pages, heads, size, hd, dtype, layout="hpd"):
    """k and v views [page][head][position][dim]: heads outside ("hpd"), positions
    outside ("phd"), or k and v side by side in one tensor ("both")."""
    raw = torch.int8 if dtype == E4 else dtype
    if layout == "hpd":
        k, v = (torch.full((pages, heads, size, hd), 3, dtype=raw, device="cuda") for _ in "kv")
    elif layout == "phd":
        k, v = (torch.full((pages, size, heads, hd), 3, dtype=raw, device="cuda").transpose(1, 2)
                for _ in "kv")
    else:
        both = torch.full((pages, 2, heads, size, hd), 3, dtype=raw, device="cuda")
        k, v = both[:, 0], both[:, 1]
    if dtype != E4:
        return k, v, None, None
    scales = [torch.full((pages, heads, size), 5.0, device="cuda") for _ in "kv"]
    return k.view(E4), v.view(E4), scales[0], scales[1]


def _values(x):
    return (x.cpu().view(torch.uint8).view(E4).float() if x.dtype == E4 else x.cpu().float())


@pytest.mark.parametrize("row", [BF, HF, F32])
@pytest.mark.parametrize("kind", [BF, HF, E4])
@pytest.mark.parametrize("hd,heads,size,layout", [(64, 1, 16, "hpd"), (128, 3, 64, "phd"),
                                                  (256, 2, 256, "both"), (256, 8, 32, "phd")])
def test_write_and_read(mk, row, kind, hd, heads, size, layout):
    gen = torch.Generator(device="cuda").manual_seed(hd + heads)
    pages, n = 5, 61
    pool = make_pool(pages, heads, size, hd, kind, layout)
    before = [None if x is None else _values(x) for x in pool]
    cache = mk.KvCache(*pool)
    fused = torch.randn(n, 3 * heads, hd, generator=gen, device="cuda")
    fused *= torch.exp(3 * torch.randn(n, 3 * heads, 1, generator=gen, device="cuda"))
    fused[3, :, :] = 0
    fused = fused.to(row)
    k, v = fused[:, heads:2 * heads], fused[:, 2 * heads:]
    slots = torch.randperm(pages * size, generator=gen, device="cuda")[:n]
    slots[::7] = -1
    slots[5], slots[6] = pages * size, 1 << 40  # outside the cache, like -1
    mk.kv_write(cache, k, v, slots)
    ko, vo = (torch.full((n, heads, hd), -9.0, dtype=row, device="cuda") for _ in "kv")
    mk.kv_read(cache, slots, ko, vo)
    torch.cuda.synchronize()
    keep = [t for t in range(n) if 0 <= int(slots[t]) < pages * size]
    for i, (x, out) in enumerate(((k, ko), (v, vo))):
        x = x.cpu()
        if kind == E4:
            codes, scale = ref.to_e4m3(x.float())
            want, ws = before[i].clone(), before[2 + i].clone()
            for t in keep:
                want[int(slots[t]) // size, :, int(slots[t]) % size] = codes[t].float()
                ws[int(slots[t]) // size, :, int(slots[t]) % size] = scale[t].float()
            assert torch.equal(_values(pool[2 + i]), ws)
            back = (codes * scale[..., None]).to(row)
        else:
            back = x.to(kind)
            want = before[i].clone()
            for t in keep:
                want[int(slots[t]) // size, :, int(slots[t]) % size] = back[t].float()
            back = back.to(row)
        assert torch.equal(_values(pool[i]), want)
        expected = torch.full((n, heads, hd), -9.0, dtype=row)
        expected[keep] = back[keep]
        assert torch.equal(out.cpu(), expected)


def test_every_scale_and_tie(mk):
    """Rows whose largest value is next to 448 * 2^e for every e of fp32's range, and
    values at and next to the ties of the code."""
    rows = []
    for e in range(-126, 119):
        for m in (1.0, 1.75 - 2.0 ** -23, 1.75, 1.75 + 2.0 ** -23, 2 - 2.0 ** -23):
            r = torch.linspace(0, 1, 64)
            r[0] = m
            rows.append(r * 2.0 ** e if e > -100 else (r.double() * 2.0 ** e).float())
    ties = torch.arange(1, 65).float() + 0.5
    rows += [ties * 7, ties * 4, torch.nextafter(ties * 4, torch.tensor(1e9)),
             torch.nextafter(ties * 4, torch.tensor(0.0)), ties * 2.0 ** -80]
    x = torch.stack(rows)[:, None].contiguous()
    n = len(rows)
    pool = make_pool((n + 15) // 16, 1, 16, 64, E4)
    cache = mk.KvCache(*pool)
    slots = torch.arange(n, device="cuda")
    mk.kv_write(cache, x.cuda(), -x.cuda(), slots)
    torch.cuda.synchronize()
    codes, scale = ref.to_e4m3(x)
    got = _values(pool[0])[:, 0].reshape(-1, 64)[:n]
    assert torch.equal(pool[2].cpu().reshape(-1)[:n].double(), scale[:, 0])
    assert torch.equal(got.double(), codes[:, 0])
    assert torch.equal(_values(pool[1])[:, 0].reshape(-1, 64)[:n], -got)


def test_nan_and_infinity(mk):
    x = torch.ones(3, 1, 64, device="cuda")
    x[0, 0, 3], x[1, 0, 4], x[1, 0, 5] = float("nan"), float("inf"), -float("inf")
    pool = make_pool(1, 1, 16, 64, E4)
    cache = mk.KvCache(*pool)
    slots = torch.arange(3, device="cuda")
    mk.kv_write(cache, x, x, slots)
    back = torch.empty_like(x)
    mk.kv_read(cache, slots, back, torch.empty_like(x))
    torch.cuda.synchronize()
    assert bool(torch.isnan(back[0, 0, 3])) and int(torch.isnan(back).sum()) == 1
    assert bool((back[0, 0, :3] == 1).all()) and bool((back[2] == 1).all())
    # the largest code times the scale of an infinite row, 448 * 2^120 > 2^128, is infinite
    assert float(back[1, 0, 4]) == math.inf == -float(back[1, 0, 5])
    assert float(pool[2][0, 0, 1]) == 2.0 ** 120


def test_offsets_past_32_bits(mk):
    """A pool of more than 2^31 values: its last page."""
    pages, heads, size, hd = 2100, 16, 256, 256  # 2.2e9 values
    k = torch.empty((pages, heads, size, hd), dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    s = [torch.ones((pages, heads, size), device="cuda") for _ in "kv"]
    cache = mk.KvCache(k.view(E4), v.view(E4), *s)
    x = torch.randn(2, heads, hd, device="cuda").to(BF)
    slots = torch.tensor([pages * size - 1, (pages - 1) * size], device="cuda")
    mk.kv_write(cache, x, -x, slots)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    mk.kv_read(cache, slots, ko, vo)
    torch.cuda.synchronize()
    codes, scale = ref.to_e4m3(x.cpu().float())
    assert torch.equal(ko.cpu().double(), codes * scale[..., None])
    assert torch.equal(vo, -ko)
    assert torch.equal(k[-1, :, -1].view(E4).cpu().float().double(), codes[0])


def test_same_slot_read_twice_and_no_tokens(mk):
    pool = make_pool(2, 2, 16, 128, BF)
    cache = mk.KvCache(*pool)
    x = torch.randn(1, 2, 128, device="cuda").to(BF)
    mk.kv_write(cache, x, x, torch.tensor([17], device="cuda"))
    out = torch.zeros(3, 2, 128, dtype=BF, device="cuda")
    mk.kv_read(cache, torch.tensor([17, 17, 17], device="cuda"), out, out.clone())
    torch.cuda.synchronize()
    assert torch.equal(out, x.expand(3, 2, 128))
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    mk.kv_write(cache, x[:0], x[:0], none)
    mk.kv_read(cache, none, x[:0], x[:0])
