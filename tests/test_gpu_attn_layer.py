"""The operators of an attention layer one after another, as a serving program
calls them: a prompt's chunks and then single tokens of several sequences, from
a fused projection's rows through norm, rotation and the paged cache to the
attention; the engine's own cache read as pages; and the binding's two ways."""
import math

import numpy as np
import pytest

import attention_ref as ref

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


class Layer:
    """One attention layer's cache and buffers for `batch` sequences of up to `most`
    tokens, and a step that takes new tokens' fused rows [q | k | v]."""

    def __init__(self, mk, hq, hk, hd, batch, most, page, kind, dtype, seed):
        self.mk, self.hq, self.hk, self.hd, self.page, self.dtype = mk, hq, hk, hd, page, dtype
        gen = torch.Generator(device="cuda").manual_seed(seed)
        per = -(-most // page)
        raw = torch.uint8 if kind == E4 else kind
        pool = [torch.zeros(batch * per, hk, page, hd, dtype=raw, device="cuda").view(kind)
                for _ in "kv"]
        scales = [torch.ones(batch * per, hk, page, device="cuda") for _ in "kv"] \
            if kind == E4 else [None, None]
        self.cache = mk.KvCache(*pool, *scales)
        self.table = torch.randperm(batch * per, generator=gen,
                                    device="cuda").to(torch.int32).view(batch, per)
        self.gain = [(1 + torch.randn(hd, generator=gen, device="cuda") / 8).to(dtype) for _ in "qk"]
        self.rope = mk.Rope(hd // 2, 1e6, scaling="yarn", factor=4.0, original_ctx=64)
        self.ws = mk.attn_workspace(hd)
        self.rows = [torch.zeros(0, hk, 2, hd, dtype=torch.float64) for _ in range(batch)]
        self.kind = kind

    def step(self, fused, positions, slots, seq_lens, cu, out):
        """The five calls; everything on the device."""
        mk, hq, hk = self.mk, self.hq, self.hk
        q, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
        mk.qk_norm_rope(self.rope, q, k, positions, q_gain=self.gain[0], k_gain=self.gain[1])
        mk.kv_write(self.cache, k, v, slots)
        mk.attn_paged(q, self.cache, self.table, seq_lens, cu, out, workspace=self.ws)

    def run(self, fused, new, past):
        """One step for sequences with new[b] tokens behind past[b], checked."""
        batch, total = len(new), sum(new)
        at = [(b, past[b] + t) for b in range(batch) for t in range(new[b])]
        positions = torch.tensor([p for _, p in at], **I32)
        seq = torch.tensor([b for b, _ in at], device="cuda")
        slots = self.table[seq, positions.long() // self.page].long() * self.page \
            + positions.long() % self.page
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **I32)
        lens = torch.tensor([p + n for p, n in zip(past, new)], **I32)
        before = fused.clone()
        out = torch.zeros(total, self.hq, self.hd, dtype=self.dtype, device="cuda")
        self.step(fused, positions, slots, lens, cu, out)
        torch.cuda.synchronize()
        # each stage from what the one before left: rotation ..
        turns, length = ref.rope_turns(self.hd // 2, 1e6, "yarn", 4.0, 64.0)
        for i, (lo, hi) in enumerate(((0, self.hq), (self.hq, self.hq + self.hk))):
            want, tol = ref.norm_rope(before[:, lo:hi].cpu(), self.gain[i].cpu(), positions.cpu(),
                                      turns, length, False, 1e-6)
            tol = tol + ref.half_step(self.dtype) * (want.abs() + tol)
            # below the type's normal numbers the step is fixed: smallest_normal * eps (fp16 2^-24)
            tol += torch.finfo(self.dtype).smallest_normal * torch.finfo(self.dtype).eps
            ref.check(fused[:, lo:hi], want, tol, "qk"[i])
        # .. the cache ..
        kv = torch.stack([fused[:, self.hq:self.hq + self.hk], fused[:, self.hq + self.hk:]], 2).cpu()
        scale = None
        if self.kind == E4:
            codes, scale = ref.to_e4m3(kv.float())
            kv = codes * scale[..., None]
        kb, vb = (torch.zeros(total, self.hk, self.hd, device="cuda") for _ in "kv")
        self.mk.kv_read(self.cache, slots, kb, vb)
        torch.cuda.synchronize()
        assert torch.equal(kb.cpu().double(), kv[:, :, 0].double())
        assert torch.equal(vb.cpu().double(), kv[:, :, 1].double())
        # .. and the attention over all that was written so far
        first = 0
        for b, n in enumerate(new):
            self.rows[b] = torch.cat([self.rows[b], kv[first:first + n].double()])
            K, V = self.rows[b][:, :, 0], self.rows[b][:, :, 1]
            want = ref.attend(fused[first:first + n, :self.hq].cpu().double(), K, V,
                              [past[b] + t + 1 for t in range(n)], self.hd ** -0.5, self.dtype,
                              HF if self.kind == E4 else self.dtype,
                              None if self.kind != E4 else
                              ref.to_e4m3(V.reshape(-1, self.hd))[1].view(V.shape[:2]))
            ref.check(out[first:first + n], want[0], want[2], "sequence %d" % b)
            first += n
        return out


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (BF, E4), (HF, HF)])
@pytest.mark.parametrize("hd,hq,hk,page", [(64, 4, 1, 16), (256, 8, 2, 64), (128, 6, 2, 32)])
def test_chunks_then_tokens(mk, dtype, kind, hd, hq, hk, page):
    batch, most = 3, 400
    layer = Layer(mk, hq, hk, hd, batch, most, page, kind, dtype, hd)
    gen = torch.Generator(device="cuda").manual_seed(hd + 1)
    past = [0] * batch
    for new in ([200, 33, 1], [97, 60, 130], [1, 1, 1], [5, 3, 4], [1, 1, 1], [0, 2, 1]):
        fused = torch.randn(sum(new), hq + 2 * hk, hd, generator=gen, device="cuda").to(dtype)
        layer.run(fused, new, past)
        past = [p + n for p, n in zip(past, new)]


def test_decode_steps_in_a_graph(mk):
    """A captured step, replayed with positions, slots and lengths that change."""
    hq, hk, hd, page, batch, past = 8, 2, 128, 16, 4, 37
    gen = torch.Generator(device="cuda").manual_seed(5)
    prompt = torch.randn(batch * past, hq + 2 * hk, hd, generator=gen, device="cuda").to(BF)
    steps = torch.randn(3, batch, hq + 2 * hk, hd, generator=gen, device="cuda").to(BF)
    layers = [Layer(mk, hq, hk, hd, batch, 64, page, BF, BF, 9) for _ in range(2)]
    for layer in layers:
        layer.run(prompt.clone(), [past] * batch, [0] * batch)
    eager = [layers[0].run(steps[i].clone(), [1] * batch, [past + i] * batch) for i in range(3)]
    layer = layers[1]
    fused, pos = steps[0].clone(), torch.full((batch,), past, **I32)
    slots, lens = torch.zeros(batch, dtype=torch.int64, device="cuda"), torch.zeros(batch, **I32)
    cu, out = torch.arange(batch + 1, **I32), torch.zeros(batch, hq, hd, dtype=BF, device="cuda")

    def place(i):
        fused.copy_(steps[i])
        pos.fill_(past + i)
        lens.fill_(past + i + 1)
        slots.copy_(layer.table[:, (past + i) // page].long() * page + (past + i) % page)

    place(0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.step(fused, pos, slots, lens, cu, out)
    for i in range(3):
        place(i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i])


def test_engine_cache_as_pages(mk):
    """The engine's cache, as get_state copies it out, is a sequence of pages."""
    from attention_decode_megakernel_b200 import synth
    cfg = synth.tiny_config(max_ctx=128)
    eng = mk.Engine(cfg, synth.make_weights(cfg))
    eng.prefill(synth.make_tokens(cfg.vocab, 96))
    _, _, kc, vc = eng.get_state(with_kv=True)
    eng.sync()
    heads, n, hd = cfg.kv_heads, eng.position, cfg.head_dim
    assert n == 96
    k, v = (x[0].view(BF).view(heads, n // 16, 16, hd).transpose(0, 1) for x in (kc, vc))
    cache = mk.KvCache(k, v)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in (1, 7):
        q = torch.randn(t, cfg.q_heads, hd, generator=gen, device="cuda").to(BF)
        out = torch.empty_like(q)
        mk.attn_paged(q, cache, torch.arange(n // 16, **I32)[None], torch.tensor([n], **I32),
                      torch.tensor([0, t], **I32), out)
        torch.cuda.synchronize()
        rows = [x[0].view(BF).transpose(0, 1).cpu().double() for x in (kc, vc)]
        want = ref.attend(q.cpu().double(), rows[0], rows[1], [n - t + i + 1 for i in range(t)],
                          hd ** -0.5, BF, BF)
        ref.check(out, want[0], want[2], "out")


def test_both_ways_of_the_binding(mk, monkeypatch):
    """What the quick way does not take goes the long way, to the same bits; what
    neither takes says why, and nothing is launched."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    hq, hk, hd = 8, 2, 64
    x = torch.randn(10, hq + 2 * hk, hd, generator=gen, device="cuda").to(BF)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    pos = torch.arange(10, **I32)
    pool = [torch.zeros(2, hk, 16, hd, dtype=BF, device="cuda") for _ in "kv"]
    cache, rope = mk.KvCache(*pool), mk.Rope(64, 1e4)
    slots, ws = torch.arange(10, device="cuda"), mk.attn_workspace(hd)
    table, lens, cu = (torch.tensor(y, **I32) for y in ([[0, 1]], [10], [0, 10]))

    def everything(**stream):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        mk.qk_norm_rope(rope, q, k, pos, qo, ko, **stream)
        mk.kv_write(cache, ko, v, slots, **stream)
        kb, vb = torch.empty_like(k), torch.empty_like(v)
        mk.kv_read(cache, slots, kb, vb, **stream)
        a, b = torch.empty_like(qo), torch.empty_like(qo)
        mk.attn_paged(qo, cache, table, lens, cu, a, workspace=ws, **stream)
        mk.attn_packed(qo, ko, v, cu, b, workspace=ws, **stream)
        torch.cuda.synchronize()
        return qo, ko, kb, vb, a, b

    for call in (mk._norm_rope_call, mk._kv_write_call, mk._kv_read_call, mk._paged_call,
                 mk._packed_call):
        taken = []
        quick = call.quick
        monkeypatch.setattr(call, "quick", lambda *a, q=quick, t=taken: t.append(q(*a)) or t[-1])
        everything()
        assert taken == [True], call.name
    want = everything()
    got = everything(stream=torch.cuda.current_stream().cuda_stream)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    out = torch.empty_like(q)
    for bad in (lambda: mk.qk_norm_rope(rope, q, k, pos.long()),
                lambda: mk.qk_norm_rope(rope, q.transpose(1, 2), k, pos),
                lambda: mk.qk_norm_rope(rope, q, k.float(), pos),
                lambda: mk.qk_norm_rope(rope, q, k[:5], pos),
                lambda: mk.qk_norm_rope(rope, q, k, pos.cpu()),
                lambda: mk.qk_norm_rope(rope, q, k, pos, q_gain=torch.ones(64, device="cuda")),
                lambda: mk.kv_write(cache, k, v[:, :1], slots),
                lambda: mk.kv_write(cache, k, v, slots[:9]),
                lambda: mk.kv_write(cache, q, q, slots),
                lambda: mk.kv_read(cache, slots.int(), k, v),
                lambda: mk.attn_paged(q, cache, table.t(), lens, cu, out, workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu[:1], out, workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu, out[:9], workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu, out.half(), workspace=ws),
                lambda: mk.attn_paged(q, cache, table, lens, cu, out, lse=torch.zeros(10, 2, device="cuda"),
                                      workspace=ws),
                lambda: mk.attn_packed(q, k, v[:9], cu, out, workspace=ws),
                lambda: mk.attn_packed(q, k, v, cu.cpu(), out, workspace=ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mk.MkError):  # too small
        mk.attn_packed(q, k, v, cu, out, workspace=ws[:4096])
    with pytest.raises(mk.MkError):
        mk.attn_paged(q[:, :7], cache, table, lens, cu, out[:, :7], workspace=ws)
    assert math.isfinite(float(out.float().nan_to_num().sum()))
