"""The operators of an attention layer served over a paged key/value cache,
each in its plain form (elementary torch operations in 32 bits) and as the
framework's call, at sizes from one decoded token to long packed prompts.

    qk_norm_rope  RMSNorm of every query and key head, then the rotation by position
    kv_write      rows of keys and values into a paged cache, rounded to 8 bits where the cache holds 8 bits
    kv_read       those rows back, as the values they stand for
    attn_paged    attention of a chunk of new tokens (one, a few, many) over the paged cache
    attn_packed   causal attention of whole prompts of different lengths packed one after another

Cases are dicts of plain values; `lengths` turns a case into the same ragged
batch for everybody, so that `work` can count its bytes.  The head shapes
are the framework's own (8 query and 2 key heads of 256, 4 and 1 of 64) or
generic ones of 128.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
EPS = 1e-6


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one decoded token of the 0.8B shape: latency alone
        dict(name="norm_rope_1", op="qk_norm_rope", tokens=1, q_heads=8, kv_heads=2, head_dim=256,
             rot_dim=256, interleaved=False, scaling="none", theta=1e7, norm=True, dtype="bf16",
             far=600),
        # the 520-token prompt of the headline benchmark in the engine's fp32 activations
        dict(name="norm_rope_520_fp32", op="qk_norm_rope", tokens=520, q_heads=8, kv_heads=2,
             head_dim=256, rot_dim=256, interleaved=False, scaling="none", theta=1e7, norm=True,
             dtype="fp32", far=520),
        # a long prompt beyond the trained context: a quarter of the head rotated in
        # interleaved pairs, frequencies scaled
        dict(name="norm_rope_32768_yarn", op="qk_norm_rope", tokens=32768, q_heads=8, kv_heads=2,
             head_dim=256, rot_dim=64, interleaved=True, scaling="yarn", theta=1e7, norm=True,
             dtype="bf16", far=131072),
        # the new keys and values of 64 decoding sequences, each into a page of its own
        dict(name="kv_write_64", op="kv_write", tokens=64, pad=0, kv_heads=2, head_dim=256, page=16,
             scattered=True, dtype="bf16", cache="e4m3"),
        # a long prompt's keys and values, the last 5 rows of the batch padding
        dict(name="kv_write_32773", op="kv_write", tokens=32768, pad=5, kv_heads=2, head_dim=256,
             page=64, scattered=False, dtype="bf16", cache="e4m3"),
        # a cached prefix read back for a path that wants it whole
        dict(name="kv_read_32767", op="kv_read", tokens=32767, pad=0, kv_heads=2, head_dim=256,
             page=64, scattered=False, dtype="bf16", cache="e4m3"),
        # batch-1 decode behind the 520-token prompt: latency alone
        dict(name="paged_decode_520", op="attn_paged", batch=1, chunk=1, longest=520, ragged=False,
             pad=0, q_heads=8, kv_heads=2, head_dim=256, page=16, dtype="bf16", cache="bf16",
             lse=False),
        # a decoding batch of 64 sequences up to 4096 over an 8-bit cache
        dict(name="paged_decode_64x4096_e4m3", op="attn_paged", batch=64, chunk=1, longest=4096,
             ragged=True, pad=0, q_heads=8, kv_heads=2, head_dim=256, page=64, dtype="bf16",
             cache="e4m3", lse=False),
        # 5 draft tokens verified in 8 sequences, contexts up to 4096, a padded batch
        dict(name="paged_verify_8x5_4096", op="attn_paged", batch=8, chunk=5, longest=4096,
             ragged=True, pad=3, q_heads=8, kv_heads=2, head_dim=256, page=16, dtype="bf16",
             cache="bf16", lse=True),
        # the last 1024-token chunk of a 32768-token prompt
        dict(name="paged_chunk_1024_32768", op="attn_paged", batch=1, chunk=1024, longest=32768,
             ragged=False, pad=0, q_heads=8, kv_heads=2, head_dim=256, page=64, dtype="bf16",
             cache="bf16", lse=False),
        # the 520-token prompt of the headline benchmark
        dict(name="packed_520", op="attn_packed", batch=1, longest=520, ragged=False, pad=0,
             q_heads=8, kv_heads=2, head_dim=256, dtype="bf16", lse=False),
        # eight prompts of up to 4096 tokens packed into one batch
        dict(name="packed_8x4096", op="attn_packed", batch=8, longest=4096, ragged=True, pad=0,
             q_heads=16, kv_heads=4, head_dim=128, dtype="bf16", lse=False),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1e15


def draw(rng):
    """A case of the listed ranges: sizes spread over their logarithm, cut until
    the case costs no more than the largest listed case of its operator."""
    op = rng.choice(["qk_norm_rope", "kv_write", "kv_read", "attn_paged", "attn_paged",
                     "attn_packed"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    head_dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128, 256])
    pad = rng.choice([0, 0, rng.randint(1, 9)])
    if op == "qk_norm_rope":
        c = dict(op=op, tokens=_log_int(rng, 1, 32768), q_heads=q_heads, kv_heads=kv_heads,
                 head_dim=head_dim, rot_dim=rng.choice([head_dim, head_dim // 2, head_dim // 4]),
                 interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
                 theta=rng.choice([1e4, 5e5, 1e7]), norm=rng.random() < 0.75,
                 dtype=rng.choice(["bf16", "fp16", "fp32"]), far=_log_int(rng, 64, 1 << 20))
        cut = ("tokens",)
    elif op in ("kv_write", "kv_read"):
        c = dict(op=op, tokens=_log_int(rng, 1, 32768), pad=pad, kv_heads=kv_heads,
                 head_dim=head_dim, page=page, scattered=rng.random() < 0.5,
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), cache="e4m3")
        if rng.random() < 0.3:
            c["cache"] = c["dtype"] = dtype
        if op == "kv_read" and c["dtype"] == "fp16":
            c["dtype"] = "bf16" if c["cache"] == "e4m3" else "fp16"
        cut = ("tokens",)
    elif op == "attn_paged":
        c = dict(op=op, batch=_log_int(rng, 1, 64),
                 chunk=rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 1024)]),
                 longest=_log_int(rng, 1, 32768), ragged=rng.random() < 0.7, pad=pad,
                 q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype,
                 cache=rng.choice([dtype, dtype, "e4m3"]), lse=rng.random() < 0.5)
        c["chunk"] = min(c["chunk"], c["longest"])
        cut = ("longest", "batch", "chunk")
    else:
        c = dict(op=op, batch=_log_int(rng, 1, 64), longest=_log_int(rng, 1, 8192),
                 ragged=rng.random() < 0.7, pad=pad, q_heads=q_heads, kv_heads=kv_heads,
                 head_dim=head_dim, dtype=dtype, lse=rng.random() < 0.5)
        cut = ("batch", "longest")
    at = 0
    while _cost(c) > most or _padded(c) > 2.2e9:
        key = cut[at % len(cut)]
        c[key] = max(1, c[key] * 5 // 8)
        if key == "longest" and "chunk" in c:
            c["chunk"] = min(c["chunk"], c["longest"])
        at += 1
    return c


def _padded(case):
    """Values of the largest array that the plain form of an attention holds."""
    if case["op"] == "attn_paged":
        rows = case["q_heads"] * case["chunk"]
        return case["batch"] * case["longest"] * max(rows, case["kv_heads"] * case["head_dim"])
    if case["op"] == "attn_packed":
        return case["batch"] * case["longest"] * max(case["longest"] * case["q_heads"],
                                                     case["q_heads"] * case["head_dim"])
    return 0


def lengths(case):
    """(new tokens, all keys) of every sequence of the batch: the first one is
    the longest, the others between a quarter and all of it where the batch is
    ragged."""
    n, longest = case["batch"], case["longest"]
    chunk = case["chunk"] if case["op"] == "attn_paged" else longest
    rng = random.Random(1000003 * n + longest)
    keys = [longest] * n
    if case["ragged"]:
        keys = [longest] + [rng.randint(max(1, longest // 4), longest) for _ in range(n - 1)]
    if case["op"] == "attn_packed":
        return keys, keys
    new = [min(chunk, k) for k in keys]
    if case["ragged"]:
        new = new[:1] + [rng.randint(max(1, m // 2), m) for m in new[1:]]
    return new, keys


def work(case):
    if case["op"] == "qk_norm_rope":
        heads = case["q_heads"] + case["kv_heads"]
        values = case["tokens"] * heads * case["head_dim"]
        return {"bytes": 2 * values * SIZE[case["dtype"]] + 4 * case["tokens"],
                "flops": 4 * values * bool(case["norm"])
                + 3 * case["tokens"] * heads * case["rot_dim"]}
    if case["op"] in ("kv_write", "kv_read"):
        rows = 2 * case["tokens"] * case["kv_heads"]
        scale = 4 * rows if case["cache"] == "e4m3" else 0
        return {"bytes": rows * case["head_dim"] * (SIZE[case["dtype"]] + SIZE[case["cache"]])
                + scale + 8 * (case["tokens"] + case["pad"]),
                "flops": 2 * rows * case["head_dim"]}
    new, keys = lengths(case)
    cache = case.get("cache", case["dtype"])
    row = case["head_dim"] * SIZE[cache] + (4 if cache == "e4m3" else 0)
    pairs = sum(t * k - t * (t - 1) // 2 for t, k in zip(new, keys))
    moved = 2 * sum(keys) * case["kv_heads"] * row
    moved += sum(new) * case["q_heads"] * (2 * case["head_dim"] * SIZE[case["dtype"]]
                                           + 4 * bool(case["lse"]))
    return {"bytes": moved, "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}


# ---- inputs -----------------------------------------------------------------

def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda", generator=gen).to(dtype)


def _pool(case, gen, pages, filled):
    """A paged cache of `pages` pages: [page][head][position][dim]."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    kind = DTYPES[case["cache"]]
    pool = {"k": torch.zeros(shape, dtype=kind, device="cuda"),
            "v": torch.zeros(shape, dtype=kind, device="cuda"), "k_scale": None, "v_scale": None}
    if case["cache"] == "e4m3":
        pool["k_scale"] = torch.ones(shape[:3], device="cuda")
        pool["v_scale"] = torch.ones(shape[:3], device="cuda")
    if filled:
        for name in ("k", "v"):
            rows = _normal(gen, *shape)
            if case["cache"] == "e4m3":  # rows of differing size, as written by kv_write
                rows *= torch.exp(0.5 * _normal(gen, *shape[:3], 1))
                rows, pool[name + "_scale"] = _to_e4m3(rows)
            pool[name] = rows.to(kind)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = DTYPES[case["dtype"]]
    s = {"case": case}
    hk, hd = case["kv_heads"], case["head_dim"]
    if case["op"] == "qk_norm_rope":
        # queries and keys lie in one projection's rows [q | k | v]
        hq, n = case["q_heads"], case["tokens"]
        rows = _normal(gen, n, hq + 2 * hk, hd, dtype=kind)
        s["q"], s["k"] = rows[:, :hq], rows[:, hq:hq + hk]
        s["q_gain"] = s["k_gain"] = None
        if case["norm"]:
            s["q_gain"] = (1 + 0.1 * _normal(gen, hd)).to(kind)
            s["k_gain"] = (1 + 0.1 * _normal(gen, hd)).to(kind)
        first = torch.randint(0, max(1, case["far"] - n + 1), (1,), device="cuda", generator=gen)
        s["positions"] = (first + torch.arange(n, device="cuda")).to(torch.int32)
        s["q_out"] = torch.zeros(n, hq, hd, dtype=kind, device="cuda")
        s["k_out"] = torch.zeros(n, hk, hd, dtype=kind, device="cuda")
        if own:
            import attention_decode_megakernel_b200 as mk
            s["rope"] = mk.Rope(case["rot_dim"], case["theta"], interleaved=case["interleaved"],
                                scaling=case["scaling"], **_scaling(case))
        return s
    if case["op"] in ("kv_write", "kv_read"):
        n, pad, page = case["tokens"], case["pad"], case["page"]
        used = n if case["scattered"] else -(-n // page)
        pages = used + used // 8 + 1
        order = torch.randperm(pages, device="cuda", generator=gen)[:used]
        if case["scattered"]:
            slots = order * page + torch.randint(0, page, (n,), device="cuda", generator=gen)
        else:
            at = torch.arange(n, device="cuda")
            slots = order[at // page] * page + at % page
        s["slots"] = torch.cat([slots, slots.new_full((pad,), -1)])
        s["valid"] = n
        s["pool"] = _pool(case, gen, pages, case["op"] == "kv_read")
        if case["op"] == "kv_write":
            rows = _normal(gen, n + pad, 2 * hk, hd, dtype=kind)
            s["k"], s["v"] = rows[:, :hk], rows[:, hk:]
        else:
            s["k_out"] = torch.zeros(n + pad, hk, hd, dtype=kind, device="cuda")
            s["v_out"] = torch.zeros(n + pad, hk, hd, dtype=kind, device="cuda")
    else:
        new, keys = lengths(case)
        hq, total = case["q_heads"], sum(new)
        starts = [0]
        for t in new:
            starts.append(starts[-1] + t)
        s["cu_q"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["total"], s["most_new"], s["most_keys"] = total, max(new), max(keys)
        s["out"] = torch.zeros(total + case["pad"], hq, hd, dtype=kind, device="cuda")
        s["lse"] = torch.zeros(total + case["pad"], hq, device="cuda") if case["lse"] else None
        if case["op"] == "attn_packed":
            rows = _normal(gen, total + case["pad"], hq + 2 * hk, hd, dtype=kind)
            s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
        else:
            s["q"] = _normal(gen, total + case["pad"], hq, hd, dtype=kind)
            page = case["page"]
            need = [-(-k // page) for k in keys]
            pages = sum(need) + 1
            s["pool"] = _pool(case, gen, pages, True)
            order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
            table = torch.zeros(len(keys), max(need), dtype=torch.int32, device="cuda")
            used = 0
            for b, m in enumerate(need):
                table[b, :m] = order[used:used + m]
                used += m
            s["table"] = table
            s["seq_lens"] = torch.tensor(keys, dtype=torch.int32, device="cuda")
    if own:
        import attention_decode_megakernel_b200 as mk
        if "pool" in s:
            s["cache"] = mk.KvCache(s["pool"]["k"], s["pool"]["v"], s["pool"]["k_scale"],
                                    s["pool"]["v_scale"])
        if case["op"] in ("attn_paged", "attn_packed"):
            s["workspace"] = mk.attn_workspace(hd)
    return s


def _scaling(case):
    """The parameters of a case's frequency scaling: four times the trained context."""
    if case["scaling"] == "none":
        return {}
    given = {"factor": 4.0}
    if case["scaling"] == "yarn":
        given.update(original_ctx=32768, low=1.0, high=32.0)
    if case["scaling"] == "banded":
        given.update(original_ctx=8192, low=1.0, high=4.0)
    return given


# ---- one pass ---------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "qk_norm_rope":
        cos, sin = _angles(case, s["positions"])
        for name in ("q", "k"):
            s[name + "_out"].copy_(_norm_rope(s[name].float(), s[name + "_gain"], cos, sin, case))
        return s["q_out"], s["k_out"]
    if case["op"] == "kv_write":
        _write(s, case)
        return {name: x for name, x in s["pool"].items() if x is not None}
    if case["op"] == "kv_read":
        page = case["page"]
        slots = s["slots"][:s["valid"]]
        for name in ("k", "v"):
            rows = _bytes(s["pool"][name])[slots // page, :, slots % page]
            rows = rows.view(s["pool"][name].dtype).float()
            if case["cache"] == "e4m3":
                rows = rows * s["pool"][name + "_scale"][slots // page, :, slots % page, None]
            s[name + "_out"][:s["valid"]] = rows.to(s[name + "_out"].dtype)
        return s["k_out"], s["v_out"]
    if case["op"] == "attn_paged":
        kf, vf = (_gather(s, case, name) for name in ("k", "v"))
        lens = s["seq_lens"].long()
    else:
        at = _padded_rows(s, s["most_keys"])
        kf, vf = (s[name][at].float().transpose(1, 2) for name in ("k", "v"))
        lens = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    return _attend(s, case, kf, vf, lens)


def _run_own(s, case):
    import attention_decode_megakernel_b200 as mk
    if case["op"] == "qk_norm_rope":
        mk.qk_norm_rope(s["rope"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"],
                        q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS)
        return s["q_out"], s["k_out"]
    if case["op"] == "kv_write":
        mk.kv_write(s["cache"], s["k"], s["v"], s["slots"])
        return {name: x for name, x in s["pool"].items() if x is not None}
    if case["op"] == "kv_read":
        mk.kv_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if case["op"] == "attn_paged":
        mk.attn_paged(s["q"], s["cache"], s["table"], s["seq_lens"], s["cu_q"], s["out"],
                      lse=s["lse"], workspace=s["workspace"])
    else:
        mk.attn_packed(s["q"], s["k"], s["v"], s["cu_q"], s["out"], lse=s["lse"],
                       workspace=s["workspace"])
    return (s["out"], s["lse"]) if case["lse"] else s["out"]


def _frequencies(case):
    """Radians per position of every rotated pair, in 64 bits."""
    rot, theta, kind = case["rot_dim"], case["theta"], case["scaling"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    p = _scaling(case)
    if kind == "ntk":
        theta = theta * p["factor"] ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if kind == "linear":
        f = f / p["factor"]
    elif kind == "yarn":
        # pairs that turn more than `high` times over the trained context stay,
        # those that turn less than `low` times are slowed, a ramp between
        def pair(turns):
            return rot * math.log(p["original_ctx"] / (2 * math.pi * turns)) / (2 * math.log(theta))
        first = max(math.floor(pair(p["high"])), 0)
        last = min(math.ceil(pair(p["low"])), rot - 1)
        ramp = ((i - first) / max(last - first, 1e-3)).clamp(0, 1)
        f = f / p["factor"] * ramp + f * (1 - ramp)
    elif kind == "banded":
        turns = p["original_ctx"] * f / (2 * math.pi)
        keep = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = f / p["factor"] * (1 - keep) + f * keep
    return f


def _angles(case, positions):
    angle = positions.double()[:, None] * _frequencies(case)
    size = 0.1 * math.log(_scaling(case)["factor"]) + 1 if case["scaling"] == "yarn" else 1.0
    return (torch.cos(angle) * size).float()[:, None], (torch.sin(angle) * size).float()[:, None]


def _norm_rope(x, gain, cos, sin, case):
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    rot = case["rot_dim"]
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _to_e4m3(x):
    """x (32 bits) as e4m3 values and one power of two for each row: the least
    that brings the row's largest magnitude to 448 or below, and 2^-64 at least."""
    mantissa, exponent = torch.frexp(x.abs().amax(-1))
    exponent = torch.where(mantissa > 0.875, exponent - 8, exponent - 9)
    scale = torch.ldexp(torch.ones_like(mantissa), exponent.clamp(min=-64))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _bytes(x):
    """e4m3 values as bytes, for indexing."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _write(s, case):
    slots = s["slots"][:s["valid"]]
    page, off = slots // case["page"], slots % case["page"]
    for name in ("k", "v"):
        rows = s[name][:s["valid"]]
        if case["cache"] == "e4m3":
            rows, scale = _to_e4m3(rows.float())
            s["pool"][name + "_scale"][page, :, off] = scale
        _bytes(s["pool"][name])[page, :, off] = _bytes(rows)


def _gather(s, case, name):
    """Every sequence's pages as [sequence][head][position][dim], 32 bits."""
    pages = s["table"].long()
    x = _bytes(s["pool"][name])[pages].view(s["pool"][name].dtype).float()
    if case["cache"] == "e4m3":
        x = x * s["pool"][name + "_scale"][pages][..., None]
    b, n, h, page, hd = x.shape
    return x.transpose(1, 2).reshape(b, h, n * page, hd)


def _padded_rows(s, most):
    at = s["cu_q"][:-1, None].long() + torch.arange(most, device="cuda")
    return at.clamp(max=s["total"] - 1)


def _attend(s, case, kf, vf, lens):
    batch, hk, n, hd = kf.shape
    group, most = case["q_heads"] // hk, s["most_new"]
    new = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    qf = s["q"][_padded_rows(s, most)].float()
    qf = qf.view(batch, most, hk, group, hd).permute(0, 2, 3, 1, 4).reshape(batch, hk, -1, hd)
    x = torch.matmul(qf, kf.transpose(2, 3)).mul_(hd ** -0.5)
    at = torch.arange(most, device="cuda")
    last = (lens - new)[:, None] + at  # the last position that each row sees
    hidden = torch.arange(n, device="cuda") > last[..., None]
    x = x.view(batch, hk, group, most, n).masked_fill_(hidden[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(batch, hk, group * most, n), vf).view(batch, hk, group, most, hd)
    o = torch.where(total > 0, o / total, 0.0)
    # back to packed rows
    row = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["cu_q"][1:].contiguous(), row.int(), right=True)
    t = row - s["cu_q"][seq]
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, most, case["q_heads"], hd)
    s["out"][:s["total"]] = o[seq, t].to(s["out"].dtype)
    if not case["lse"]:
        return s["out"]
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(batch, most, -1)
    s["lse"][:s["total"]] = lse[seq, t]
    return s["out"], s["lse"]


# ---- the same in 64 bits ----------------------------------------------------

def _exact_turns(case):
    """Radians per position of each pair, and the length of the rotation, pair by pair."""
    rot, theta, kind, speeds = case["rot_dim"], case["theta"], case["scaling"], []
    factor = 1.0 if kind == "none" else 4.0
    for i in range(rot // 2):
        base = theta if kind != "ntk" else theta * math.pow(factor, rot / (rot - 2))
        f = math.exp(-2 * i / rot * math.log(base))
        wave = 2 * math.pi / f  # positions for one whole turn
        if kind == "linear":
            f /= factor
        elif kind == "yarn":
            ends = [rot / 2 * math.log(32768 / (turns * 2 * math.pi), theta) for turns in (32, 1)]
            first, last = max(0, math.floor(ends[0])), min(rot - 1, math.ceil(ends[1]))
            slow = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
            f = slow * (f / factor) + (1 - slow) * f
        elif kind == "banded" and wave > 8192:
            f /= factor
        elif kind == "banded" and wave > 8192 / 4:
            keep = (8192 / wave - 1) / (4 - 1)
            f = (1 - keep) * f / factor + keep * f
        speeds.append(f)
    size = 1 + 0.1 * math.log(factor) if kind == "yarn" else 1.0
    return torch.tensor(speeds, dtype=torch.float64, device="cuda"), size


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk_norm_rope":
        rot = case["rot_dim"]
        speeds, size = _exact_turns(case)
        turn = torch.polar(torch.full((1, 1), size, dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None] * speeds)
        outs = []
        for name in ("q", "k"):
            x = s[name].double()
            if case["norm"]:
                x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
                                   / case["head_dim"] + EPS) * s[name + "_gain"].double()
            pairs = x[..., :rot]
            shape = (-1, 2) if case["interleaved"] else (2, -1)
            pairs = pairs.unflatten(-1, shape)
            if not case["interleaved"]:
                pairs = pairs.transpose(-1, -2)
            z = torch.view_as_complex(pairs.contiguous()) * turn[:, None]
            z = torch.view_as_real(z)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            outs.append(torch.cat([z.flatten(-2), x[..., rot:]], -1))
        return tuple(outs)
    if case["op"] == "kv_write":
        pool = {name: x.double() for name, x in s["pool"].items() if x is not None}
        where = s["slots"][:s["valid"]]
        for name in ("k", "v"):
            x = s[name][:s["valid"]].double()
            if case["cache"] == "e4m3":
                part, power = torch.frexp(x.abs().amax(-1) / 448)
                power = torch.where(part == 0.5, power - 1, power).clamp(min=-64)
                scale = torch.ldexp(torch.ones_like(part), power)
                y = x / scale[..., None]
                power = torch.frexp(y)[1].clamp(min=-5) - 4  # of the last bit kept
                x = torch.ldexp(torch.round(torch.ldexp(y, -power)), power)
                flat = pool[name + "_scale"].transpose(1, 2).reshape(-1, case["kv_heads"])
                flat[where] = scale
                pool[name + "_scale"] = flat.view(-1, case["page"], case["kv_heads"]).transpose(1, 2)
            flat = pool[name].transpose(1, 2).reshape(-1, case["kv_heads"], case["head_dim"])
            flat[where] = x
            pool[name] = flat.view(-1, case["page"], *flat.shape[1:]).transpose(1, 2)
        return pool
    if case["op"] == "kv_read":
        outs = []
        for name in ("k", "v"):
            x = s["pool"][name].double()
            if case["cache"] == "e4m3":
                x = x * s["pool"][name + "_scale"].double()[..., None]
            x = x.transpose(1, 2).reshape(-1, case["kv_heads"], case["head_dim"])
            o = s[name + "_out"].double()
            o[:s["valid"]] = x[s["slots"][:s["valid"]]]
            outs.append(o)
        return tuple(outs)
    new, keys = lengths(case)
    out = s["out"].double()
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    group, first = case["q_heads"] // case["kv_heads"], 0
    for b, (t, n) in enumerate(zip(new, keys)):
        below = torch.ones(t, n, dtype=torch.bool, device="cuda").tril(n - t)
        for h in range(case["kv_heads"]):
            if case["op"] == "attn_packed":
                k, v = (s[name][first:first + n, h].double() for name in ("k", "v"))
            else:
                pages = s["table"][b, :-(-n // case["page"])].long()
                k, v = (s["pool"][name][pages.tolist(), h] if case["cache"] != "e4m3" else
                        s["pool"][name].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn)
                        for name in ("k", "v"))
                k, v = k.double(), v.double()
                if case["cache"] == "e4m3":
                    k = k * s["pool"]["k_scale"][pages, h].double()[..., None]
                    v = v * s["pool"]["v_scale"][pages, h].double()[..., None]
                k, v = k.flatten(0, 1)[:n], v.flatten(0, 1)[:n]
            for g in range(h * group, (h + 1) * group):
                x = s["q"][first:first + t, g].double() @ k.T / math.sqrt(case["head_dim"])
                x = x.masked_fill(~below, -math.inf)
                lse[first:first + t, g] = torch.logsumexp(x, -1)
                out[first:first + t, g] = torch.softmax(x, -1) @ v
        first += t
    return (out, lse) if case["lse"] else out
