"""The operators of an attention layer over a paged cache in 64 bits, one row
at a time, on the CPU, with the error that a kernel of 32-bit sums may make.

`attend` also returns a bound for every output value, derived from the
operation's own roundings (u = 2^-24):
* a score is a sum of hd products and is off by at most d = 2 (hd + 4) u B with
  B = scale * sum |q_i k_i| (twice the textbook hd u, for matrix units that
  cut instead of rounding), and its exponent by 2^-21 more for the
  exponential itself;
* every weight p is rounded once to the values' type (eps / 2 relative; an
  e4m3 cache's values are multiplied as fp16), and so is the output;
* numerator and denominator each carry d and 1000 u for sums and rescaling.
* fp16 weights are 2^7 or more at the largest, and below 2^-14 they are rounded
  to steps of 2^-24: each is off by up to 2^-25, in numbers whose sum is 2^7 or
  more.  Weights that carry the scale s of an e4m3 row multiply codes v / s: the sum
  of weights then is 2^7 / s or more at the row of the largest one.
With A = sum p |v| / sum p the output is off by at most
  eps_out / 2 |o| + A (eps_w / 2 + 2 (d + 2^-21 + 1000 u))
  + (fp16 weights) 2^-32 sum |v / s| max s over the row's keys,
and lse by d + 2^-21 + 1000 u + 4 u |lse|.
"""
import math

import torch

U = 2.0 ** -24


def rope_turns(rot, theta, scaling="none", factor=1.0, original_ctx=0.0, low=1.0, high=32.0):
    """(turns per position of every pair, length) by the formulas, pair by pair."""
    out = []
    base = theta * factor ** (rot / (rot - 2)) if scaling == "ntk" else theta
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        turns = original_ctx * f / (2 * math.pi)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            at = [rot * math.log(original_ctx / (2 * math.pi * n)) / (2 * math.log(theta))
                  for n in (high, low)]
            a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            ramp = min(max((i - a) / max(b - a, 1e-3), 0.0), 1.0)
            f = f / factor * ramp + f * (1 - ramp)
        elif scaling == "banded":
            if turns <= low:
                f /= factor
            elif turns < high:
                keep = (turns - low) / (high - low)
                f = f / factor * (1 - keep) + f * keep
        out.append(f / (2 * math.pi))
    return out, 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


def norm_rope(x, gain, positions, turns, length, interleaved, eps):
    """x [tokens][heads][dim] (any type) -> (y, bound) in 64 bits."""
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.double()
    rot = 2 * len(turns)
    angle = positions.double()[:, None, None] * torch.tensor(turns, dtype=torch.float64)
    angle = 2 * math.pi * (angle - torch.floor(angle))
    c, s = torch.cos(angle) * length, torch.sin(angle) * length
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    y, size = x.clone(), x.abs()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    both = (x[..., ia].abs() + x[..., ib].abs()) * length
    size[..., ia] = both
    size[..., ib] = both
    # sums of 256 squares, root, divide, sine and cosine in fp32: 16 u together
    return y, 16 * U * size


def to_e4m3(x):
    """(values, scales) of rows x [..., dim]: the least power of two, 2^-64 at
    least, that brings the largest magnitude to 448 or below; values in steps."""
    x = x.double()
    part, power = torch.frexp(x.abs().amax(-1) / 448)
    power = torch.where(part == 0.5, power - 1, power).clamp(min=-64)
    power = torch.where(x.abs().amax(-1) == 0, torch.full_like(power, -64), power)
    y = torch.ldexp(x, -power[..., None])
    step = torch.frexp(y)[1].clamp(min=-5) - 4
    return torch.ldexp(torch.round(torch.ldexp(y, -step)), step), torch.ldexp(
        torch.ones_like(part), power)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attend(q, k, v, seen, scale, out_type, weight_type, v_scale=None):
    """One sequence: q [T][hq][hd], k, v [n][hk][hd] (64 bits), row t sees the
    keys 0 .. seen[t] - 1; v_scale [n][hk] of an e4m3 cache.  Returns (out, lse,
    out's bound, lse's bound)."""
    T, hq, hd = q.shape
    n, hk = k.shape[0], k.shape[1]
    g = hq // hk
    out, tol = torch.zeros(T, hq, hd, dtype=torch.float64), torch.zeros(T, hq, hd,
                                                                         dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros(T, hq, dtype=torch.float64)
    hidden = torch.arange(n)[None, :] >= torch.as_tensor(seen)[:, None]
    some = torch.as_tensor(seen) > 0
    if n == 0 or not bool(some.any()):
        return out, lse, tol, ltol
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        x = (q[:, h] @ kh.T) * scale
        size = (q[:, h].abs() @ kh.abs().T) * scale
        d = 2 * (hd + 4) * U * size.masked_fill(hidden, 0).amax(-1) + 2.0 ** -21 + 1000 * U
        x = x.masked_fill(hidden, -math.inf)
        le = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(some, le, 0.0)[:, None])
        o = p @ vh
        a = p @ vh.abs()
        out[:, h] = torch.where(some[:, None], o, 0.0)
        tol[:, h] = half_step(out_type) * o.abs() + a * (half_step(weight_type) + 2 * d[:, None])
        if weight_type == torch.float16:
            s = torch.ones(n, dtype=torch.float64) if v_scale is None else v_scale[:, h // g].double()
            top = s[None].expand(T, n).masked_fill(hidden, 0).amax(-1)
            tol[:, h] += 2.0 ** -32 * top[:, None] * ((~hidden).double() @ (vh.abs() / s[:, None]))
        # results below the type's normal range are rounded to its smallest step
        tol[:, h] += torch.finfo(out_type).smallest_normal * torch.finfo(out_type).eps
        lse[:, h] = le
        ltol[:, h] = d + 4 * U * le.abs().nan_to_num(posinf=0.0)
    return out, lse, tol, ltol


def check(got, want, tol, what):
    got = got.detach().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN"
    off = (got - want).abs()
    off = torch.where(got == want, 0.0, off)  # infinities
    bad = ~(off <= tol)
    assert not bool(bad.any()), "%s: %d values off, worst %.3g against a bound of %.3g" % (
        what, int(bad.sum()), float(off[bad].max()), float(tol[bad].min()))
