"""GPU tests of mk_qk_norm_rope against the 64-bit formulas: every value within
half a step of its type plus the derived fp32 error of attention_ref.norm_rope.
"""
import pytest

import attention_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def mk():
    import attention_decode_megakernel_b200 as m
    from attention_decode_megakernel_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def _check(got, x, gain, pos, rope_args, inter, eps, what):
    turns, length = ref.rope_turns(**rope_args)
    want, tol = ref.norm_rope(x.cpu(), None if gain is None else gain.cpu(), pos.cpu(), turns,
                              length, inter, eps)
    t = got.dtype
    tol = tol + ref.half_step(t) * (want.abs() + tol)
    tol += torch.finfo(t).smallest_normal * torch.finfo(t).eps
    ref.check(got, want, tol, what)


def _rows(gen, n, heads, hd, dtype, spare=0):
    return torch.randn(n, heads + spare, hd, generator=gen, device="cuda").to(dtype)[:, :heads]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("hd,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 64)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hk,norm", [(1, 8, 2, True), (37, 5, 1, True), (3, 16, 0, False),
                                          (130, 1, 3, True)])
def test_norm_rope(mk, dtype, hd, rot, inter, n, hq, hk, norm):
    gen = torch.Generator(device="cuda").manual_seed(n * hd + rot)
    q, k = _rows(gen, n, hq, hd, dtype, 3), _rows(gen, n, hk, hd, dtype, 1) if hk else None
    pos = torch.randint(0, 5000, (n,), generator=gen, device="cuda", dtype=torch.int32)
    qg = (1 + torch.randn(hd, generator=gen, device="cuda") / 4).to(dtype) if norm else None
    kg = (1 + torch.randn(hd, generator=gen, device="cuda") / 4).to(dtype) if norm and n > 1 else None
    args = dict(rot=rot, theta=1e6, scaling="none")
    rope = mk.Rope(rot, 1e6, interleaved=inter)
    qo = torch.full((n + 1, hq, hd), 7.0, dtype=dtype, device="cuda")
    ko = torch.full((n + 1, max(hk, 1), hd), 7.0, dtype=dtype, device="cuda")
    q0 = q.clone()
    mk.qk_norm_rope(rope, q, k, pos, qo[:n], ko[:n] if hk else None, qg, kg, eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(q, q0) and bool((qo[n:] == 7).all()) and bool((ko[n:] == 7).all())
    _check(qo[:n], q, qg, pos, args, inter, 1e-5, "q")
    if hk:
        _check(ko[:n], k, kg, pos, args, inter, 1e-5, "k")
    # in place, through the strided views
    mk.qk_norm_rope(rope, q, k, pos, q_gain=qg, k_gain=kg, eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(q, qo[:n])
    if hk:
        assert torch.equal(k, ko[:n])


@pytest.mark.parametrize("scaling,given", [
    ("linear", dict(factor=4.0)), ("ntk", dict(factor=4.0)),
    ("yarn", dict(factor=4.0, original_ctx=32768, low=1.0, high=32.0)),
    ("banded", dict(factor=8.0, original_ctx=8192, low=1.0, high=4.0))])
def test_far_positions(mk, scaling, given):
    """Positions up to 2^31 - 1 and below zero, in fp32."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.tensor([0, 1, -1, -70000, 131071, (1 << 20) + 1, (1 << 24) + 1, (1 << 31) - 1],
                       dtype=torch.int32, device="cuda")
    q, k = _rows(gen, len(pos), 8, 128, F32), _rows(gen, len(pos), 2, 128, F32)
    rope = mk.Rope(128, 1e6, scaling=scaling, **given)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    mk.qk_norm_rope(rope, q, k, pos, qo, ko)
    torch.cuda.synchronize()
    # a position of 2^31 in turns has an error of 2^31 * 64 * 2^-53 in the tests' and the
    # operator's 64-bit frequencies alike: 2^-16 turns at most, which the last rows are given
    turns, length = ref.rope_turns(128, 1e6, scaling, **given)
    for got, x in ((qo, q), (ko, k)):
        want, tol = ref.norm_rope(x.cpu(), None, pos.cpu(), turns, length, False, 0.0)
        far = pos.cpu().double().abs()[:, None, None] * 2.0 ** -47 * 2 * 3.1416
        tol = tol + ref.U * want.abs() + far * (x.cpu().double().abs().amax() * 2)
        ref.check(got, want, tol, scaling)


def test_rotation_identity_norm_and_relative_positions(mk):
    """Position 0 changes nothing; lengths are kept; scores depend on the distance."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k = _rows(gen, 1, 1, 64, F32), _rows(gen, 1, 1, 64, F32)
    rope = mk.Rope(64, 1e4)
    scores = []
    for p in (0, 1000):
        a, b = q.clone(), k.clone()
        mk.qk_norm_rope(rope, a, None, torch.tensor([p + 17], dtype=torch.int32, device="cuda"))
        mk.qk_norm_rope(rope, b, None, torch.tensor([p], dtype=torch.int32, device="cuda"))
        if p == 0:
            assert torch.equal(b, k)
        assert abs(float(a.norm() / q.norm()) - 1) < 2.0 ** -20
        scores.append(float((a.double() * b.double()).sum()))
    assert abs(scores[0] - scores[1]) < 64 * 16 * ref.U * float(q.norm() * k.norm())


def test_zero_rows_infinities_and_nan(mk):
    """A row of zeros stays zero; an infinity or NaN spoils its own row alone."""
    x = torch.ones(4, 2, 128, dtype=BF, device="cuda")
    x[0, 0] = 0
    x[1, 0, 5] = float("inf")
    x[2, 1, 7] = float("nan")
    g = torch.ones(128, dtype=BF, device="cuda")
    out = torch.empty_like(x)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    mk.qk_norm_rope(mk.Rope(128, 1e4), x, None, pos, out, None, g)
    torch.cuda.synchronize()
    assert bool((out[0, 0] == 0).all())
    fine = torch.isfinite(out).all(-1).cpu()
    assert fine.tolist() == [[True, True], [False, True], [True, False], [True, True]]


def test_no_tokens(mk):
    x = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    mk.qk_norm_rope(mk.Rope(64, 1e4), x, None, torch.zeros(0, dtype=torch.int32, device="cuda"))
