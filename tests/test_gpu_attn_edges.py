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
