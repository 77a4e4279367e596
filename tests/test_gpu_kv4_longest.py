"""Attention over the longest sequence that a call takes, 2^31 - 1024 keys, and over longer ones, which are cut to it:
nothing is looked up past the table, and the last keys are not lost.

The page table names pages of equal contents over and over and another page at its end, so that the reference is a
softmax over 32 keys with multiplicities.  Even heads look at the last page only: it outweighs the others by e^40 / 2^27.
The others weigh all keys.  Tolerance, with A = sum w |v|: 2^-10 A for weights in float16 and the result's rounding, A
2^-12 for scores (|s| under 50, 64 products) and exponentials, and for what lies on the pages that repeat, B of A, the
sums' chain: as many additions as a run has products of 16 keys, at most 2^27 / 152 and 2^-23 each (a tensor core's sums
are cut off, not rounded).
"""
import pytest

from tests import kv4_layout as layout
from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("news,heads,kind", [(1, 4, torch.float16), (1, 16, torch.bfloat16), (1, 32, torch.float16),
                                             (5, 32, torch.bfloat16)])
def test_the_longest_sequence(news, heads, kind):
    mmq = require_gpu()
    D, page, same = 64, 16, 4096
    keys = 2 ** 31 - 1024
    width, used = (2 ** 31 - 1) // page, keys // page   # the widest table
    g = torch.Generator(device="cuda").manual_seed(81)
    k, v = torch.randn((2, 32, 1, D), device="cuda", generator=g)
    k[..., :32] = 0
    k[16:, :, 0] = 8                         # the last page
    q = torch.randn((news, heads, D), device="cuda", generator=g)
    q[..., :32] = 0
    q[:, ::2, 0] = 40
    q = q.to(kind)
    cache = mmq.empty_kv4_cache(same + 1, 1, D, page)
    mmq.kv4_write(k[:16], v[:16], torch.arange(16, dtype=torch.int32, device="cuda"), cache)
    cache[1:same] = cache[0]
    mmq.kv4_write(k[16:], v[16:], torch.arange(16, dtype=torch.int32, device="cuda") + same * page, cache)
    table = torch.arange(width, dtype=torch.int32, device="cuda").remainder_(same).view(1, width)
    table[0, used - 1] = same
    lens = torch.tensor([keys], dtype=torch.int32, device="cuda")
    out = mmq.kv4_attention(q, cache, table, lens)
    assert mmq.status() == 0
    for more in (1, 1008, 1023):             # 1008: all of the table
        assert torch.equal(mmq.kv4_attention(q, cache, table, lens + more), out)
        assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
    got = out.double()
    slots = torch.cat([torch.arange(16, device="cuda"), torch.arange(16, device="cuda") + same * page])
    kd, vd = (x[:, 0] for x in layout.values(cache, slots))
    s = torch.einsum("jhd,nd->jhn", q.double(), kd) * D ** -0.5
    # token j sees all but the last news - 1 - j keys
    count = torch.cat([torch.full((news, 16), float(used - 1), dtype=torch.float64, device="cuda"),
                       (torch.arange(16, device="cuda") < 16 - (news - 1 - torch.arange(news, device="cuda"))[:, None]).double()], 1)
    e = torch.exp(s - s.amax(-1, keepdim=True)) * count[:, None]
    w = e / e.sum(-1, keepdim=True)
    A, B = w @ vd.abs(), w[..., :16] @ vd[:16].abs()
    tol = A * (2.0 ** -10 + 2.0 ** -12) + B * (2.0 ** 27 / 152 * 2.0 ** -23) + 2.0 ** -8 * (kind is torch.bfloat16) * (w @ vd).abs()
    off = (got - w @ vd).abs()
    assert (off <= tol).all(), float((off / tol).max())
    assert float(B[:, ::2].max()) < 1e-6     # the even heads' tolerance is that of their last page
