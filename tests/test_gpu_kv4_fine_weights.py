"""float32 results of the 4-bit attention have weights of 22 bits in every form that a sequence's rows may take, whatever
the other sequences of the batch.

Queries and keys are small integers and the scale a power of two, so that q.k is exact and what is left shows the weights.
Per output, with A = sum w |v| and scores |s| <= 16:
  2^-22 A       the weights as sums of two float16 values
  2^-24 sum |v| / l     and what both lose absolutely, against a largest weight of at least one
  2 E A, E = 2^-20 + 2^-20 + 2^-22     the base change of a score (23 x 2^-24), its difference from the reference (under
                32, half a unit 2^-20), the exponential
  28 x 2^-23 A  the sums over at most 160 keys, two products per 16, and the joins' factors
which is under (2^-22 + 2^-16.8) A; one float16 value alone would be off by up to 2^-12.
"""
import pytest

from tests import kv4_layout as layout
from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def make(mmq, news, lens, heads, kv, D, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    page, width = 16, -(-max(lens) // 16)
    table = torch.randperm(len(lens) * width, device="cuda", generator=g).view(len(lens), width).to(torch.int32)
    cache = mmq.empty_kv4_cache(len(lens) * width, kv, D, page).zero_()
    for b, n in enumerate(lens):
        i = torch.arange(n, device="cuda")
        k = torch.randint(-8, 8, (n, kv, D), device="cuda", generator=g).float()
        k[..., ::32] = -8     # each block's scale is one
        mmq.kv4_write(k, torch.randn(k.shape, device="cuda", generator=g),
                      (table[b, i // page].long() * page + i % page).to(torch.int32), cache)
    starts = torch.tensor([0] + news).cumsum(0).to(torch.int32).cuda()
    q = torch.randint(-1, 2, (sum(news), heads, D), device="cuda", generator=g).to(kind)
    q[..., ::32] = 0
    return dict(q=q, cache=cache, page_table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q_starts=starts)


def check(got, d, scale):
    q = d["q"].double()
    kv, heads = d["cache"].shape[1], q.shape[1]
    starts = d["q_starts"].tolist()
    for b, n in enumerate(d["lens"].tolist()):
        lo, hi = starts[b], starts[b + 1]
        i = torch.arange(n, device="cuda")
        k, v = layout.values(d["cache"], d["page_table"][b, i // 16] * 16 + i % 16)
        s = torch.einsum("jhgd,nhd->jhgn", q[lo:hi].view(hi - lo, kv, heads // kv, -1), k) * scale
        hidden = i >= (n - (hi - lo) + 1 + torch.arange(hi - lo, device="cuda"))[:, None, None, None]
        assert float(s.abs().max()) <= 16
        s = s.masked_fill(hidden, float("-inf"))
        e = torch.exp(s - s.amax(-1, keepdim=True))
        l = e.sum(-1, keepdim=True)
        mean = lambda w, x: (torch.einsum("jhgn,nhd->jhgd", w, x) / l).reshape(hi - lo, heads, -1)  # noqa: E731
        tol = mean(e, v.abs()) * (2.0 ** -22 + 2.0 ** -16.8) + mean((~hidden).double().expand_as(s), v.abs()) * 2.0 ** -24
        off = (got[lo:hi].double() - mean(e, v)).abs()
        assert (off <= tol).all(), (b, float((off / tol).max()))


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("news,lens,heads,kv,D", [
    ([1] * 5, [17, 90, 160, 33, 2], 8, 2, 128),                # units of eight rows
    ([2] * 9, [150 - 11 * i for i in range(9)], 16, 2, 64),    # of sixteen
    ([9] * 17, [9 + 8 * i for i in range(17)], 16, 4, 128),    # 128 rows, two streams
    ([30] * 400, [30 + i % 131 for i in range(400)], 1, 1, 64),
    ([70] * 20, [70 + 4 * i for i in range(20)], 8, 2, 128),   # 256 rows
    ([150], [160], 16, 4, 64),
    ([1, 60, 3, 150, 1], [160, 100, 64, 155, 1], 8, 2, 128),   # both kernels
    ([1, 60, 3, 1, 1, 1, 1, 1, 1, 1], [160, 100, 64] + [50] * 7, 8, 2, 64),
])
def test_float32_results(news, lens, heads, kv, D, kind):
    mmq = require_gpu()
    d = make(mmq, news, lens, heads, kv, D, kind, 71)
    out = torch.empty(d["q"].shape, device="cuda")
    for power in (2.0 ** -4, 2.0 ** -6):
        mmq.kv4_attention(d["q"], d["cache"], d["page_table"], d["lens"], q_starts=d["q_starts"], out=out, scale=power)
        assert mmq.status() == 0
        check(out, d, power)


def test_scores_past_the_usual_path():
    """Weights after the many-row form's border at 2^20: scores are exact there too (a sum of integers), spread over 0 to
    10 in steps of 1/8, with the scale whose product with log2(e) is one."""
    from tests.test_gpu_kv4_wide_scores import unit_scale
    mmq = require_gpu()
    scale, D, n, heads = unit_scale(), 128, 160, 64
    g = torch.Generator(device="cuda").manual_seed(73)
    k = torch.zeros((n, 1, D), device="cuda")
    k[:, 0, 0] = 1024
    k[:, 0, 32:64] = torch.randint(-8, 8, (n, 32), device="cuda", generator=g).float()
    k[:, 0, 32] = -8
    cache = mmq.empty_kv4_cache(10, 1, D, 16).zero_()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    mmq.kv4_write(k, torch.randn(k.shape, device="cuda", generator=g), slots, cache)
    q = torch.zeros((4, heads, D), dtype=torch.float16, device="cuda")
    q[:, ::2, 0] = 1536
    q[:, :, 33:64] = torch.randint(-1, 2, (4, heads, 31), device="cuda", generator=g).half() / 8
    table = torch.arange(10, dtype=torch.int32, device="cuda").view(1, 10)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for rows in (1, 4):        # 128 rows, 256
        out = torch.empty((rows, heads, D), device="cuda")
        mmq.kv4_attention(q[:rows], cache, table, lens, out=out, scale=scale)
        assert mmq.status() == 0
        kd, v = (x[:, 0] for x in layout.values(cache, slots))
        y = torch.einsum("jhd,nd->jhn", q[:rows].double(), kd)    # base two
        y = y.masked_fill(torch.arange(n, device="cuda") >= (n - rows + 1 + torch.arange(rows, device="cuda"))[:, None, None], float("-inf"))
        w = torch.exp2(y - y.amax(-1, keepdim=True))
        l = w.sum(-1, keepdim=True)
        A = w @ v.abs() / l
        tol = A * (2.0 ** -22 + 2.0 ** -16.8) + v.abs().sum(0) / l * 2.0 ** -24
        off = (out.double() - w @ v / l).abs()
        assert (off <= tol).all(), float((off / tol).max())
