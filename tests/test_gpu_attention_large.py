"""Shared-prefix attention with scores so large that their units in the last
place matter: finite inputs give finite results, and the right ones.

A score is a b (one product, exact in f32), or a b + c with a b near 2^20 /
log2(e) and small c.  In the first kind scores differ by thousands or not at
all, so the result is the mean of the values whose keys tie for the largest
(the weights of those are equal: 2^-11 / 2^-8 for their rounding, 2^-18 for sums
and joins).  In the second the score in units of log2 is rounded to 2^-3, so
each weight is off by up to 2^(2^-4), 4.5 %, either way, and a result by up to
twice that of the mean of |v|, plus the weights' rounding.
"""
import math

import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KIND = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def attend(mmq, batch, heads, kv, D, kind, q0, keys, where):
    """(out, v in 64 bits): every row has the query q0 (two values, then zeros), every head the same keys [n][2]."""
    dt, page, n = KIND[kind], 16, keys.shape[0]
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.zeros((batch, heads, D), device="cuda", dtype=dt)
    q[..., :2] = torch.tensor(q0, device="cuda").to(dt)
    k = torch.zeros((n, kv, D), device="cuda", dtype=dt)
    k[..., :2] = keys.to(dt)[:, None]
    assert torch.equal(k[:, 0, :2].double(), keys.double().cuda())     # exact in the type
    v = torch.randn((n, kv, D), device="cuda", generator=g).to(dt)
    empty = torch.zeros((0, kv, D), device="cuda", dtype=dt)
    width = -(-n // page)
    if where == "prefix":
        kp, vp, kc, vc = k, v, empty.view(0, page, kv, D), empty.view(0, page, kv, D)
        table = torch.zeros((batch, 0), dtype=torch.int32, device="cuda")
        lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    else:
        kp, vp = empty, empty
        kc, vc = (torch.zeros((width * page, kv, D), device="cuda", dtype=dt) for _ in range(2))
        kc[:n], vc[:n] = k, v
        kc, vc = kc.view(width, page, kv, D), vc.view(width, page, kv, D)
        table = torch.arange(width, dtype=torch.int32, device="cuda").expand(batch, width).contiguous()
        lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out = torch.empty((batch, heads, D), device="cuda")
    mmq.shared_prefix_attention(q, kp, vp, kc, vc, table, lens, scale=1.0, out=out)
    assert mmq.status() == mmq.MMQ_OK
    return out.double(), v.double()


def compare(out, v, score, slack, kv):
    w = torch.softmax(score.cuda(), 0)
    want, mag = (torch.einsum("n,nhd->hd", w, x) for x in (v, v.abs()))
    got = out.view(out.shape[0], kv, -1, out.shape[-1])
    assert torch.isfinite(got).all()
    off = (got - want[None, :, None]).abs()
    assert (off <= slack * mag[None, :, None]).all(), float((off / mag[None, :, None]).max())


SHAPES = pytest.mark.parametrize("where,batch,heads,kv,D", [
    ("prefix", 2, 4, 2, 64), ("prefix", 40, 8, 4, 128), ("suffix", 3, 8, 2, 128), ("suffix", 2, 4, 4, 64)])


@SHAPES
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("a", [2.0 ** k for k in (3, 5, 8, 9, 11, 12, 13, 14, 15)])
def test_the_largest_scores_take_all(where, batch, heads, kv, D, kind, sign, a):
    mmq = require_gpu()
    g = torch.Generator().manual_seed(int(a))
    step = 32.0 if kind == "f16" else 256.0
    b = 33024.0 + step * torch.randint(0, 60, (700,), generator=g)
    for order in (b, b.sort().values, b.sort(descending=True).values):
        keys = torch.stack([sign * order, torch.zeros(700)], 1)
        out, v = attend(mmq, batch, heads, kv, D, kind, (a, 0.0), keys, where)
        compare(out, v, a * keys[:, 0].double(), UNIT[kind] + 2.0 ** -18, kv)


@SHAPES
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_cross_the_limit(where, batch, heads, kv, D, sign):
    """Scores in units of log2 that rise from 9 under sign 2^20 to 4 over it."""
    mmq = require_gpu()
    at = sign * 2.0 ** 20 / math.log2(math.e)
    b = 32.0 * round((at - sign * 290) / 16 / 32)
    c = torch.round((at - 16 * b - 6 + 9 * torch.arange(700) / 700) * 4) / 4
    keys = torch.stack([torch.full((700,), b), c], 1)
    out, v = attend(mmq, batch, heads, kv, D, "f16", (16.0, 1.0), keys, where)
    compare(out, v, (16 * b + c).double(), 2 * (2.0 ** 2.0 ** -4 - 1) + 2.0 ** -11 + 2.0 ** -18, kv)
