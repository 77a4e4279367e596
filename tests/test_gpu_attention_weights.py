"""Shared-prefix attention where one key outweighs a long tail: the tail's
share of the result must not get lost in the rounding of its weights.

One key scores 17.5 above n others, whose values are 1 and its own 0, so that
every output is n e / (1 + n e), e = exp(-17.5) = 2^-25.2.  Tolerance, relative
to that: 2^-11 for the weights' rounding to float16 (2^-8 to bfloat16), (n / 16
+ 64) 2^-23 for the sums over keys, 2^-19 for exponentials and joins, and twice
the error of a score, 64 2^-23 17.5; and 2^-32 n absolute, for weights that
float16 holds below its normal range.  (The scores themselves are exact here.)
"""
import math

import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KIND = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("place", [0, 700, 1500])
@pytest.mark.parametrize("where,batch,heads,kv,D,keys", [
    ("prefix", 1, 1, 1, 64, 2049),         # few rows: one row tile
    ("prefix", 64, 32, 8, 128, 16385),     # two row tiles
    ("suffix", 1, 1, 1, 64, 4097),
    ("suffix", 9, 8, 8, 128, 4097),
])
def test_tail_under_one_large_key(where, batch, heads, kv, D, keys, place, kind):
    mmq = require_gpu()
    dt, page = KIND[kind], 64
    q = torch.zeros((batch, heads, D), dtype=dt, device="cuda")
    q[..., 0] = 1
    width = -(-keys // page) if where == "suffix" else 1
    prefix = keys if where == "prefix" else 0
    k_prefix, v_prefix = (torch.full((prefix, kv, D), v, dtype=dt, device="cuda") for v in (0.0, 1.0))
    k_cache, v_cache = (torch.full((batch * width, page, kv, D), v, dtype=dt, device="cuda") for v in (0.0, 1.0))
    table = torch.arange(batch * width, device="cuda", dtype=torch.int32).view(batch, width)
    lens = torch.full((batch,), 0 if prefix else keys, dtype=torch.int32, device="cuda")
    if prefix:
        k_prefix[place, :, 0] = 17.5
        v_prefix[place] = 0
    else:
        k_cache[table[:, place // page].long(), place % page, :, 0] = 17.5
        v_cache[table[:, place // page].long(), place % page] = 0
    out = torch.empty((batch, heads, D), device="cuda")
    mmq.shared_prefix_attention(q, k_prefix, v_prefix, k_cache, v_cache, table, lens, scale=1.0, out=out)
    assert mmq.status() == 0
    n = keys - 1
    tail = n * math.exp(-17.5)
    want = tail / (1 + tail)
    tol = want * ((2.0 ** -11 if kind == "f16" else 2.0 ** -8) + (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -19
                  + 2 * 64 * 2.0 ** -23 * 17.5) + (n * 2.0 ** -32 if kind == "f16" else 0.0)
    off = float((out.double() - want).abs().max())
    assert off <= tol, (off, tol, want)
