"""Scores on either side of 2^20 (in log2), where the many-row form of the 4-bit attention takes another path.

A row of scores just under 2^20 goes a little over it in a step in which another row of the same warp rises by much, and
a third row later takes the warp to the other path.  All products, sums and scores are exact in float32: keys and
queries are powers of two, and the scale is the float32 number whose product with log2(e) is one.  So weights are powers
of two but for the exponential's 2^-22 or so, each exact in float16, and a result is off by its rounding and, for the
exponentials and the sums of up to 320 keys, by 2^-14 of A = sum w |v| at most.
"""
import math

import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_kv4_attention import reference

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def unit_scale():
    """A float32 scale whose product with log2(e) rounds to one, in float32."""
    for steps in range(-4, 5):
        x = torch.tensor(math.log(2.0)).view(torch.int32) + steps
        if float(x.view(torch.float32) * torch.tensor(LOG2E)) == 1.0:
            return float(x.view(torch.float32))
    raise AssertionError("no such scale")


def make(mmq, n_seq, new, n_keys, change, huge):
    """n_seq sequences alike.  Row 0 of a token has scores of 2^20 - 2 for keys under `change` and 2^20 + 2 from there on,
    row 1 rises by 20 there, row 2 by 2^21 from key `huge` on; the other rows' scores are zeros."""
    D, page, heads = 128, 64, 32
    q = torch.zeros((n_seq * new, heads, D), dtype=torch.float16, device="cuda")
    k = torch.zeros((n_keys, 1, D), device="cuda")
    k[:, 0, 0], k[:, 0, 32] = 1024, 1
    q[:, 0, 0], q[:, 0, 32] = 1024, -2
    k[change:, 0, 64] = 1
    q[:, 0, 64], q[:, 1, 64] = 4, 20
    k[huge:, 0, 96] = 64
    q[:, 2, 96] = 32768
    v = torch.ones((n_keys, 1, D), device="cuda")
    v[huge:] = -1
    width = -(-n_keys // page)
    cache = mmq.empty_kv4_cache(width, 1, D, page).zero_()
    mmq.kv4_write(k, v, torch.arange(n_keys, dtype=torch.int32, device="cuda"), cache)
    table = torch.arange(width, dtype=torch.int32, device="cuda").expand(n_seq, width).contiguous()
    return dict(q=q, cache=cache, page_table=table, lens=torch.full((n_seq,), n_keys, dtype=torch.int32, device="cuda"),
                q_starts=torch.arange(n_seq + 1, dtype=torch.int32, device="cuda") * new)


@pytest.mark.parametrize("new", [1, 5])                                  # units of 128 rows, of 256
@pytest.mark.parametrize("n_seq", [1, 7, 152, 228, 304, 456])            # a unit in many runs, in one, in parts of two
@pytest.mark.parametrize("change,huge", [(64, 192), (64, 256), (128, 256), (100, 130)])
def test_a_row_that_passes_the_border_beside_one_that_rises(n_seq, new, change, huge):
    mmq = require_gpu()
    d = make(mmq, n_seq, new, 320, change, huge)
    scale = unit_scale()
    got = mmq.kv4_attention(d["q"], d["cache"], d["page_table"], d["lens"], scale=scale).double()
    assert mmq.status() == 0
    one = {**d, "q": d["q"][:new], "lens": d["lens"][:1], "page_table": d["page_table"][:1], "q_starts": d["q_starts"][:2]}
    ref, _ = reference(one, scale)
    off = (got.view(n_seq, new, 32, 128) - ref).abs()
    assert float(off.max()) <= 2.0 ** -11 + 2.0 ** -14      # A = 1, as all values are 1 or -1
