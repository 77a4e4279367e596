"""A call in which one CTA works on a single unit for longer than the limit of its waits, and on many short ones after it:
what the roles are told ahead waits for the long unit as long as that takes."""
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_kv4_attention import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_short_units_behind_one_of_over_a_second():
    mmq = require_gpu()
    kv, heads, D, page, rows, short = 16, 32, 64, 1024, 128, 10    # 256 rows of a kv head to a sequence
    g = torch.Generator(device="cuda").manual_seed(91)
    long = 2 ** 31 - 1024                                          # 2^25 tiles, 16 heads, 152 CTAs
    width = long // page
    pages = 1 + short
    cache = mmq.empty_kv4_cache(pages, kv, D, page)
    k, v = torch.randn((2, pages * page, kv, D), device="cuda", generator=g)
    mmq.kv4_write(k, v, torch.arange(pages * page, dtype=torch.int32, device="cuda"), cache)
    table = torch.zeros((1 + short, width), dtype=torch.int32, device="cuda")
    table[1:, 0] = torch.arange(1, 1 + short, dtype=torch.int32, device="cuda")
    lens = torch.tensor([long] + [rows + 30 * i for i in range(short)], dtype=torch.int32, device="cuda")
    q = torch.randn(((1 + short) * rows, heads, D), device="cuda", generator=g).half()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    out = mmq.kv4_attention(q, cache, table, lens)
    end.record()
    assert mmq.status() == 0
    assert begin.elapsed_time(end) > 1500
    assert torch.isfinite(out).all()
    d = dict(q=q[rows:], cache=cache, page_table=table[1:].contiguous(), lens=lens[1:].contiguous(),
             q_starts=torch.arange(short + 1, dtype=torch.int32, device="cuda") * rows)
    check(out[rows:], d)
