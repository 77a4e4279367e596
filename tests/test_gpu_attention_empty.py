"""Shared-prefix attention with nothing to attend to: no prefix and no page."""
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_attention import call, check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,q_len,heads,kv,D,kind", [(1, 1, 1, 1, 64, "f16"), (5, 3, 8, 2, 128, "bf16")])
def test_no_prefix_and_an_empty_page_table_is_zero(batch, q_len, heads, kv, D, kind):
    mmq = require_gpu()
    d = make(batch, q_len, heads, kv, D, 0, [0] * batch, 16, kind, 3)
    d["page_table"] = d["page_table"][:, :0].contiguous()
    out = torch.full((batch * q_len, heads, D), 7.0, device="cuda")
    got = call(mmq, d)
    call(mmq, d, out=out)
    assert (got == 0).all() and (out == 0).all() and got.shape == out.shape
    d["k_cache"], d["v_cache"] = d["k_cache"][:0], d["v_cache"][:0]
    assert (call(mmq, d) == 0).all() and mmq.status() == mmq.MMQ_OK


@pytest.mark.parametrize("prefix", [0, 70])
def test_lengths_past_an_empty_page_table_are_reported(prefix):
    """Any length is past it; it counts as 0, and the prefix is all that a token sees."""
    mmq = require_gpu()
    d = make(4, 2, 8, 2, 64, prefix, [0, 0, 0, 0], 16, "f16", 6)
    d["page_table"] = d["page_table"][:, :0].contiguous()
    check(call(mmq, d), d)
    assert mmq.status() == mmq.MMQ_OK
    for lens in ([0, 0, 0, 1], [3, 0, 0, 0]):
        got = call(mmq, dict(d, lens=torch.tensor(lens, dtype=torch.int32, device="cuda")))
        assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == mmq.MMQ_OK
        check(got, d)
    call(mmq, dict(d, lens=torch.tensor([0, -5, 0, 0], dtype=torch.int32, device="cuda")))
    assert mmq.status() == mmq.MMQ_OK
