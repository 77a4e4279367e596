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
