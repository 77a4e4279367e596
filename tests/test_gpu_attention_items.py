"""Shared-prefix attention with more pieces of work (row block, kv head, part of
the prefix) than SMs, so that a CTA of the prefix kernel takes several: key
tiles in odd and even numbers, one tile only (where the second group of a CTA
has none), one and two row tiles.  Values and tolerances as in the other tests
of this operator."""
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_attention import call, check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def pieces(mmq, d):
    """Items of the prefix kernel for these sizes without a suffix, from the workspace: 8 + 4 D bytes per part, token
    and head.  Up to 48 rows per kv head an item makes two parts, of up to 128 rows; else one, of up to 256."""
    T, heads, D = d["q"].shape
    P, kv, _ = d["k_prefix"].shape
    p = mmq.mmq_shared_prefix_attention_t(
        q_stride=heads * D, prefix=P, prefix_token_stride=kv * D, prefix_head_stride=D, n_pages=1, table_width=0, batch=T,
        q_len=1, heads=heads, kv_heads=kv, head_dim=D, page_size=16, type=0, out_type=0, scale=1.0)
    parts = mmq.mmq_shared_prefix_attention_workspace(p) // (T * heads * (8 + 4 * D))
    rows = T * heads // kv
    return parts // 2 * kv if rows <= 48 else parts * kv * -(-rows // 256)


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("batch,heads,kv,D,prefix,kind,per_sm", [
    # up to 48 rows per kv head: one row tile, the groups take key tiles in turn
    (2, 500, 500, 64, 100, "f16", 3),
    (3, 500, 500, 64, 128, "bf16", 3),
    (1, 480, 480, 128, 1, "f16", 3),
    (2, 500, 500, 64, 300, "f16", 3),
    (1, 320, 320, 128, 257, "bf16", 2),
    (2, 170, 170, 128, 500, "f16", 1),
    (2, 100, 100, 64, 3665, "f16", 1),       # parts of ten key tiles and of nine
    (3, 104, 104, 128, 8993, "bf16", 2),
    # two row tiles, of which the second may be empty
    (60, 500, 500, 64, 100, "bf16", 3),
    (60, 170, 170, 128, 300, "f16", 1),
    (60, 100, 100, 64, 2333, "bf16", 1),
    (300, 90, 90, 64, 257, "f16", 1),
    (150, 320, 80, 128, 700, "bf16", 1),
    (700, 64, 64, 64, 130, "f16", 1),
])
def test_several_pieces_per_sm(batch, heads, kv, D, prefix, kind, per_sm, own):
    mmq = require_gpu()
    d = make(batch, 1, heads, kv, D, prefix, [1 + i % 20 for i in range(batch)] if own else [0] * batch, 16, kind, 70 + batch,
             spare=0)
    if not own:
        d["page_table"] = d["page_table"][:, :0].contiguous()
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert pieces(mmq, d) > per_sm * sms
    got = call(mmq, d)
    assert mmq.status() == mmq.MMQ_OK
    check(got, d)
