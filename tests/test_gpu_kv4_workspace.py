"""What a 4-bit attention call's workspace depends on: its sizes, and whether q_starts is given."""
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_kv4_attention import call, check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def bytes_of(mmq, d, starts):
    T, heads, D = d["q"].shape
    pages, kv, tiles, _ = d["cache"].shape
    kind = mmq.MMQ_TYPE_F16 if d["q"].dtype is torch.float16 else mmq.MMQ_TYPE_BF16
    return mmq.mmq_kv4_attention_workspace(mmq.mmq_kv4_attention_t(
        q_starts=d["q_starts"].data_ptr() if starts else None, q_stride=heads * D, tokens=T, n_pages=pages,
        table_width=d["page_table"].shape[1], batch=len(d["lens"]), heads=heads, kv_heads=kv, head_dim=D,
        page_size=16 * tiles, type=kind, out_type=kind, scale=D ** -0.5))


@pytest.mark.parametrize("news,n_seq,heads,kv,D", [(1, 64, 32, 8, 128), (4, 9, 16, 2, 64), (9, 17, 28, 4, 128), (300, 2, 8, 2, 64)])
def test_what_is_asked_for_is_enough(news, n_seq, heads, kv, D):
    """With q_starts or without; no byte past it is written; and a workspace for the call without is refused where it is
    too small for the call with."""
    mmq = require_gpu()
    d = make(mmq, [news] * n_seq, [news + 50 * i for i in range(n_seq)], heads, kv, D, 16, "f16", 5)
    sizes = {}
    for starts in (False, True):
        n = sizes[starts] = bytes_of(mmq, d, starts)
        assert n > 0
        room = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
        more = dict(q_starts=d["q_starts"]) if starts else {}
        got = mmq.kv4_attention(d["q"], d["cache"], d["page_table"], d["lens"], workspace=room[:n], **more)
        assert mmq.status() == 0 and (room[n:] == 77).all()
        check(got, d)
    assert sizes[True] >= sizes[False]
    if news == 1:
        assert sizes[True] > sizes[False]
        with pytest.raises(mmq.MMQError) as e:
            call(mmq, d, workspace=room[:sizes[False]])
        assert e.value.code == mmq.MMQ_ERR_ARG
