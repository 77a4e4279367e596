"""Failure detection in the 4-bit attention without a GPU fault: a copy that is
not made lets the bounded waits of its two kernels run out; they record
MMQ_ERR_DEVICE_TIMEOUT, let what is in flight finish, and return, and the next
call is as before."""
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_kv4_attention import call, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("news,lens,heads,kv,D,kind", [
    ([1] * 3, [700, 40, 9], 8, 2, 128, "f16"),           # a row per head, units of eight
    ([2] * 40, [500] * 40, 16, 2, 64, "bf16"),           # units of sixteen rows
    ([20], [900], 8, 2, 128, "bf16"),                    # 128 rows, two streams to a CTA
    ([30] * 20, [400] * 20, 4, 1, 64, "f16"),
    ([300], [2000], 8, 2, 128, "f16"),                   # 256 rows
    ([200] * 9, [300] * 9, 8, 2, 64, "bf16"),
    ([1, 40], [900, 900], 8, 2, 128, "f16"),             # a sequence for either kernel
])
def test_waits_that_run_out(news, lens, heads, kv, D, kind):
    mmq = require_gpu()
    d = make(mmq, news, lens, heads, kv, D, 16, kind, 3)
    want = call(mmq, d).clone()
    assert mmq.status() == mmq.MMQ_OK
    mmq.mmq_debug_inject_timeout(True)
    call(mmq, d)
    assert mmq.status() == mmq.MMQ_ERR_DEVICE_TIMEOUT
    assert mmq.status() == mmq.MMQ_OK
    for _ in range(3):   # one shot, and the context is as before
        assert torch.equal(call(mmq, d), want)
    assert mmq.status() == mmq.MMQ_OK


def test_other_operators_leave_the_flag():
    """Nothing in them waits; the next attention takes it."""
    mmq = require_gpu()
    d = make(mmq, [1, 1], [40, 50], 8, 2, 64, 16, "f16", 4)
    slots = torch.arange(16, dtype=torch.int32, device="cuda")
    mmq.mmq_debug_inject_timeout(True)
    k, v = mmq.kv4_read(d["cache"], slots)
    mmq.kv4_write(k, v, slots, d["cache"])
    mmq.pages_copy([d["cache"]], slots[:1], slots[1:2])
    assert mmq.status() == mmq.MMQ_OK
    call(mmq, d)
    assert mmq.status() == mmq.MMQ_ERR_DEVICE_TIMEOUT
