"""Failure detection in the layer operators without a GPU fault: a copy that is
not made lets the bounded waits of the prefix attention and of the experts'
products run out; the kernels record MMQ_ERR_DEVICE_TIMEOUT, let what is in
flight finish, and return, and the next call is as before."""
import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_attention import call as attention
from tests.test_gpu_attention import make as attention_inputs
from tests.test_gpu_moe import call as moe
from tests.test_gpu_moe import make as moe_inputs

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def timed_out_once(mmq, f):
    want = [v.clone() for v in f()]
    assert mmq.status() == mmq.MMQ_OK
    mmq.mmq_debug_inject_timeout(True)
    f()
    assert mmq.status() == mmq.MMQ_ERR_DEVICE_TIMEOUT
    assert mmq.status() == mmq.MMQ_OK
    assert all(torch.equal(a, b) for a, b in zip(f(), want))   # one shot, and the context is as before
    assert mmq.status() == mmq.MMQ_OK


@pytest.mark.parametrize("batch,heads,kv,D,prefix", [
    (4, 8, 2, 128, 300),      # one row tile, three key tiles
    (2, 4, 4, 64, 100),       # one key tile, none for the second group
    (70, 8, 2, 128, 900),     # two row tiles
    (40, 90, 45, 64, 3000),   # two row tiles, more key tiles than fit the ring
])
def test_prefix_attention(batch, heads, kv, D, prefix):
    mmq = require_gpu()
    d = attention_inputs(batch, 1, heads, kv, D, prefix, [1 + i % 30 for i in range(batch)], 16, "f16", 5)
    timed_out_once(mmq, lambda: [attention(mmq, d)])


@pytest.mark.parametrize("T,model,ffn,E,top_k", [(1, 512, 256, 8, 2), (9, 4352, 512, 8, 2), (33, 2048, 1024, 4, 4)])
def test_experts(T, model, ffn, E, top_k):
    mmq = require_gpu()
    d = moe_inputs(T, model, ffn, E, top_k, True, True, 5)
    timed_out_once(mmq, lambda: list(moe(mmq, d)))


def test_attention_without_a_prefix_leaves_the_flag():
    """Nothing in it waits; the next call with a prefix takes the flag."""
    mmq = require_gpu()
    d = attention_inputs(3, 1, 8, 2, 64, 0, [5, 6, 7], 16, "f16", 5)
    e = attention_inputs(3, 1, 8, 2, 64, 40, [5, 6, 7], 16, "f16", 5)
    mmq.mmq_debug_inject_timeout(True)
    attention(mmq, d)
    assert mmq.status() == mmq.MMQ_OK
    attention(mmq, e)
    assert mmq.status() == mmq.MMQ_ERR_DEVICE_TIMEOUT
