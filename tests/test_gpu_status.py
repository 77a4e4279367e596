"""The device status word when two kernels have something to say: a wait that
ran out makes a whole output invalid, and is told even if an argument out of
range, which makes one token's, came first."""
import pytest

from q4_q8_int8_gb300 import synthetic
from tests.gpu_util import require_gpu, to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", ["argument", "timeout"])
def test_a_timeout_is_told_before_an_argument(first):
    mmq = require_gpu()
    M, N, K = 128, 256, 512
    aq = mmq.quantize_q8_1(to_dev(synthetic.activations(M, K, 5)))
    w = to_dev(synthetic.q4K_weights(N, K, 6).reshape(-1))
    cache = torch.zeros((4, 1, 64), dtype=torch.float16, device="cuda")
    at = torch.zeros(1, dtype=torch.int32, device="cuda")

    def argument():          # a slot past the cache
        mmq.qk_norm_rope(torch.ones((1, 3 * 64), device="cuda"), 1, torch.ones((1, 32), device="cuda"),
                         torch.ones((1, 32), device="cuda"), at, at + 4, cache, cache)

    def timeout():
        mmq.mmq_debug_inject_timeout(True)
        mmq.q4K_gemm(aq, w, N, path=mmq.MMQ_PATH_TC)

    assert mmq.status() == mmq.MMQ_OK
    for f in (argument, timeout) if first == "argument" else (timeout, argument):
        f()
    assert mmq.status() == mmq.MMQ_ERR_DEVICE_TIMEOUT
    assert mmq.status() == mmq.MMQ_OK
    argument()
    assert mmq.status() == mmq.MMQ_ERR_ARG
