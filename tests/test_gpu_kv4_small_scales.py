"""Attention over a 4-bit cache whose key scales are float16 subnormals, under queries that make their scores count.

A float16 under 2^-14 is an integer times 2^-24, and eight significant bits may be its lowest eight.  The reference and
its tolerance are those of the other attention tests.
"""
import pytest

from tests import kv4_layout as layout
from tests.gpu_util import require_gpu
from tests.test_gpu_kv4_attention import KIND, call, check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# eight rows, sixteen (two units of eight and one of sixteen), the tensor-core form's 128 and 256
FORMS = [([1, 1], 8, 2), ([1, 1, 1], 32, 2), ([4, 2], 8, 2), ([60, 33], 8, 2), ([300], 8, 2)]


def loud(d, kind, size):
    d["q"] = (d["q"].float() * size).clamp(-65000, 65000).to(KIND[kind]) if kind == "f16" else (d["q"].float() * size).to(KIND[kind])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,k_scale,size", [("f16", 1e-4, 1e4), ("f16", 5e-5, 1.5e4), ("f16", 5e-6, 2e4), ("bf16", 1e-5, 1e5),
                                               ("bf16", 1e-6, 1e6)])
@pytest.mark.parametrize("news,heads,kv", FORMS)
def test_small_keys_under_large_queries(news, heads, kv, kind, k_scale, size, D):
    mmq = require_gpu()
    d = make(mmq, news, [400 + 37 * i for i in range(len(news))], heads, kv, D, 16, kind, 61, k_scale=k_scale)
    loud(d, kind, size)
    check(call(mmq, d), d)
    check(call(mmq, d, out=torch.empty(d["q"].shape, device="cuda")), d)
    assert mmq.status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news,heads,kv", FORMS)
def test_every_subnormal_scale_of_eight_bits(news, heads, kv, D):
    """Key scales of either sign drawn from all of them, and some normal ones beside."""
    mmq = require_gpu()
    lens = [333 + 50 * i for i in range(len(news))]
    d = make(mmq, news, lens, heads, kv, D, 16, "bf16", 62)
    g = torch.Generator(device="cuda").manual_seed(63)
    pages, _, tiles, _ = d["cache"].shape
    slots = torch.arange(pages * tiles * 16, device="cuda")
    _, ks, _, _, _ = layout.places(slots, kv, 16 * tiles, D)
    at = ks[..., ::32] // 2
    bits = torch.randint(0, 256, at.shape, device="cuda", generator=g) << torch.randint(0, 3, at.shape, device="cuda", generator=g)
    bits = torch.where(torch.rand(at.shape, device="cuda", generator=g) < 0.1, 0x0400 + 8 * (bits & 127), bits)   # 2^-14 and on
    bits |= torch.randint(0, 2, at.shape, device="cuda", generator=g) << 15
    half = d["cache"].view(-1).view(torch.int16)
    half[at.flatten()] = torch.where(bits < 32768, bits, bits - 65536).to(torch.int16).flatten()
    for size in (1.0, 1e3, 3e4):
        d["q"] = torch.randn(d["q"].shape, device="cuda", generator=g).mul_(size).to(torch.bfloat16)
        check(call(mmq, d), d)
    assert mmq.status() == 0
