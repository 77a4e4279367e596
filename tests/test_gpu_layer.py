"""The decode layer of examples/moe_decode_layer.py: every step's result
against the layer's formulas in 64 bits on what the step before handed on, so
that the roundings that belong to the path (q8_1 activations, float16 caches)
are in both.  Bounds on the 2-norm of the difference over that of the result:
  projections        1e-4   the GEMM's bound against sums of magnitudes
  head norms, rotary 2^-11  one rounding to float16
  attention          2^-10  the weights' rounding to float16, at most 2^-11 of
                            each term, and the sums in f32
  experts            1e-5   f32 arithmetic on the dequantized weights
"""
import importlib.util
import math
import os

import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_decode_layer", os.path.join(ROOT, "examples", "moe_decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def weights(w):
    """q4_K bytes [..][sb][144] -> 64-bit [..][256 sb]."""
    d, dmin = w[..., :4].contiguous().view(torch.float16).double().unbind(-1)
    s = w[..., 4:16].long()
    lo, mid, hi = s[..., :4], s[..., 4:8], s[..., 8:]
    sc = torch.cat([lo & 63, (hi & 15) + ((lo >> 6) << 4)], -1) * d[..., None]
    mn = torch.cat([mid & 63, (hi >> 4) + ((mid >> 6) << 4)], -1) * dmin[..., None]
    q = w[..., 16:].unflatten(-1, (4, 32))
    q = torch.stack([q & 15, q >> 4], -2).flatten(-3, -2).double()
    return (q * sc[..., None] - mn[..., None]).flatten(-3)


def norm(x, w):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()


def dequantize(mmq, x):
    qs, da, _ = mmq.quantize_q8_1(x)
    return qs.double() * da.double().repeat_interleave(32, 1)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_decode_steps():
    mmq = require_gpu()
    ex = example()
    batch = 5
    L = ex.Layer(hidden=1024, heads=8, kv_heads=2, dim=128, ffn=512, experts=8, top_k=2, prompt=333, batch=batch, new=40)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    D, half = L.dim, L.dim // 2
    for step in range(18):          # past the end of the first page
        x = torch.randn((batch, 1024), device="cuda", generator=g)
        keep = {}
        out, ids = ex.decode_step(L, x, lens, keep)
        assert mmq.status() == mmq.MMQ_OK
        # projection
        a = dequantize(mmq, ex.rms_norm(x, L.norm_attn))
        assert off(keep["qkv"], a @ weights(L.w_qkv).T) < 1e-4
        # head norms, rotary positions, cache
        q, k, v = keep["qkv"].double().view(batch, -1, D).split([L.heads, L.kv_heads, L.kv_heads], 1)
        q, k = norm(q, L.q_weight), norm(k, L.k_weight)
        at = (lens + L.prompt).long()
        c, s = L.cos[at].double()[:, None], L.sin[at].double()[:, None]
        q, k = (torch.cat([a[..., :half] * c - a[..., half:] * s, a[..., :half] * s + a[..., half:] * c], -1) for a in (q, k))
        pages = L.k_cache.view(-1, L.kv_heads, D), L.v_cache.view(-1, L.kv_heads, D)
        slot = [int(L.page_table[b, int(lens[b]) // L.page]) * L.page + int(lens[b]) % L.page for b in range(batch)]
        assert keep["slots"].tolist() == slot
        for got, want in ((keep["q"], q), (pages[0][slot], k), (pages[1][slot], v)):
            assert off(got, want) < 2.0 ** -11
        # attention, on the cache as it is
        q = keep["q"].double()
        seen = torch.empty_like(q)
        for b in range(batch):
            own = [int(L.page_table[b, i // L.page]) * L.page + i % L.page for i in range(int(lens[b]) + 1)]
            ks, vs = (torch.cat([p.double(), own_p[own].double()]) for p, own_p in zip((L.k_prompt, L.v_prompt), pages))
            w = torch.softmax(torch.einsum("hgd,nhd->hgn", q[b].view(L.kv_heads, -1, D), ks) / math.sqrt(D), -1)
            seen[b] = torch.einsum("hgn,nhd->hgd", w, vs).reshape(-1, D)
        assert off(keep["seen"], seen) < 2.0 ** -10
        # output projection and residual
        a = dequantize(mmq, keep["seen"].view(batch, -1))
        assert off(keep["x"], x.double() + a @ weights(L.w_o).T) < 1e-4
        # experts
        z = keep["z"].double()
        p = torch.softmax(z @ L.w_router.double().T, -1)
        best, want = p.sort(-1, descending=True)
        best, want = best[:, :L.top_k], want[:, :L.top_k]
        assert (ids == want).all()
        w = best / best.sum(-1, keepdim=True)
        ref = keep["x"].double()
        for b in range(batch):
            for j in range(L.top_k):
                gu = weights(L.w_gu[want[b, j]]) @ z[b]
                ref[b] += w[b, j] * (weights(L.w_down[want[b, j]]) @ (gu[0::2] * torch.sigmoid(gu[0::2]) * gu[1::2]))
        assert off(out, ref) < 1e-5
        lens += 1


def test_decode_step_in_a_graph():
    """Captured and replayed with other inputs, the step gives what it gives directly."""
    mmq = require_gpu()
    ex = example()
    L = ex.Layer(hidden=512, heads=4, kv_heads=2, dim=64, ffn=256, experts=8, top_k=2, prompt=200, batch=6, new=16)
    x = torch.randn((6, 512), device="cuda")
    lens = torch.zeros(6, dtype=torch.int32, device="cuda")
    ex.decode_step(L, x, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = ex.decode_step(L, x, lens)
    for step in range(3):
        x.normal_()
        lens.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(ex.decode_step(L, x, lens)[0], got)
    assert mmq.status() == mmq.MMQ_OK


@pytest.mark.parametrize("programmatic", [False, True])
def test_steps_with_programmatic_launch(programmatic):
    """Many steps back to back, every kernel reading what the one before wrote: the same bits with and without it."""
    mmq = require_gpu()
    ex = example()
    L = ex.Layer(hidden=512, heads=4, kv_heads=2, dim=128, ffn=256, experts=8, top_k=2, prompt=300, batch=40, new=48)
    g = torch.Generator(device="cuda").manual_seed(2)
    x0 = torch.randn((40, 512), device="cuda", generator=g)

    def steps():
        L.k_cache.zero_()
        L.v_cache.zero_()
        x, lens = x0, torch.zeros(40, dtype=torch.int32, device="cuda")
        for _ in range(20):
            x, _ = ex.decode_step(L, x, lens)
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True))
            lens = lens + 1
        return x

    plain = steps()
    try:
        mmq.mmq_set_programmatic_launch(programmatic)
        for _ in range(5):
            assert torch.equal(steps(), plain)
    finally:
        mmq.mmq_set_programmatic_launch(False)
    assert mmq.status() == mmq.MMQ_OK and torch.isfinite(plain).all()
