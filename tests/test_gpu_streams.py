"""The operators between the projections on several streams: calls that follow
one another on different streams with no wait between them, and calls from
several host threads.  Inputs are finished beforehand and each call allocates
what it needs, so every result has the bits of the same call made alone."""
import threading

import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def q4k(g, n, k):
    """q4_K bytes [n][k/256][144] of weights with about unit gain."""
    raw = torch.randint(0, 256, (n, k // 256, 144), generator=g, dtype=torch.uint8, device="cuda")
    d = torch.full((n, k // 256, 1), 1 / (184 * k ** 0.5), device="cuda").half()
    raw[..., 0:2] = d.view(torch.uint8)
    raw[..., 2:4] = (d.float() * 7.5).half().view(torch.uint8)
    return raw


def rope(mmq, seed, tokens=700, heads=8, kv=2, D=128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((tokens, (heads + 2 * kv) * D), device="cuda", generator=g)
    angle = torch.rand((tokens, D // 2), device="cuda", generator=g) * 6
    at = torch.arange(tokens, device="cuda", dtype=torch.int32)
    cos, sin = angle.cos(), angle.sin()
    k, v = (torch.zeros((tokens, kv, D), device="cuda", dtype=torch.float16) for _ in range(2))
    return lambda **more: mmq.qk_norm_rope(qkv, heads, cos, sin, at, at, k, v, **more)


def attention(mmq, seed, batch=48, heads=16, kv=4, D=128, prefix=3000, page=16, most=200):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, device="cuda", generator=g).half()

    width = -(-most // page)
    q, kp, vp = normal(batch, heads, D), normal(prefix, kv, D), normal(prefix, kv, D)
    kc, vc = normal(batch * width, page, kv, D), normal(batch * width, page, kv, D)
    table = torch.randperm(batch * width, device="cuda", generator=g).view(batch, width).to(torch.int32)
    lens = torch.randint(1, most + 1, (batch,), device="cuda", generator=g).to(torch.int32)
    return lambda **more: mmq.shared_prefix_attention(q, kp, vp, kc, vc, table, lens, **more)


def moe(mmq, seed, T=17, model=1024, ffn=512, E=16, k=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, router = torch.randn((T, model), device="cuda", generator=g), torch.randn((E, model), device="cuda", generator=g)
    gu, down = q4k(g, E * 2 * ffn, model).view(E, 2 * ffn, -1, 144), q4k(g, E * model, ffn).view(E, model, -1, 144)
    router /= model ** 0.5
    return lambda **more: mmq.q4K_moe(x, router, gu, down, k, **more)


def flat(got):
    return list(got) if isinstance(got, tuple) else [got]


@pytest.mark.parametrize("make", [rope, attention, moe])
def test_streams_in_turn_without_a_wait(make):
    mmq = require_gpu()
    one, two = make(mmq, 1), make(mmq, 2)
    torch.cuda.synchronize()
    want = [[v.clone() for v in flat(f())] for f in (one, two)]
    torch.cuda.synchronize()
    sides = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = []
        for i in range(12):
            got.append((i % 2, (one, two)[i % 2](stream=sides[i % 3])))
        torch.cuda.synchronize()
        for which, g in got:
            assert all(torch.equal(a, b) for a, b in zip(flat(g), want[which]))
    assert mmq.status() == mmq.MMQ_OK


def test_threads_on_separate_streams():
    mmq = require_gpu()
    calls = [make(mmq, seed) for seed in (3, 4) for make in (rope, attention, moe)]
    torch.cuda.synchronize()
    want = [[v.clone() for v in flat(f())] for f in calls]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                outs = [calls[i]() for _ in range(30)]
                s.synchronize()
            got[i] = outs
        except Exception as e:
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    torch.cuda.synchronize()
    assert mmq.status() == mmq.MMQ_OK
    for i, outs in got.items():
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(flat(o), want[i]))
