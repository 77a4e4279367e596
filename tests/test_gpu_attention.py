"""Shared-prefix attention against softmax in 64 bits.

Tolerance per output, with e_i = exp(s_i - max s), l = sum e, w = e / l,
A = sum w |v|, u the type's unit (2^-11 float16, 2^-8 bfloat16), n keys:
  u |out|                 the output's rounding (none for a float32 output)
  u A                     the weights' rounding before the product with v
  2^-25 sum |v_i| / l     float16 weights under 2^-14 lose absolutely (those i)
  2 A (E + 2^-20)         a score is D products summed in f32, E = D 2^-23
                          scale max_i sum |q k_i|; an exponential and the joins'
                          factors are good to 2^-20
  A (n / 16 + 64) 2^-23   the sums over keys, 16 per matrix instruction, and
                          the joins (a truncating f32 add is off by 2^-23)
  2^-25                   half the float16 subnormal step of a small output
"""
import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KIND = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def make(batch, q_len, heads, kv, D, prefix, lens, page, kind, seed, spare=3, scale_v=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = KIND[kind]

    def normal(*s):
        return torch.randn(s, device="cuda", generator=g).to(dt)

    width = -(-max(max(lens), 1) // page) + 1
    pages = batch * width + spare
    return dict(q=normal(batch * q_len, heads, D), k_prefix=normal(prefix, kv, D), v_prefix=normal(prefix, kv, D),
                k_cache=normal(pages, page, kv, D), v_cache=normal(pages, page, kv, D),
                page_table=torch.randperm(pages, device="cuda", generator=g)[:batch * width].view(batch, width)
                .to(torch.int32).contiguous(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q_len=q_len)


def reference(d, scale=None):
    """(out, tolerance without the output's own rounding), 64 bits."""
    q = d["q"].double()
    T, heads, D = q.shape
    P, kv = d["k_prefix"].shape[:2]
    G, n_new = heads // kv, d["q_len"]
    scale = D ** -0.5 if scale is None else scale
    u = UNIT[d["q"].dtype]
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    page = d["k_cache"].shape[1]
    for t in range(T):
        b = t // n_new
        see = max(0, int(d["lens"][b]) - n_new + 1 + t % n_new)
        ids = d["page_table"][b, :-(-see // page)].long()
        for which, name in ((0, "k"), (1, "v")):
            own = d[name + "_cache"][ids].double().reshape(-1, kv, D)[:see]
            every = torch.cat([d[name + "_prefix"].double(), own])
            if which == 0:
                k = every
        v = every
        n = k.shape[0]
        if n == 0:
            continue
        qt = q[t].view(kv, G, D)
        s = torch.einsum("hgd,nhd->hgn", qt, k) * scale
        E = D * 2.0 ** -23 * scale * torch.einsum("hgd,nhd->hgn", qt.abs(), k.abs()).amax(-1, keepdim=True)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        l = e.sum(-1, keepdim=True)
        out[t] = (torch.einsum("hgn,nhd->hgd", e, v) / l).reshape(heads, D)
        A = torch.einsum("hgn,nhd->hgd", e, v.abs()) / l
        small = torch.einsum("hgn,nhd->hgd", (e < 2.0 ** -14).double(), v.abs()) / l * 2.0 ** -25
        tol[t] = (A * (u + 2 * (E + 2.0 ** -20) + (n / 16 + 64) * 2.0 ** -23) + small).reshape(heads, D) + 2.0 ** -25
    return out, tol


def check(got, d, scale=None):
    ref, tol = reference(d, scale)
    if got.dtype != torch.float32:
        tol = tol + UNIT[got.dtype] * ref.abs() * (1 + 2.0 ** -7)
    assert torch.isfinite(got).all()
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), float((off / tol.clamp_min(1e-300)).max())


def call(mmq, d, **more):
    return mmq.shared_prefix_attention(d["q"], d["k_prefix"], d["v_prefix"], d["k_cache"], d["v_cache"],
                                       d["page_table"], d["lens"], q_len=d["q_len"], **more)


@pytest.mark.parametrize("batch,q_len,heads,kv,D,prefix,lens,page,kind", [
    (1, 1, 1, 1, 64, 1, [1], 1, "f16"),
    (1, 1, 4, 1, 128, 0, [5], 16, "f16"),
    (2, 1, 8, 2, 128, 7, [1, 0], 16, "bf16"),
    (3, 1, 8, 8, 64, 63, [64, 65, 17], 32, "f16"),
    (5, 1, 32, 8, 128, 300, [1, 16, 33, 100, 257], 16, "f16"),
    (5, 1, 32, 8, 128, 2049, [700, 1, 3, 5, 64], 64, "bf16"),
    (4, 3, 12, 4, 64, 130, [3, 4, 90, 35], 16, "bf16"),
    (2, 5, 8, 2, 128, 129, [5, 40], 8, "f16"),
    (3, 2, 40, 2, 128, 500, [2, 9, 33], 4, "f16"),       # 20 heads per kv head: two row tiles
    (70, 1, 8, 2, 128, 1000, [1 + i % 50 for i in range(70)], 16, "f16"),
    (33, 1, 16, 16, 64, 5001, [1 + 9 * i for i in range(33)], 32, "bf16"),
    (40, 1, 32, 8, 128, 4100, [20 + i for i in range(40)], 16, "bf16"),
    (150, 2, 8, 1, 64, 777, [2 + i % 30 for i in range(150)], 16, "f16"),
    (130, 1, 32, 4, 128, 2500, [1 + i % 90 for i in range(130)], 64, "f16"),
])
def test_values(batch, q_len, heads, kv, D, prefix, lens, page, kind):
    mmq = require_gpu()
    d = make(batch, q_len, heads, kv, D, prefix, lens, page, kind, 1000 + batch)
    got = call(mmq, d)
    assert mmq.status() == 0
    check(got, d)


def test_float32_output_and_a_given_scale():
    mmq = require_gpu()
    d = make(6, 1, 16, 4, 128, 900, [1, 2, 30, 40, 50, 300], 16, "f16", 5)
    out = torch.empty((6, 16, 128), device="cuda")
    assert call(mmq, d, out=out, scale=0.3) is out
    check(out, d, 0.3)


def test_no_key_at_all_is_zero():
    mmq = require_gpu()
    d = make(3, 2, 8, 2, 128, 0, [0, 1, 7], 16, "f16", 6)
    got = call(mmq, d)
    assert (got[:2] == 0).all()          # sequence 0 has no key for either token
    assert (got[2] == 0).all()           # sequence 1's first token neither
    check(got, d)
    d = make(3, 1, 8, 2, 64, 0, [0, 0, 0], 16, "bf16", 6)
    assert (call(mmq, d) == 0).all() and mmq.status() == 0


def test_empty_page_table():
    mmq = require_gpu()
    d = make(3, 1, 8, 2, 64, 70, [0, 0, 0], 16, "bf16", 6)
    d["page_table"] = d["page_table"][:, :0].contiguous()
    check(call(mmq, d), d)
    assert mmq.status() == 0


def test_what_lies_past_a_token_is_never_used():
    """NaN and Inf in every place that a token must not see: the rest of its
    last page, unused pages, and (several new tokens) the later tokens."""
    mmq = require_gpu()
    d = make(4, 3, 8, 2, 128, 40, [3, 10, 33, 64], 16, "f16", 8)
    clean = call(mmq, d).clone()
    page = 16
    seen = torch.zeros(d["k_cache"].shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(d["lens"].tolist()):
        for i in range(n):
            seen[d["page_table"][b, i // page].long(), i % page] = True
    for name, bad in (("k_cache", float("nan")), ("v_cache", float("inf"))):
        d[name][~seen] = bad
    assert torch.equal(call(mmq, d), clean)
    for b, n in enumerate(d["lens"].tolist()):   # the newest token of each sequence
        at = d["page_table"][b, (n - 1) // page].long()
        d["k_cache"][at, (n - 1) % page] = float("nan")
        d["v_cache"][at, (n - 1) % page] = float("nan")
    got = call(mmq, d).view(4, 3, 8, 128)
    assert torch.equal(got[:, :2], clean.view(4, 3, 8, 128)[:, :2])
    assert torch.isnan(got[:, 2]).all()


def test_nan_in_a_query_stays_in_its_row():
    mmq = require_gpu()
    d = make(40, 1, 8, 2, 128, 600, [4 + i for i in range(40)], 16, "f16", 8)
    clean = call(mmq, d).clone()
    d["q"][17, 3, 5] = float("nan")
    got = call(mmq, d)
    bad = torch.isnan(got).any(-1)
    assert bad.nonzero().tolist() == [[17, 3]] and torch.isnan(got[17, 3]).all()
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("rows", ["few", "many"])
def test_scores_that_grow_and_one_key_that_takes_all(rows):
    """A maximum that rises along the prefix, far past what one exponent range holds, and a last key that outweighs
    everything."""
    mmq = require_gpu()
    batch = 3 if rows == "few" else 64
    d = make(batch, 1, 8, 2, 128, 3000, [9] * batch, 16, "bf16", 21)
    ramp = torch.linspace(0.1, 12, 3000, device="cuda")[:, None, None]
    d["k_prefix"] = (d["q"][0, 0].float() * ramp * torch.ones((1, 2, 1), device="cuda")).to(torch.bfloat16)
    check(call(mmq, d), d)
    d["k_prefix"] = d["k_prefix"].flip(0).contiguous()
    check(call(mmq, d), d)


def test_strides_and_another_stream():
    mmq = require_gpu()
    d = make(40, 1, 8, 2, 128, 333, [1 + i for i in range(40)], 16, "f16", 31)
    plain = call(mmq, d).clone()
    fused = torch.randn((40, 12, 128), device="cuda").half()
    fused[:, :8] = d["q"]
    kv = torch.randn((2, 333, 2, 2, 136), device="cuda").half()    # [layer][token][k/v][head][padded]
    kv[1, :, 0, :, :128] = d["k_prefix"]
    kv[1, :, 1, :, :128] = d["v_prefix"]
    d.update(q=fused[:, :8], k_prefix=kv[1, :, 0, :, :128], v_prefix=kv[1, :, 1, :, :128])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(mmq, d, stream=side)
    side.synchronize()
    assert torch.equal(got, plain) and mmq.status() == 0


def test_head_major_prefix():
    mmq = require_gpu()
    d = make(20, 1, 8, 2, 64, 200, [5] * 20, 16, "f16", 33)
    plain = call(mmq, d).clone()
    for name in ("k_prefix", "v_prefix"):
        d[name] = d[name].transpose(0, 1).contiguous().transpose(0, 1)
    assert d["k_prefix"].stride(1) == 200 * 64
    assert torch.equal(call(mmq, d), plain)


def test_pages_past_32_bit_offsets():
    mmq = require_gpu()
    d = make(2, 1, 4, 4, 128, 64, [40, 33], 16, "f16", 41)
    pages = 280_000   # x 16 x 4 x 128 values: past 2^31
    for name in ("k_cache", "v_cache"):
        big = torch.empty((pages, 16, 4, 128), dtype=torch.float16, device="cuda")
        big[pages - d[name].shape[0]:] = d[name]
        d[name] = big
    d["page_table"] += pages - d["page_table"].numel() - 3
    check(call(mmq, d), d)
    assert mmq.status() == 0


def test_long_prefix_past_32_bit_offsets():
    mmq = require_gpu()
    d = make(64, 1, 8, 2, 128, 0, [8] * 64, 16, "f16", 43)
    row = 2 ** 21   # values between tokens: 1100 tokens span past 2^31
    kv = torch.empty((1100, row), dtype=torch.float16, device="cuda")
    for i, name in enumerate(("k_prefix", "v_prefix")):
        part = kv[:, 256 * i:256 * (i + 1)]
        part.copy_(torch.randn((1100, 256), device="cuda"))
        d[name] = part.view(1100, 2, 128)
    check(call(mmq, d), d)


def test_bad_pages_and_lengths_are_reported():
    mmq = require_gpu()
    d = make(3, 1, 8, 2, 64, 30, [20, 20, 20], 16, "f16", 51)
    clean = call(mmq, d).clone()
    for bad in (-1, d["k_cache"].shape[0]):
        table = d["page_table"].clone()
        table[1, 1] = bad
        got = call(mmq, dict(d, page_table=table))
        assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
        assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    room = d["page_table"].shape[1] * 16
    got = call(mmq, dict(d, lens=torch.tensor([20, room + 1, -5], dtype=torch.int32, device="cuda")))
    assert mmq.status() == mmq.MMQ_ERR_ARG
    want = dict(d, lens=torch.tensor([20, room, 0], dtype=torch.int32, device="cuda"))
    check(got, want)


def test_runs_are_bit_identical_and_workspace_may_be_given():
    mmq = require_gpu()
    d = make(64, 1, 32, 8, 128, 5000, [1 + 5 * i for i in range(64)], 16, "f16", 61)
    a = call(mmq, d).clone()
    ws = torch.full((200 << 20,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(mmq, d, workspace=ws), a)
    with pytest.raises(mmq.MMQError) as e:
        call(mmq, d, workspace=ws[:1024])
    assert e.value.code == mmq.MMQ_ERR_ARG


def test_no_sequences():
    mmq = require_gpu()
    d = make(1, 1, 8, 2, 64, 30, [20], 16, "f16", 51)
    d.update(q=d["q"][:0], page_table=d["page_table"][:0], lens=d["lens"][:0])
    assert call(mmq, d).shape == (0, 8, 64)
