"""Attention over the 4-bit cache against softmax in 64 bits on the cache's own values.

Tolerance per output, with e_i = exp(s_i - max s), l = sum e, w = e / l,
A = sum w |v|, u the output type's unit (2^-11 float16, 2^-8 bfloat16, 0
float32), n keys:
  u |out|                 the output's rounding
  2^-22 A                 the weights as sums of two float16 values
  2^-24 sum |v_i| / l     and what both lose absolutely, against a largest weight of at least one
  2 A E                   a score's error E: D products of up to 24 |q| d summed in f32 (the codes, and 8 |q| d taken off),
                          2^-23 each, and roundings of 2^-22 of the score itself
  A 2^-20                 exponentials and the joins' factors
  A (n / 8 + 64) 2^-23    the sums over keys, two products per 16, and the joins
  2^-25                   half the float16 subnormal step of a small output
In a call that takes the tensor-core form weights are one float16 value: 2^-11 A instead of 2^-22 A, and those under
2^-14 of the reference lose up to 2^-25 of it (the term above covers them).
"""
import pytest

from tests import kv4_layout as layout
from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KIND = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def make(mmq, news, lens, heads, kv, D, page, kind, seed, spare=3, k_scale=1.0):
    """A batch with `news` new tokens and `lens` tokens per sequence, in pages anywhere; unused places hold random bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, device="cuda", generator=g)

    width = -(-max(max(lens), 1) // page) + 1
    pages = len(lens) * width + spare
    table = torch.randperm(pages, device="cuda", generator=g)[:len(lens) * width].view(len(lens), width).to(torch.int32)
    cache = mmq.empty_kv4_cache(pages, kv, D, page).random_(0, 256, generator=g)
    for b, n in enumerate(lens):
        if n:
            i = torch.arange(n, device="cuda")
            slots = (table[b, i // page].long() * page + i % page).to(torch.int32)
            mmq.kv4_write(normal(n, kv, D) * k_scale, normal(n, kv, D), slots, cache)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    return dict(q=normal(starts[-1], heads, D).to(KIND[kind]), cache=cache, page_table=table.contiguous(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                q_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))


def reference(d, scale=None, weight_unit=2.0 ** -11):
    """(out, tolerance without the output's own rounding), 64 bits."""
    q = d["q"].double()
    T, heads, D = q.shape
    kv, page = d["cache"].shape[1], d["cache"].shape[2] * 16
    G = heads // kv
    scale = D ** -0.5 if scale is None else scale
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    starts, lens = d["q_starts"].tolist(), d["lens"].tolist()
    for b, L in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi or L <= 0:
            continue
        i = torch.arange(L, device="cuda")
        kq, ks, vq, vs = layout.codes_and_scales(d["cache"], d["page_table"][b, i // page] * page + i % page)
        k, v = (kq - 8) * ks, (vq - 8) * vs
        qs = q[lo:hi].view(hi - lo, kv, G, D)
        s = torch.einsum("jhgd,nhd->jhgn", qs, k) * scale
        see = L - (hi - lo) + 1 + torch.arange(hi - lo, device="cuda")
        hidden = (i >= see[:, None])[:, None, None, :]
        big = torch.einsum("jhgd,nhd->jhgn", qs.abs(), ks.abs()) * (24 * scale)
        E = (D * 2.0 ** -23 * big + 2.0 ** -22 * s.abs()).masked_fill(hidden, 0).amax(-1, keepdim=True)
        s = s.masked_fill(hidden, float("-inf"))
        none = hidden.expand_as(s).all(-1, keepdim=True)
        e = torch.exp(s - s.amax(-1, keepdim=True).masked_fill(none, 0))
        l = e.sum(-1, keepdim=True).masked_fill(none, 1)
        out[lo:hi] = (torch.einsum("jhgn,nhd->jhgd", e, v) / l).reshape(hi - lo, heads, D)
        A = torch.einsum("jhgn,nhd->jhgd", e, v.abs()) / l
        lost = torch.einsum("jhgn,nhd->jhgd", (~hidden).double().expand_as(s), v.abs()) / l * 2.0 ** -24
        n = see.clamp_min(0)[:, None, None, None]
        tol[lo:hi] = (A * (weight_unit + 2 * E + 2.0 ** -20 + (n / 8 + 64) * 2.0 ** -23) + lost).reshape(hi - lo, heads, D) + 2.0 ** -25
    return out, tol


def check(got, d, scale=None, weight_unit=2.0 ** -11):
    ref, tol = reference(d, scale, weight_unit)
    tol = tol + UNIT[got.dtype] * ref.abs() * (1 + 2.0 ** -7)
    n = int(d["q_starts"][-1])
    assert torch.isfinite(got[:n]).all()
    off = (got.double() - ref).abs()[:n]
    assert (off <= tol[:n]).all(), float((off / tol[:n].clamp_min(1e-300)).max())


def fill(mmq, d):
    """Numbers in every place of the cache, for lengths past those that make() wrote."""
    pages, kv, tiles, size = d["cache"].shape
    n = pages * tiles * 16
    k, v = torch.randn((2, n, kv, size // 18), device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    mmq.kv4_write(k, v, torch.arange(n, dtype=torch.int32, device="cuda"), d["cache"])


def call(mmq, d, **more):
    return mmq.kv4_attention(d["q"], d["cache"], d["page_table"], d["lens"], q_starts=d["q_starts"], **more)


@pytest.mark.parametrize("news,lens,heads,kv,D,page,kind", [
    ([1], [1], 1, 1, 64, 16, "f16"),
    ([1], [5], 4, 1, 128, 16, "f16"),
    ([1], [16], 8, 8, 64, 32, "bf16"),
    ([1, 1, 1], [17, 1, 300], 32, 8, 128, 16, "f16"),
    ([1] * 5, [1, 16, 33, 100, 2570], 32, 8, 128, 64, "bf16"),
    ([1] * 3, [15, 16, 31], 28, 4, 64, 16, "f16"),              # seven heads to a kv head
    ([1] * 2, [900, 40], 40, 2, 128, 32, "bf16"),               # twenty: units of sixteen rows and the rest
    ([1] * 70, [1 + 37 * i % 400 for i in range(70)], 8, 2, 128, 16, "f16"),
    ([1] * 300, [1 + 7 * i % 60 for i in range(300)], 4, 4, 64, 16, "bf16"),
    ([1], [20000], 8, 2, 128, 64, "f16"),                        # one long sequence over all CTAs
    ([1], [9001], 64, 4, 64, 16, "bf16"),                        # sixteen rows
    ([3, 1, 5], [3, 40, 700], 12, 4, 64, 16, "bf16"),
    ([5, 2, 0, 4, 1], [100, 2, 50, 33, 1], 28, 4, 128, 32, "f16"),
    ([0, 0, 3, 0], [9, 0, 64, 0], 8, 2, 128, 16, "f16"),
    ([40, 1, 17], [40, 500, 130], 8, 2, 64, 16, "f16"),
    ([130], [131], 4, 1, 128, 16, "bf16"),
    ([700, 300], [1500, 300], 32, 8, 128, 64, "f16"),
])
def test_values(news, lens, heads, kv, D, page, kind):
    mmq = require_gpu()
    d = make(mmq, news, lens, heads, kv, D, page, kind, 1000 + len(news))
    got = call(mmq, d)
    assert mmq.status() == 0
    check(got, d)
    if len(set(news)) == 1:
        same = mmq.kv4_attention(d["q"], d["cache"], d["page_table"], d["lens"])
        assert mmq.status() == 0
        check(same, d)


def test_float32_output_a_given_scale_and_precision():
    """A decode step's float32 output shows the weights' 22 bits."""
    mmq = require_gpu()
    d = make(mmq, [1] * 6, [1, 2, 30, 40, 500, 3000], 16, 4, 128, 16, "f16", 5)
    out = torch.empty((6, 16, 128), device="cuda")
    assert call(mmq, d, out=out, scale=0.3) is out
    check(out, d, 0.3, weight_unit=2.0 ** -22)


def test_no_key_at_all_is_zero():
    mmq = require_gpu()
    d = make(mmq, [2, 2, 2, 1], [0, 1, 7, 0], 8, 2, 128, 16, "f16", 6)
    got = call(mmq, d)
    assert (got[:3] == 0).all() and (got[6] == 0).all() and mmq.status() == 0
    check(got, d)


def test_empty_page_table_and_empty_cache():
    mmq = require_gpu()
    d = make(mmq, [1, 1], [0, 0], 8, 2, 64, 16, "bf16", 6)
    d["page_table"] = d["page_table"][:, :0].contiguous()
    assert (call(mmq, d) == 0).all() and mmq.status() == 0
    d["cache"] = d["cache"][:0].contiguous()
    assert (call(mmq, d) == 0).all() and mmq.status() == 0


def test_rows_of_no_sequence_are_left_alone():
    mmq = require_gpu()
    d = make(mmq, [3, 2], [20, 9], 8, 2, 64, 16, "f16", 6)
    d["q"] = torch.cat([d["q"], torch.full_like(d["q"][:4], float("nan"))])
    out = torch.full_like(d["q"], 7)
    call(mmq, d, out=out)
    assert (out[5:] == 7).all() and mmq.status() == 0
    check(out, d)
    d["q_starts"] += 1                       # and those before the first
    d["q"] = d["q"].roll(1, 0).contiguous()
    shifted = call(mmq, d, out=torch.full_like(out, 3))
    assert torch.equal(shifted[1:6], out[:5]) and (shifted[[0, 6, 7, 8]] == 3).all()


@pytest.mark.parametrize("news,lens", [([1, 1, 1], [3, 33, 64]), ([3, 3, 5], [3, 10, 40]), ([90, 40], [100, 60])])
def test_what_lies_past_a_token_is_never_used(news, lens):
    """Scales that are no numbers in every place that a token must not see: the rest of its last tile and page, unused
    pages, and the later new tokens."""
    mmq = require_gpu()
    d = make(mmq, news, lens, 8, 2, 128, 32, "f16", 8)
    clean = call(mmq, d).clone()
    page, kv, D = 32, 2, 128
    pages = d["cache"].shape[0]
    seen = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        i = torch.arange(n, device="cuda")
        seen[d["page_table"][b, i // page].long() * page + i % page] = True

    def spoil(slots, key, value):
        _, ks, _, vs, _ = layout.places(slots, kv, page, D)
        half = d["cache"].view(-1).view(torch.float16)
        half[ks.flatten() // 2] = key
        half[vs.flatten() // 2] = value

    spoil((~seen).nonzero().flatten(), float("nan"), float("inf"))
    assert torch.equal(call(mmq, d), clean)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    last = torch.zeros(starts[-1], dtype=torch.bool, device="cuda")
    newest = []
    for b, n in enumerate(lens):
        newest.append(int(d["page_table"][b, (n - 1) // page]) * page + (n - 1) % page)
        last[starts[b + 1] - 1] = True
    spoil(torch.tensor(newest, device="cuda"), 0.25, float("nan"))
    got = call(mmq, d)
    assert torch.equal(got[~last], clean[~last]) and torch.isnan(got[last]).all()
    spoil(torch.tensor(newest, device="cuda"), float("nan"), 0.25)
    got = call(mmq, d)
    assert torch.equal(got[~last], clean[~last]) and torch.isnan(got[last]).all()
    # a value block of its own: the other dimensions stay numbers
    spoil(torch.tensor(newest, device="cuda"), 0.25, 0.25)
    whole = call(mmq, d).clone()
    _, _, _, vs, _ = layout.places(torch.tensor(newest, device="cuda"), kv, page, D)
    d["cache"].view(-1).view(torch.float16)[vs[..., 32:64].flatten() // 2] = float("-inf")
    got = call(mmq, d)
    assert torch.equal(got[~last], clean[~last])
    assert not torch.isfinite(got[last][..., 32:64]).any()
    assert torch.equal(got[last][..., 64:], whole[last][..., 64:]) and torch.equal(got[last][..., :32], whole[last][..., :32])


def test_nan_in_a_query_stays_in_its_row():
    mmq = require_gpu()
    d = make(mmq, [2] * 20, [4 + i for i in range(20)], 8, 2, 128, 16, "f16", 8)
    clean = call(mmq, d).clone()
    d["q"][17, 3, 5] = float("nan")
    got = call(mmq, d)
    bad = torch.isnan(got).any(-1)
    assert bad.nonzero().tolist() == [[17, 3]] and torch.isnan(got[17, 3]).all()
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("news,kind", [(1, "bf16"), (1, "f16"), (90, "bf16")])
def test_scores_that_grow_and_one_key_that_takes_all(news, kind):
    """A maximum that rises along the keys, far past what one exponent range holds, rising and falling."""
    mmq = require_gpu()
    d = make(mmq, [news] * 2, [3000, 1700], 8, 2, 128, 16, kind, 21)
    for flip in (False, True):
        for b, n in enumerate((3000, 1700)):
            i = torch.arange(n, device="cuda")
            slots = (d["page_table"][b, i // 16] * 16 + i % 16).to(torch.int32)
            ramp = torch.linspace(0.1, 12, n, device="cuda")
            k = d["q"][0, 0].float() * (ramp.flip(0) if flip else ramp)[:, None, None] * torch.ones((1, 2, 1), device="cuda")
            mmq.kv4_write(k, torch.randn((n, 2, 128), device="cuda"), slots, d["cache"])
        check(call(mmq, d), d)


@pytest.mark.parametrize("news", [1, 60])
@pytest.mark.parametrize("size", [1e2, 1e5, 1e18, 1e36])
def test_finite_scores_of_any_size(size, news):
    """Large queries: the largest score takes all, whatever its size, and rows of zeros among them stay even."""
    mmq = require_gpu()
    d = make(mmq, [news] * 3, [100, 61, 333], 4, 2, 64, 16, "bf16", 23)
    d["q"] = (d["q"].float() * size).to(torch.bfloat16)
    d["q"][::2, 1] = 0
    got = call(mmq, d)
    assert torch.isfinite(got).all()
    if size < 1e3:
        check(got, d)
        return
    ref, _ = reference(d)
    close = ((got.double() - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -9).all(-1)
    assert close[::2, 1].all()
    # all weight is on one key, but where the two largest scores are nearer than f32 sums tell (24 x 64 x 2^-23 of them)
    at = 0
    for b, n in enumerate(d["lens"].tolist()):
        i = torch.arange(n, device="cuda")
        k, _ = layout.values(d["cache"], d["page_table"][b, i // 16] * 16 + i % 16)
        for j in range(news):
            s = torch.einsum("hgd,nhd->hgn", d["q"][at].double().view(2, 2, 64), k[:n - news + 1 + j]).view(4, -1)
            top = s.topk(2).values
            clear = top[:, 0] - top[:, 1] > 2.0 ** -10 * s.abs().amax(-1)
            assert close[at][clear].all()
            at += 1


def test_tiny_queries_and_tiny_values():
    mmq = require_gpu()
    d = make(mmq, [1, 2], [100, 61], 4, 2, 64, 16, "bf16", 24, k_scale=1e-3)
    d["q"] = (d["q"].float() * 1e-38).to(torch.bfloat16)
    check(call(mmq, d), d)
    d["q"] = torch.full_like(d["q"], 1e-3)
    check(call(mmq, d), d)


def test_long_tail_under_one_key():
    """Many keys far under one that takes most: their weights are not lost."""
    mmq = require_gpu()
    n = 40000
    d = make(mmq, [1], [n], 1, 1, 64, 64, "f16", 25)
    i = torch.arange(n, device="cuda")
    slots = (d["page_table"][0, i // 64] * 64 + i % 64).to(torch.int32)
    k = torch.zeros((n, 1, 64), device="cuda")
    k[n // 3] = 1.0
    v = torch.ones((n, 1, 64), device="cuda")
    v[n // 3] = -1.0
    mmq.kv4_write(k, v, slots, d["cache"])
    d["q"] = torch.full((1, 1, 64), 1.0, dtype=torch.float16, device="cuda")
    for gap in (8.0, 10.5, 14.0):
        out = torch.empty((1, 1, 64), device="cuda")
        call(mmq, d, out=out, scale=gap / 64)
        check(out, d, gap / 64, weight_unit=2.0 ** -22)


def test_strides_and_another_stream():
    mmq = require_gpu()
    d = make(mmq, [1] * 40, [1 + i for i in range(40)], 8, 2, 128, 16, "f16", 31)
    plain = call(mmq, d).clone()
    fused = torch.randn((40, 12, 128), device="cuda").half()
    fused[:, :8] = d["q"]
    d["q"] = fused[:, :8]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(mmq, d, stream=side)
    side.synchronize()
    assert torch.equal(got, plain) and mmq.status() == 0


def test_pages_past_32_bit_offsets():
    mmq = require_gpu()
    d = make(mmq, [1, 3], [40, 33], 4, 4, 128, 16, "f16", 41)
    pages = 240_000   # x 4 x 2304 bytes: past 2^31
    big = torch.empty((pages,) + d["cache"].shape[1:], dtype=torch.uint8, device="cuda")
    big[pages - d["cache"].shape[0]:] = d["cache"]
    d["page_table"] = d["page_table"] + pages - d["cache"].shape[0]
    d["cache"] = big
    check(call(mmq, d), d)
    assert mmq.status() == 0


def test_bad_pages_lengths_and_starts_are_reported():
    mmq = require_gpu()
    d = make(mmq, [1, 1, 1], [20, 20, 20], 8, 2, 64, 16, "f16", 51)
    fill(mmq, d)
    clean = call(mmq, d).clone()
    for bad in (-1, d["cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        table = d["page_table"].clone()
        table[1, 1] = bad
        got = call(mmq, dict(d, page_table=table))
        assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
        assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
        zeros = dict(d, cache=torch.cat([d["cache"], torch.zeros_like(d["cache"][:1])]))
        zeros["page_table"] = table.clone()
        zeros["page_table"][1, 1] = d["cache"].shape[0]
        check(got, zeros)
    room = d["page_table"].shape[1] * 16
    got = call(mmq, dict(d, lens=torch.tensor([20, room + 1, -5], dtype=torch.int32, device="cuda")))
    assert mmq.status() == mmq.MMQ_ERR_ARG
    check(got, dict(d, lens=torch.tensor([20, room, 0], dtype=torch.int32, device="cuda")))
    for starts in ([0, 1, 0, 3], [0, 1, 2, 4], [-1, 1, 2, 3], [0, 2 ** 31 - 1, 2, 3]):
        out = torch.full_like(clean, 5)
        call(mmq, dict(d, q_starts=torch.tensor(starts, dtype=torch.int32, device="cuda")), out=out)
        assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
        for b in range(3):   # a sequence of one row that lies in order
            if starts[b + 1] == starts[b] + 1 and 0 <= starts[b] and starts[b + 1] <= 3:
                assert torch.isfinite(out[starts[b]]).all() and not (out[starts[b]] == 5).all()


def test_runs_are_bit_identical_and_workspace_may_be_given():
    mmq = require_gpu()
    for news in (1, 7, 100):
        d = make(mmq, [news] * 16, [news + 100 * i for i in range(16)], 32, 8, 128, 16, "f16", 61)
        a = call(mmq, d).clone()
        ws = torch.full((200 << 20,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(call(mmq, d, workspace=ws), a)
        with pytest.raises(mmq.MMQError) as e:
            call(mmq, d, workspace=ws[:1024])
        assert e.value.code == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("news", [1, 50])
def test_captured_and_replayed(news):
    """One graph over changing inputs, its tokens' lengths among them."""
    mmq = require_gpu()
    d = make(mmq, [news] * 4, [60, 100, 301, 75], 8, 2, 128, 16, "bf16", 71)
    fill(mmq, d)
    out = torch.empty_like(d["q"])
    call(mmq, d, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(mmq, d, out=out)
    for lens in ([60, 100, 301, 75], [50, 90, 77, 310], [99, 50, 51, 52]):
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        d["q"].normal_()
        out.fill_(9)
        graph.replay()
        check(out, d)
    assert mmq.status() == 0


def test_no_sequences():
    mmq = require_gpu()
    d = make(mmq, [1], [20], 8, 2, 64, 16, "f16", 51)
    none = mmq.kv4_attention(d["q"][:0], d["cache"], d["page_table"][:0], d["lens"][:0])
    assert none.shape == (0, 8, 64)
    none = mmq.kv4_attention(d["q"][:0], d["cache"], d["page_table"], d["lens"], q_starts=torch.zeros_like(d["q_starts"]))
    assert none.shape == (0, 8, 64)
