"""Calls of the 4-bit cache's operators as programs make them: many at once, on
several streams, in graphs that share memory, behind one another with
programmatic launch, on tensors that are aligned to no more than they have to."""
import pytest

from tests import kv4_layout as layout
from tests.gpu_util import require_gpu
from tests.test_gpu_kv4 import check_written, empty, normal
from tests.test_gpu_kv4_attention import call, check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# a call of each kernel: eight and sixteen rows, 128 rows by two streams, 256 rows, and one of both kinds
CALLS = [
    ([1] * 5, [1, 16, 33, 100, 2570], 32, 8, 128, 64, "bf16"),
    ([2] * 30, [37 * i % 900 + 2 for i in range(30)], 16, 2, 64, 16, "f16"),
    ([9] * 17, [211 * i % 1500 + 9 for i in range(17)], 28, 4, 128, 32, "bf16"),
    ([500, 20], [1500, 800], 16, 4, 64, 64, "bf16"),
    ([900], [5000], 8, 2, 128, 128, "f16"),
    ([1, 40, 2, 7], [300, 300, 41, 900], 12, 4, 128, 16, "f16"),
]


@pytest.mark.parametrize("news,lens,heads,kv,D,page,kind", [
    ([1] * 3000, [i % 41 for i in range(3000)], 2, 1, 64, 16, "f16"),          # more sequences than threads
    ([5] * 700, [5 + i % 30 for i in range(700)], 16, 2, 128, 16, "bf16"),
    ([1] * 3, [700, 1, 64], 48, 1, 128, 32, "f16"),                            # 48 query heads to a kv head
    ([1, 1, 0, 0], [300, 65, 9, 9], 130, 1, 64, 16, "bf16"),                   # more rows than a unit of 128
    ([1, 2], [300, 65], 600, 2, 128, 16, "f16"),                               # and than one of 256
    ([77, 300], [1000, 300], 6, 2, 64, 256, "bf16"),                           # large pages
    ([64, 64, 64], [64, 65, 129], 4, 1, 128, 1024, "f16"),                     # a page past the sequence
])
def test_values_of_more_shapes(news, lens, heads, kv, D, page, kind):
    mmq = require_gpu()
    d = make(mmq, news, lens, heads, kv, D, page, kind, 7)
    got = call(mmq, d)
    assert mmq.status() == 0
    check(got, d)
    check(call(mmq, d, out=torch.empty(d["q"].shape, device="cuda")), d)


@pytest.mark.parametrize("c", CALLS)
def test_repeated_calls_are_bit_identical(c):
    """Hundreds of calls: no sum depends on who comes first."""
    mmq = require_gpu()
    d = make(mmq, *c, 11)
    want = call(mmq, d).clone()
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        bad += (call(mmq, d) != want).sum()
    assert int(bad) == 0 and mmq.status() == 0


def test_calls_on_several_streams_at_once():
    mmq = require_gpu()
    ds = [make(mmq, *c, 20 + i) for i, c in enumerate(CALLS)]
    want = [call(mmq, d).clone() for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    outs = [[] for _ in ds]
    for _ in range(20):
        for i, (d, s) in enumerate(zip(ds, streams)):
            with torch.cuda.stream(s):
                outs[i].append(call(mmq, d))
    torch.cuda.synchronize()
    assert mmq.status() == 0
    assert all(torch.equal(o, w) for os, w in zip(outs, want) for o in os)


def test_graphs_that_share_a_workspace():
    """Replayed in turn on one stream: each call's parts are written before they are read."""
    mmq = require_gpu()
    ds = [make(mmq, *c, 30 + i) for i, c in enumerate(CALLS)]
    want = [call(mmq, d).clone() for d in ds]
    workspace = torch.full((200 << 20,), 255, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for d in ds:
        out = torch.empty_like(d["q"])
        call(mmq, d, out=out, workspace=workspace)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(mmq, d, out=out, workspace=workspace)
        graphs.append(g)
        outs.append(out)
    for order in ([0, 1, 2, 3, 4, 5], [5, 4, 3, 2, 1, 0], [0, 3, 0, 5, 2, 2, 4, 1]):
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], want[i])
    assert mmq.status() == 0


def test_a_chain_with_programmatic_launch():
    """Each kernel starts before the one ahead has finished, and takes what that wrote."""
    mmq = require_gpu()
    kv, D, page, pages = 4, 128, 16, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((3, 16, D), device="cuda", generator=g).half()
    news = [torch.randn((2, 3, kv, D), device="cuda", generator=g).half() for _ in range(12)]
    table = torch.randperm(36, device="cuda", generator=g).view(3, 12).to(torch.int32)

    def run():
        cache = mmq.empty_kv4_cache(pages, kv, D, page).zero_()
        t, outs = table, []
        for step, (k, v) in enumerate(news):
            at = 15 * step
            lens = torch.full((3,), at + 1, dtype=torch.int32, device="cuda")
            slots = t[:, at // page] * page + at % page
            mmq.kv4_write(k, v, slots, cache)
            outs.append(mmq.kv4_attention(q, cache, t, lens))
            outs.append(torch.cat(mmq.kv4_read(cache, slots)))
            if step % 4 == 3:
                t, _, live = mmq.pages_compact([cache], t, torch.full((3,), 192, dtype=torch.int32, device="cuda"), page)
                mmq.pages_copy([cache], t[0, :1], live)
        return outs

    want = run()
    mmq.mmq_set_programmatic_launch(True)
    try:
        got = run()
    finally:
        mmq.mmq_set_programmatic_launch(False)
    assert mmq.status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_addresses_aligned_to_16_bytes_only(kind, D):
    """Inputs and outputs that start 16 bytes past a multiple of 32, and rows that do so in turn."""
    mmq = require_gpu()
    T, kv, page = 70, 3, 16
    off = 16 // torch.empty((), dtype=kind).element_size()
    k, v = normal(2, T, kv, D)
    slots = torch.arange(5, 5 + T, dtype=torch.int32, device="cuda")

    def shifted(x):
        y = torch.empty(x.numel() + off, dtype=kind, device="cuda")[off:].view(T, kv, D)
        return y.copy_(x)

    ks, vs = shifted(k), shifted(v)
    assert ks.data_ptr() % 32 == 16
    cache = empty(mmq, 6, kv, D, page)
    before = cache.clone()
    mmq.kv4_write(ks, vs, slots, cache)
    check_written(cache, before, ks, vs, slots)
    want = mmq.kv4_read(cache, slots, dtype=kind)
    got = mmq.kv4_read(cache, slots, out=(shifted(k), shifted(v)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if kind is not torch.float32:   # eight values between rows: strides of 16 bytes
        wide = torch.randn((T, kv, D + 8), device="cuda").to(kind)[:, :, :D]
        mmq.kv4_write(wide, wide, slots, cache)
        check_written(cache, before, wide, wide, slots)
    assert mmq.status() == 0


def test_whole_tiles_in_other_orders():
    """A chunk that starts inside a tile, tiles out of order, and one whose tokens are in order but not its tile's."""
    mmq = require_gpu()
    kv, D, page = 2, 64, 32
    places = list(range(9, 64)) + list(range(96, 112)) + list(range(64, 80)) + list(range(121, 137)) + [-1] * 3 + list(range(144, 160))
    slots = torch.tensor(places, dtype=torch.int32, device="cuda")
    k, v = normal(2, len(places), kv, D)
    cache = empty(mmq, 6, kv, D, page)
    before = cache.clone()
    mmq.kv4_write(k, v, slots, cache)
    here = slots >= 0
    check_written(cache, before, k[here], v[here], slots[here])
    a, b = mmq.kv4_read(cache, slots, dtype=torch.float32)
    kq, ksc, vq, vsc = layout.codes_and_scales(cache, slots.clamp_min(0))
    here = here[:, None, None]
    assert torch.equal(a.double(), torch.where(here, (kq - 8) * ksc, 0.0))
    assert torch.equal(b.double(), torch.where(here, (vq - 8) * vsc, 0.0))
    assert mmq.status() == 0


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
@pytest.mark.parametrize("news,kind", [([1, 1, 1], "f16"), ([3, 0, 9], "bf16"), ([60, 1, 31], "f16"), ([300, 5, 1], "bf16"),
                                       ([257, 64, 65], "f16")])
def test_a_padded_batch_of_strided_queries(news, kind, out_dtype):
    """Rows before the first sequence and behind the last: not read (they hold NaN), and left as they were."""
    mmq = require_gpu()
    d = make(mmq, news, [n + 70 * i for i, n in enumerate(news)], 8, 2, 64, 32, kind, 9)
    T, heads, D = d["q"].shape
    wide = torch.full((T + 9, heads, 2 * D), float("nan"), dtype=d["q"].dtype, device="cuda").view(T + 9, heads * 2, D)
    q = wide[:, :heads]
    q[2:2 + T] = d["q"]
    out = torch.full((T + 9, heads, D), 7.0, dtype=out_dtype or q.dtype, device="cuda")
    mmq.kv4_attention(q, d["cache"], d["page_table"], d["lens"], q_starts=d["q_starts"] + 2, out=out)
    assert mmq.status() == 0
    assert (out[:2] == 7).all() and (out[2 + T:] == 7).all()
    check(out[2:2 + T], d)


def test_one_long_sequence_of_each_form_past_many_short_ones():
    """Units of one step and of hundreds side by side: cuts between runs anywhere in the layout."""
    mmq = require_gpu()
    for seed, (long, new) in enumerate([(9000, 1), (9000, 12), (5000, 70), (5000, 300)]):
        news = [1] * 40 + [new] + [1, 0, 2] * 11
        lens = [1 + i % 5 for i in range(40)] + [long] + [3 + i % 7 for i in range(33)]
        d = make(mmq, news, lens, 8, 2, 128, 16, "bf16" if seed % 2 else "f16", 50 + seed)
        got = call(mmq, d)
        assert mmq.status() == 0
        check(got, d)
        assert torch.equal(call(mmq, d), got)
