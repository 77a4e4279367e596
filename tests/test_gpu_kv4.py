"""The 4-bit key/value cache: what is written and read, bit for bit, against
the format's definition in 64 bits."""
import pytest

from tests import kv4_layout as layout
from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KIND = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def normal(*shape, seed=1):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def empty(mmq, pages, kv, D, page):
    cache = mmq.empty_kv4_cache(pages, kv, D, page)
    return cache.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(9))


def check_written(cache, before, k, v, slots):
    """The slots hold k and v as the definition has them, every other byte is as it was."""
    kq, ks, vq, vs = layout.codes_and_scales(cache, slots)
    for got_q, got_s, x in ((kq, ks, k), (vq, vs, v)):
        q, s = layout.quantize(x)
        assert torch.equal(got_s.nan_to_num(1e9), s.nan_to_num(1e9))
        assert torch.equal(got_q, q)
    pages, kv, tiles, size = cache.shape
    touched = torch.zeros(cache.numel(), dtype=torch.bool, device="cuda")
    a, b, c, d, _ = layout.places(slots, kv, 16 * tiles, size // 18)
    for at in (a, b, b + 1, c, d, d + 1):
        touched[at.flatten()] = True
    assert torch.equal(cache.view(-1)[~touched], before.view(-1)[~touched])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,kv,page,order", [
    (1, 1, 16, "any"), (5, 8, 16, "any"), (16, 2, 16, "row"), (17, 3, 32, "row"), (100, 2, 64, "any"),
    (333, 4, 128, "row"), (333, 1, 16, "late"), (31, 2, 32, "late")])
def test_written_bytes(T, kv, page, order, kind, D):
    mmq = require_gpu()
    pages = -(-T // page) + 2
    cache = empty(mmq, pages, kv, D, page)
    before = cache.clone()
    k, v = (normal(T, kv, D, seed=s).to(KIND[kind]) for s in (1, 2))
    k[..., 3] *= 20
    if order == "any":
        slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T].to(torch.int32).cuda()
    else:   # one after the other, from a tile's start or from its middle
        slots = torch.arange(T, dtype=torch.int32, device="cuda") + (0 if order == "row" else 11)
    mmq.kv4_write(k, v, slots, cache)
    assert mmq.status() == 0
    check_written(cache, before, k, v, slots)


def test_borders_between_codes():
    """float32 values at, just under and just over every border of every scale sign, and the largest values."""
    mmq = require_gpu()
    rows = []
    for top in (8.0, -8.0, 7.96875, -1.0, 3e-5, 1e-7, 60000.0, -65504.0):
        d = float((torch.tensor(top) / -8).to(torch.bfloat16).to(torch.float16))
        edges = torch.tensor([(n + 0.5) * d for n in range(-8, 8)], dtype=torch.float64).float()
        for x in (edges, torch.nextafter(edges, torch.full_like(edges, 1e30)), torch.nextafter(edges, torch.full_like(edges, -1e30))):
            row = torch.cat([x, x.flip(0) * 0.999])
            row = row.clamp(-abs(top), abs(top))
            row[17] = top
            rows.append(row)
    x = torch.stack(rows).cuda()                 # [24][32]
    x = torch.cat([x, x.flip(0)]).view(-1, 1, 64)
    T = x.shape[0]
    cache = empty(mmq, 4, 1, 64, 16)
    before = cache.clone()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    v = x.flip(0).contiguous()
    mmq.kv4_write(x, v, slots, cache)
    check_written(cache, before, x, v, slots)


def test_zeros_large_values_and_no_numbers():
    mmq = require_gpu()
    x = torch.zeros((6, 1, 128), device="cuda")
    x[1] = 3e38
    x[2, 0, 5] = -3e38
    x[3, 0, 40] = float("nan")
    x[4, 0, 70] = float("inf")
    x[5, 0, 100] = float("-inf")
    x[5, 0, :32] = 1e-30
    cache = empty(mmq, 1, 1, 128, 16)
    before = cache.clone()
    slots = torch.tensor([3, 0, 15, 8, 7, 1], dtype=torch.int32, device="cuda")
    mmq.kv4_write(x, x, slots, cache)
    check_written(cache, before, x, x, slots)
    k, v = mmq.kv4_read(cache, slots)
    assert torch.equal(k[0], torch.zeros_like(k[0])) and (k[1] == 65280).all() and float(k[2, 0, 5]) == -65280
    bad = torch.isnan(k).view(6, 4, 32)
    assert bad.all(-1).nonzero().tolist() == [[3, 1], [4, 2], [5, 3]] and torch.equal(bad.all(-1), bad.any(-1))
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,kv,page", [(1, 1, 16), (7, 8, 16), (16, 2, 32), (50, 3, 64), (333, 2, 16), (4097, 1, 64)])
def test_read(T, kv, page, D):
    mmq = require_gpu()
    pages = -(-T // page) + 1
    cache = empty(mmq, pages, kv, D, page)
    k, v = (normal(pages * page, kv, D, seed=s) for s in (1, 2))
    mmq.kv4_write(k, v, torch.arange(pages * page, dtype=torch.int32, device="cuda"), cache)
    for slots in (torch.arange(T, dtype=torch.int32, device="cuda") + 1,
                  torch.randint(0, pages * page, (T,), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()):
        want = layout.values(cache, slots)
        for kind in (torch.float16, torch.float32, torch.bfloat16):
            got = mmq.kv4_read(cache, slots, kind)
            for a, b in zip(got, want):
                assert a.dtype is kind and torch.equal(a, b.to(kind))   # exact in the first two, rounded once in the last
    assert mmq.status() == 0


def test_slots_out_of_range_and_left_out():
    mmq = require_gpu()
    cache = empty(mmq, 2, 2, 64, 16)
    k, v = (normal(6, 2, 64, seed=s).half() for s in (1, 2))
    before = cache.clone()
    slots = torch.tensor([-1, 4, 32, 31, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    mmq.kv4_write(k, v, slots, cache)
    assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
    check_written(cache, before, k[[1, 3]], v[[1, 3]], slots[[1, 3]])
    a, b = mmq.kv4_read(cache, slots)
    assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
    for x in (a, b):
        assert (x[[0, 2, 4, 5]] == 0).all() and (x[[1, 3]] != 0).any()
    slots[2] = slots[5] = -7   # left out without a word
    mmq.kv4_write(k, v, slots, cache)
    mmq.kv4_read(cache, slots)
    assert mmq.status() == 0


def test_strided_inputs_given_outputs_and_another_stream():
    mmq = require_gpu()
    fused = normal(40, 12, 128).to(torch.bfloat16)         # rows of a fused projection: 8 query, 2 key, 2 value heads
    k, v = fused[:, 8:10], fused[:, 10:]
    slots = torch.randperm(64)[:40].to(torch.int32).cuda()
    plain = torch.zeros((4, 2, 1, 18 * 128), dtype=torch.uint8, device="cuda")
    cache = plain.clone()
    mmq.kv4_write(k.contiguous(), v.contiguous(), slots, plain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mmq.kv4_write(k, v, slots, cache, stream=side)
    out = torch.empty((2, 40, 2, 128), dtype=torch.bfloat16, device="cuda")
    got = mmq.kv4_read(cache, slots, out=(out[0], out[1]), stream=side)
    side.synchronize()
    assert torch.equal(cache, plain) and got[0].data_ptr() == out.data_ptr()
    headfirst = k.transpose(0, 1).contiguous().transpose(0, 1)
    mmq.kv4_write(headfirst, v, slots, cache)
    assert torch.equal(cache, plain)
    for a, b in zip(mmq.kv4_read(plain, slots, torch.bfloat16), out):
        assert torch.equal(a, b)


def test_past_32_bit_offsets():
    mmq = require_gpu()
    pages = 130_000       # x 2 x 4 x 2304 bytes: past 2^31
    cache = torch.empty((pages, 2, 4, 18 * 128), dtype=torch.uint8, device="cuda")
    slots = (torch.arange(70, dtype=torch.int32, device="cuda") * 64 + (pages - 70) * 64 + 5)
    k, v = (normal(70, 2, 128, seed=s).half() for s in (1, 2))
    mmq.kv4_write(k, v, slots, cache)
    got = mmq.kv4_read(cache, slots)
    assert mmq.status() == 0
    for x, y in zip(got, (k, v)):
        q, d = layout.quantize(y)
        assert torch.equal(x, ((q - 8) * d).half())


def test_no_tokens():
    mmq = require_gpu()
    cache = empty(mmq, 1, 2, 64, 16)
    before = cache.clone()
    none = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    slots = torch.empty(0, dtype=torch.int32, device="cuda")
    mmq.kv4_write(none, none, slots, cache)
    k, v = mmq.kv4_read(cache, slots)
    assert k.shape == v.shape == (0, 2, 64) and torch.equal(cache, before)
