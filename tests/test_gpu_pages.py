"""Page copies and compaction, exactly, against plain loops on the host."""
import random

import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def pool(n, pages, shape, dtype=torch.uint8, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    raw = torch.randint(0, 256, (n, pages) + shape[:-1] + (shape[-1] * dtype.itemsize,), dtype=torch.uint8, device="cuda", generator=g)
    return list(raw.view(dtype).unbind())


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("n,pages,shape,dtype", [
    (1, 4, (16,), torch.uint8), (3, 40, (16, 8, 128), torch.float16), (64, 20, (2, 1, 1152), torch.uint8),
    (2, 12, (64, 8, 128), torch.bfloat16), (1, 9, (33000,), torch.float32), (256, 6, (48,), torch.uint8)])
def test_copy(n, pages, shape, dtype):
    mmq = require_gpu()
    caches = pool(n, pages, shape, dtype)
    before = [c.clone() for c in caches]
    order = list(range(pages))
    random.Random(pages).shuffle(order)
    m = pages // 2
    src, dst = order[:m], order[m:2 * m]
    src[0] = src[-1]                       # a source may be one twice
    mmq.pages_copy(caches, torch.tensor(src, dtype=torch.int32, device="cuda"), torch.tensor(dst, dtype=torch.int32, device="cuda"))
    assert mmq.status() == 0
    for a, b in zip(before, caches):
        for s, d in zip(src, dst):
            a[d] = a[s]
    assert same(before, caches)


def test_pairs_left_out_and_out_of_range():
    mmq = require_gpu()
    caches = pool(2, 8, (64,))
    before = [c.clone() for c in caches]
    i32 = dict(dtype=torch.int32, device="cuda")
    mmq.pages_copy(caches, torch.tensor([-1, 2, 3], **i32), torch.tensor([1, -2 ** 31, 3], **i32))
    assert mmq.status() == 0 and same(before, caches)
    mmq.pages_copy(caches, torch.tensor([8, 2, 0, 2 ** 31 - 1], **i32), torch.tensor([1, 8, 5, -1], **i32))
    assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
    for c in before:
        c[5] = c[0]
    assert same(before, caches)
    none = torch.empty(0, **i32)
    mmq.pages_copy(caches, none, none)
    mmq.pages_copy([], none, none)
    assert mmq.status() == 0 and same(before, caches)


def test_copy_past_32_bit_offsets():
    mmq = require_gpu()
    cache = torch.zeros((70_000, 65536), dtype=torch.uint8, device="cuda")
    cache[5].random_(0, 256)
    i32 = dict(dtype=torch.int32, device="cuda")
    mmq.pages_copy([cache], torch.tensor([5], **i32), torch.tensor([69_999], **i32))
    assert mmq.status() == 0 and torch.equal(cache[5], cache[69_999]) and not cache[69_998].any()


def expected(table, lens, pages, page_size):
    """(table, map, live, moves) by the definition, with lists."""
    width = len(table[0]) if table else 0
    held = [min(max(-(-n // page_size), 0), width) for n in lens]
    live = sorted({p for row, n in zip(table, held) for p in row[:n] if 0 <= p < pages})
    n = len(live)
    holes = [p for p in range(n) if p not in set(live)]
    moves = dict(zip([p for p in live if p >= n], holes))
    new = {p: moves.get(p, p) for p in live}
    return ([[new.get(p, -1) if i < m else -1 for i, p in enumerate(row)] for row, m in zip(table, held)],
            [new.get(p, -1) for p in range(pages)], n, moves)


def compact_and_check(mmq, caches, table, lens, page_size, pages, **more):
    i32 = dict(dtype=torch.int32, device="cuda")
    width = len(table[0]) if table else 0
    want, want_map, n, moves = expected(table, lens, pages, page_size)
    before = [c.clone() for c in caches]
    got, page_map, live = mmq.pages_compact(caches, torch.tensor(table, **i32).view(len(table), width),
                                            torch.tensor(lens, **i32), page_size, pages=pages, **more)
    assert got.tolist() == want and page_map.tolist() == want_map and live.tolist() == [n]
    for c in before:
        for s, d in moves.items():
            c[d] = c[s]
    assert same(before, caches)
    return got


@pytest.mark.parametrize("pages,batch,width,share", [(1, 1, 1, 1.0), (8, 2, 3, 0.5), (31, 3, 9, 0.6), (32, 4, 8, 1.0),
                                                    (33, 4, 8, 0.9), (64, 2, 32, 1.0), (1000, 17, 40, 0.5),
                                                    (5000, 40, 130, 0.2), (70000, 64, 300, 0.25), (100, 5, 20, 0.0)])
def test_compact(pages, batch, width, share):
    mmq = require_gpu()
    rng = random.Random(pages)
    ids = list(range(pages))
    rng.shuffle(ids)
    table, lens, room = [], [], int(pages * share)
    for b in range(batch):
        n = min(width, room, rng.randrange(width + 1) if batch > 1 else width)
        room -= n
        row = [ids.pop() for _ in range(n)] + [rng.randrange(-5, pages + 5) for _ in range(width - n)]
        lens.append(max(0, n * 16 - rng.randrange(16)))
        table.append(row)
        if b % 3 == 1 and min(lens[b], lens[b - 1]) > 16:   # a fork: full pages shared
            k = min(lens[b], lens[b - 1]) // 16
            row[:k] = table[b - 1][:k]
    caches = pool(3, pages, (32,))
    compact_and_check(mmq, caches, table, lens, 16, pages)
    assert mmq.status() == 0


def test_compact_all_live_reversed_and_without_caches():
    mmq = require_gpu()
    for pages in (32, 96, 100):
        caches = pool(2, pages, (16, 4, 64), torch.float16)
        table = [list(range(pages - 1, -1, -1))]
        compact_and_check(mmq, caches, table, [pages * 64], 64, pages)
        table = [list(range(pages - 1, pages // 2 - 1, -1))]    # the upper half
        compact_and_check(mmq, caches, table, [len(table[0]) * 64], 64, pages)
        compact_and_check(mmq, [], table, [len(table[0]) * 64], 64, pages)
    assert mmq.status() == 0


def test_compact_in_place_and_a_given_workspace():
    mmq = require_gpu()
    caches = pool(2, 50, (16,))
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[49, 3, 40], [7, 48, -9]], **i32)
    lens = torch.tensor([33, 20], **i32)
    want, _, n, _ = expected(table.tolist(), lens.tolist(), 50, 16)
    ws = torch.full((4096,), 255, dtype=torch.uint8, device="cuda")
    got, _, live = mmq.pages_compact(caches, table, lens, 16, table_out=table, workspace=ws)
    assert got is table and table.tolist() == want and int(live) == n
    again, _, _ = mmq.pages_compact(caches, table, lens, 16)     # nothing moves any more
    assert torch.equal(again, table)
    with pytest.raises(mmq.MMQError) as e:
        mmq.pages_compact(caches, table, lens, 16, workspace=ws[:256])
    assert e.value.code == mmq.MMQ_ERR_ARG


def test_compact_reports_what_is_out_of_range():
    mmq = require_gpu()
    caches = pool(1, 20, (16,))
    compact_and_check(mmq, caches, [[3, 25, 19], [-1, 2, 4]], [40, 20], 16, 20)
    assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0
    compact_and_check(mmq, caches, [[3, 11, 19], [5, 2, 4]], [49, -7], 16, 20)
    assert mmq.status() == mmq.MMQ_ERR_ARG and mmq.status() == 0


def test_compact_nothing():
    mmq = require_gpu()
    compact_and_check(mmq, pool(1, 20, (16,)), [[3, 11, 19]], [0], 16, 20)
    compact_and_check(mmq, pool(1, 20, (16,)), [[]], [0], 16, 20)
    compact_and_check(mmq, pool(1, 20, (16,)), [], [], 16, 20)
    compact_and_check(mmq, [], [], [], 16, 0)
    assert mmq.status() == 0


def test_captured_and_another_stream():
    mmq = require_gpu()
    caches = pool(4, 64, (16, 2, 64), torch.float16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.zeros((3, 8), **i32), torch.zeros(3, **i32)
    out = torch.empty_like(table)
    src, dst = torch.tensor([-1], **i32), torch.tensor([-1], **i32)
    side = torch.cuda.Stream()

    def step(**more):
        mmq.pages_copy(caches, src, dst, **more)
        return mmq.pages_compact(caches, table, lens, 16, table_out=out, **more)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, page_map, live = step()
    rng = random.Random(4)
    for again in range(3):
        rows = [rng.sample(range(64), 8) for _ in range(3)]
        table.copy_(torch.tensor(rows))
        lens.copy_(torch.tensor([rng.randrange(129) for _ in range(3)]))
        src.fill_(rows[0][0])
        dst.fill_(next(p for p in range(64) if p not in sum(rows, [])))
        before = [c.clone() for c in caches]
        want, want_map, n, moves = expected(rows, lens.tolist(), 64, 16)
        if again < 2:
            graph.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            _, page_map, live = step(stream=side)
            side.synchronize()
        for c in before:
            c[int(dst)] = c[int(src)]
            for s, d in moves.items():
                c[d] = c[s]
        assert out.tolist() == want and page_map.tolist() == want_map and live.tolist() == [n] and same(before, caches)
    assert mmq.status() == 0


def test_a_pool_of_the_largest_size():
    mmq = require_gpu()
    pages = 1 << 20
    caches = [torch.arange(pages, dtype=torch.int64, device="cuda").view(pages, 1).expand(pages, 2).contiguous()]
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randperm(pages, device="cuda", generator=g)[:512 * 1000].view(512, 1000).to(torch.int32)
    lens = torch.randint(0, 16001, (512,), device="cuda", generator=g).to(torch.int32)
    got, page_map, live = mmq.pages_compact(caches, table, lens, 16)
    assert mmq.status() == 0
    used = torch.arange(1000, device="cuda") < ((lens + 15) // 16)[:, None]
    n = int(used.sum())
    assert int(live) == n and int((page_map >= 0).sum()) == n
    assert torch.equal(got[used].sort().values, torch.arange(n, dtype=torch.int32, device="cuda")) and (got[~used] == -1).all()
    assert torch.equal(caches[0][got[used].long(), 0], table[used].long())    # each page's contents went with it
    assert torch.equal(page_map[table[used].long()], got[used])
    with pytest.raises(mmq.MMQError):
        mmq.pages_compact([], table, lens, 16, pages=pages + 1)
