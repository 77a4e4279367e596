"""Programmatic launch through every kernel of the 4-bit attention: calls of all forms, one behind the other, over one
workspace, with writes to the cache and moves of its pages between them, are bit for bit what they are without it."""
import pytest

from tests.gpu_util import require_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# new tokens of three sequences: both kernels in one call, the tensor-core kernel alone (128 rows, 256), few rows alone
STEPS = [[1, 40, 300], [1, 1, 1], [9, 9, 9], [90, 90, 90], [70, 0, 2], [2, 2, 2], [1, 200, 1], [1, 1, 1]]


@pytest.mark.parametrize("kind,out_dtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                            (torch.float16, torch.float32)])
def test_calls_of_all_forms_over_one_workspace(kind, out_dtype):
    mmq = require_gpu()
    kv, heads, D, page, batch, width = 2, 8, 128, 16, 3, 50
    pages = batch * width + 6
    g = torch.Generator(device="cuda").manual_seed(17)
    table = torch.randperm(batch * width, device="cuda", generator=g).view(batch, width).to(torch.int32)
    workspace = torch.zeros(200 << 20, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    todo, lens = [], [0] * batch
    for news in STEPS:
        T = sum(news)
        where = [(b, i) for b, n in enumerate(news) for i in range(lens[b], lens[b] + n)]
        lens = [m + n for m, n in zip(lens, news)]
        todo.append(dict(q=torch.randn((T, heads, D), device="cuda", generator=g).to(kind),
                         kv=torch.randn((2, T, kv, D), device="cuda", generator=g).to(kind),
                         where=torch.tensor(where, device="cuda"), lens=torch.tensor(lens, **i32),
                         starts=torch.tensor([0] + news, device="cuda").cumsum(0).to(torch.int32), alike=len(set(news)) == 1))
    assert max(lens) <= width * page
    outs = [torch.empty(s["q"].shape, dtype=out_dtype, device="cuda") for s in todo for _ in range(2)]

    def run():
        cache = mmq.empty_kv4_cache(pages, kv, D, page).zero_()
        t, full = table.clone(), torch.full((batch,), width * page, **i32)
        kept = []
        for n, s in enumerate(todo):
            slots = (t[s["where"][:, 0], s["where"][:, 1] // page] * page + s["where"][:, 1] % page).to(torch.int32)
            torch.cuda.synchronize()     # from here on, kernels of the library alone
            mmq.kv4_write(s["kv"][0], s["kv"][1], slots, cache)
            for again in range(2):
                mmq.kv4_attention(s["q"], cache, t, s["lens"], q_starts=None if s["alike"] and again else s["starts"],
                                  out=outs[2 * n + again], workspace=workspace)
            mmq.kv4_write(s["kv"][1], s["kv"][0], slots, cache)     # over what the call before still reads, if it may
            mmq.kv4_attention(s["q"], cache, t, s["lens"], q_starts=s["starts"], out=outs[2 * n], workspace=workspace)
            kept.append(mmq.kv4_read(cache, slots))
            t, _, live = mmq.pages_compact([cache], t, full, page, workspace=workspace)
            mmq.pages_copy([cache], t[0, :1], live)
        torch.cuda.synchronize()
        return [x.clone() for x in outs] + [x for pair in kept for x in pair] + [t, cache]

    want = run()
    for _ in range(3):
        for x in outs:
            x.fill_(3)
        workspace.fill_(255)
        mmq.mmq_set_programmatic_launch(True)
        try:
            got = run()
        finally:
            mmq.mmq_set_programmatic_launch(False)
        assert mmq.status() == 0
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("on", [False, True])
def test_a_step_captured_and_replayed(on):
    """A whole step in one graph, its launches programmatic or not: new inputs at each replay, results as of plain calls."""
    mmq = require_gpu()
    kv, heads, D, page, width = 2, 8, 64, 16, 40
    g = torch.Generator(device="cuda").manual_seed(19)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(2 * width, device="cuda", generator=g).view(2, width).to(torch.int32)
    cache = mmq.empty_kv4_cache(2 * width + 2, kv, D, page)
    k, v = torch.empty((2, 310, kv, D), dtype=torch.float16, device="cuda")
    q = torch.empty((310, heads, D), dtype=torch.float16, device="cuda")
    slots, lens = torch.empty(310, **i32), torch.empty(2, **i32)
    starts, last = torch.tensor([0, 3, 310], **i32), torch.tensor([0, 1, 2], **i32)
    moved, free = torch.empty((2, width), **i32), torch.tensor([2 * width], **i32)
    outs = [torch.empty_like(q), torch.empty_like(q[:2]), torch.empty((310, kv, D), dtype=torch.float16, device="cuda"),
            torch.empty((310, kv, D), dtype=torch.float16, device="cuda")]

    def step():
        mmq.kv4_write(k, v, slots, cache)
        mmq.kv4_attention(q, cache, table, lens, q_starts=starts, out=outs[0])
        mmq.kv4_attention(q[:2], cache, table, lens, out=outs[1])
        mmq.kv4_read(cache, slots, out=(outs[2], outs[3]))
        mmq.pages_compact([cache], table, lens, page, table_out=moved)
        mmq.pages_copy([cache], moved[1, :1], free)
        mmq.kv4_attention(q[:3], cache, moved, lens, q_starts=last, out=q[3:6])

    def fill(seed):
        g.manual_seed(seed)
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        cache.random_(0, 16, generator=g)      # scales that are small numbers
        n = [3 + 97 * seed % 400, 307 + 31 * seed % 300]
        lens.copy_(torch.tensor(n))
        at = torch.cat([torch.arange(n[0] - 3, n[0]), torch.arange(n[1] - 307, n[1])]).cuda()
        slots.copy_(table.flatten()[at // page + torch.tensor([0] * 3 + [width] * 307).cuda()] * page + at % page)

    def results():
        torch.cuda.synchronize()
        assert mmq.status() == 0
        return [x.clone() for x in outs + [moved, cache, q]]

    fill(0)
    step()
    torch.cuda.synchronize()
    mmq.mmq_set_programmatic_launch(on)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    finally:
        mmq.mmq_set_programmatic_launch(False)
    for seed in range(1, 6):
        fill(seed)
        step()
        want = results()
        fill(seed)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
