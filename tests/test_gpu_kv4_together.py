"""The 4-bit cache's operators as a serving loop uses them: prompts in chunks,
decode steps, forks, ended sequences and a compacted pool."""
import pytest

from tests import kv4_layout as layout
from tests.gpu_util import require_gpu
from tests.test_gpu_kv4_attention import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Serving:
    """Two layers' caches over one pool of pages, and the sequences' tables."""

    def __init__(self, mmq, pages=96, batch=6, width=12, heads=8, kv=2, D=64, page=16):
        self.mmq, self.page, self.kv, self.D, self.heads, self.pages = mmq, page, kv, D, heads, pages
        self.caches = [mmq.empty_kv4_cache(pages, kv, D, page).random_(0, 256) for _ in range(2)]
        self.table = torch.zeros((batch, width), dtype=torch.int32)
        self.lens = [0] * batch
        self.free = list(range(pages))[::-1]
        self.g = torch.Generator(device="cuda").manual_seed(5)

    def dev(self, x):
        return torch.as_tensor(x, dtype=torch.int32).cuda()

    def step(self, news):
        """News tokens per sequence: their keys and values written, their attention checked in both layers."""
        slots = []
        for b, n in enumerate(news):
            for i in range(self.lens[b], self.lens[b] + n):
                if i % self.page == 0:
                    self.table[b, i // self.page] = self.free.pop()
                slots.append(int(self.table[b, i // self.page]) * self.page + i % self.page)
            self.lens[b] += n
        T = len(slots)
        starts = [0]
        for n in news:
            starts.append(starts[-1] + n)
        outs = []
        for cache in self.caches:
            k, v, q = (torch.randn((T, h, self.D), device="cuda", generator=self.g).half() for h in (self.kv, self.kv, self.heads))
            self.mmq.kv4_write(k, v, self.dev(slots), cache)
            d = dict(q=q, cache=cache, page_table=self.table.cuda(), lens=self.dev(self.lens), q_starts=self.dev(starts))
            outs.append(self.mmq.kv4_attention(q, cache, d["page_table"], d["lens"], q_starts=d["q_starts"]))
            check(outs[-1], d)
        return outs

    def contents(self, b):
        i = torch.arange(self.lens[b], device="cuda")
        slots = (self.table[b].cuda()[i // self.page] * self.page + i % self.page).to(torch.int32)
        return [x for cache in self.caches for x in self.mmq.kv4_read(cache, slots)]


def test_a_serving_loop():
    mmq = require_gpu()
    s = Serving(mmq)
    s.step([37, 5, 64, 0, 0, 0])
    for _ in range(3):
        s.step([1, 1, 1, 0, 0, 0])
    # sequence 3 forks from 0, 4 from 2: full pages are shared, the last one is copied in both layers
    src, dst = [], []
    for parent, child in ((0, 3), (2, 4)):
        s.table[child] = s.table[parent]
        s.lens[child] = s.lens[parent]
        if s.lens[parent] % s.page:
            src.append(int(s.table[parent, s.lens[parent] // s.page]))
            dst.append(s.free.pop())
            s.table[child, s.lens[parent] // s.page] = dst[-1]
    mmq.pages_copy(s.caches, s.dev(src), s.dev(dst))
    for a, b in ((0, 3), (2, 4)):
        assert all(torch.equal(x, y) for x, y in zip(s.contents(a), s.contents(b)))
    parent = s.contents(0)
    s.step([0, 0, 0, 1, 2, 0])
    assert all(torch.equal(x, y) for x, y in zip(parent, s.contents(0)))   # the child's tokens are not its parent's
    # 1 and 2 end; what is left moves to the front and reads the same
    s.lens[1] = s.lens[2] = 0
    before = [s.contents(b) for b in (0, 3, 4)]
    table, page_map, live = mmq.pages_compact(s.caches, s.table.cuda(), s.dev(s.lens), s.page)
    n = int(live)
    held = {int(p) for b in (0, 3, 4) for p in s.table[b, :-(-s.lens[b] // s.page)]}
    assert n == len(held)
    s.table = table.cpu().clamp_min(0)
    assert {int(p) for b in (0, 3, 4) for p in s.table[b, :-(-s.lens[b] // s.page)]} == set(range(n))
    for b, was in zip((0, 3, 4), before):
        assert all(torch.equal(x, y) for x, y in zip(was, s.contents(b)))
    s.free = list(range(n, s.pages))[::-1]
    s.step([1, 20, 1, 1, 1, 1])
    assert mmq.status() == 0


def test_behind_the_head_norms_and_before_shared_prefix_attention():
    """qk_norm_rope leaves 16-bit rows, kv4_write takes them; a document in the 4-bit cache, expanded, is the prefix of a
    batch, and gives what the pages give."""
    mmq = require_gpu()
    T, heads, kv, D, page = 200, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    qkv = torch.randn((T, (heads + 2 * kv) * D), device="cuda", generator=g)
    angle = torch.arange(256, device="cuda")[:, None] * 10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    k, v = torch.empty((2, T, kv, D), dtype=torch.float16, device="cuda")
    q = mmq.qk_norm_rope(qkv, heads, angle.cos(), angle.sin(), rows, rows, k, v)
    cache = mmq.empty_kv4_cache(20, kv, D, page)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    slots = (table[rows.cpu().long() // page] * page + rows.cpu() % page).to(torch.int32).cuda()
    mmq.kv4_write(k, v, slots, cache)
    d = dict(q=q, cache=cache, page_table=table[None, :13].cuda().contiguous(), lens=torch.tensor([T], dtype=torch.int32, device="cuda"),
             q_starts=torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    check(mmq.kv4_attention(q, cache, d["page_table"], d["lens"]), d)
    kq, vq = mmq.kv4_read(cache, slots)
    want = layout.values(cache, slots)
    assert torch.equal(kq.double(), want[0]) and torch.equal(vq.double(), want[1])
    # rounding errors of the cache: half a step of each block, and one part in 256 of the scale
    step = kq.float().unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True) / 8
    off = (kq.float() - k.float()).unflatten(-1, (4, 32)).abs()
    # -8 d is the block's largest; on the other side 7 d is the last code, up to a whole step under the largest
    assert (off <= step * (1 + 2.0 ** -7) * 1.02).all()
    batch = 5
    qs = torch.randn((batch, heads, D), device="cuda", generator=g).half()
    own = torch.empty((batch, page, kv, D), dtype=torch.float16, device="cuda")
    nothing = torch.zeros(batch, dtype=torch.int32, device="cuda")
    shared = mmq.shared_prefix_attention(qs, kq, vq, own, own, torch.arange(batch, dtype=torch.int32, device="cuda")[:, None].contiguous(), nothing)
    paged = mmq.kv4_attention(qs, cache, d["page_table"].expand(batch, -1).contiguous(), torch.full_like(nothing, T))
    # both are within their weights' rounding (2^-11 of sum w |v| here) of the same values
    bound = 4 * 2.0 ** -11 * vq.float().abs().amax()
    assert (shared.float() - paged.float()).abs().max() <= bound
    assert mmq.status() == 0
