"""The operators of a key/value cache held in 4 bits, as measured: the cases,
their inputs, their plain form in torch, the library's calls and their values
in 64 bits.

  write    quantization of new keys and values into the pages of the cache,
           and the expansion of every slot (so that the outputs are values)
  read     expansion of a sequence's slots to 16 bits
  attn     causal attention of a ragged batch over the 4-bit pages
  copy     copies of pages in the caches of all layers (a fork's last pages)
  compact  live pages moved to the front of every cache, with the page tables

A cache is uint8 [pages][kv_heads][page_size / 16][18 D].  The last dimension
is a tile: 16 tokens of one head, of which 8 D bytes are the keys' codes, D
bytes their scales, then 8 D and D bytes of the values'.  A value is (code - 8)
times its scale, one float16 scale per 32 values of a token.  A byte holds the
codes of dimensions x (low) and x + 8 (high) of a token, x % 16 < 8:

  keys    [D / 64][token % 8][x % 8 / 2][x / 16 % 4][x % 2][token / 8]
  values  [D / 64][x % 8][token % 8 / 2][x / 16 % 4][token % 2][token / 8]

and scales lie as [token % 8][token / 8][block] (keys) and [token % 8 / 2]
[block][token / 8][token % 2] (values).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
TOP = 8160.0   # largest scale: 8 times it is a float16


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a few sequences: latency
        dict(name="write_decode_5", op="write", tokens=5, slots=80, kv_heads=8, dim=128, page=16, type="f16"),
        # a long prefill chunk
        dict(name="write_prefill_8192", op="write", tokens=8192, slots=8256, kv_heads=8, dim=128, page=64, type="bf16"),
        # a ragged prompt with as many kv heads as heads, narrow heads, handed to a kernel that reads 16 bits
        dict(name="read_prompt_5001", op="read", tokens=5001, kv_heads=32, dim=64, page=32, type="bf16"),
        # a long shared document, expanded once for the batch that shares it
        dict(name="read_prefix_32768", op="read", tokens=32768, kv_heads=8, dim=128, page=16, type="f16"),
        # one new token of one sequence: latency only
        dict(name="attn_decode_b1_701", op="attn", batch=1, new=1, context=701, heads=32, kv_heads=8, dim=128, page=16,
             type="f16"),
        # speculative steps of one to five tokens, an odd group of heads
        dict(name="attn_spec_b33_5001", op="attn", batch=33, new=5, context=5001, heads=28, kv_heads=4, dim=128, page=32,
             type="bf16"),
        # a full decode batch over long documents
        dict(name="attn_decode_b64_32k", op="attn", batch=64, new=1, context=32768, heads=32, kv_heads=8, dim=128,
             page=64, type="bf16"),
        # prefill chunks on top of what is cached: tensor-core products
        dict(name="attn_prefill_2047_12k", op="attn", batch=3, new=2047, context=12288, heads=32, kv_heads=8, dim=128,
             page=16, type="f16"),
        # two beams fork: latency
        dict(name="copy_fork_3", op="copy", pairs=3, pages=40, caches=4, kv_heads=8, dim=128, page=16, type="f16"),
        # samples of 64 prompts fork in every layer's keys and values
        dict(name="copy_fork_64", op="copy", pairs=64, pages=256, caches=64, kv_heads=8, dim=128, page=16, type="bf16"),
        # a small pool after a few sequences ended
        dict(name="compact_100", op="compact", pages=100, batch=5, width=20, live=0.4, caches=4, kv_heads=4, dim=64,
             page=16, type="bf16"),
        # a large pool, one quarter of it live, before it is cut down
        dict(name="compact_4096", op="compact", pages=4096, batch=64, width=128, live=0.25, caches=8, kv_heads=4, dim=128,
             page=16, type="f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "copy", "compact"])
    kind = rng.choice(["f16", "bf16"])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64])
    if op == "write":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, slots=-(-(tokens + rng.randrange(64)) // page) * page, kv_heads=kv, dim=dim,
                    page=page, type=kind)
    if op == "read":
        return dict(op=op, tokens=_log(rng, 1, 32768), kv_heads=kv, dim=dim, page=page, type=kind)
    if op == "attn":
        form = rng.choice(["decode", "decode", "spec", "prefill"])
        batch, new, context = {"decode": (_log(rng, 1, 64), 1, _log(rng, 1, 32768)),
                               "spec": (_log(rng, 1, 48), rng.randrange(2, 9), _log(rng, 8, 16384)),
                               "prefill": (rng.randrange(1, 4), _log(rng, 16, 2047), _log(rng, 2047, 12288))}[form]
        return dict(op=op, batch=batch, new=new, context=context, heads=kv * rng.choice([1, 2, 4, 4] if kv == 8 else [1, 3, 4, 8]),
                    kv_heads=kv, dim=dim, page=page, type=kind)
    if op == "copy":
        pairs = _log(rng, 1, 64)
        return dict(op=op, pairs=pairs, pages=2 * pairs + rng.randrange(2, 100), caches=_log(rng, 1, 64), kv_heads=kv,
                    dim=dim, page=16, type=kind)
    batch, width = _log(rng, 1, 64), _log(rng, 1, 128)
    return dict(op=op, pages=max(8, batch * width // 2), batch=batch, width=width, live=rng.choice([0.1, 0.25, 0.4]),
                caches=_log(rng, 1, 8), kv_heads=min(kv, 4), dim=dim, page=16, type=kind)


def _news(c):
    """New tokens of each sequence: `new`, or for several sequences one to `new`."""
    return [1 + (i * 7919 + c["new"] - 1) % c["new"] for i in range(c["batch"])]


def _lens(c):
    """Tokens of each sequence, its new ones among them: ragged, the first as long as the context."""
    return [n + (i * 104729 + c["context"] - c["new"]) % (max(1, c["context"] - c["new"] + 1)) for i, n in enumerate(_news(c))]


def _held(c):
    """Pages of each sequence, as many as `live` of the pool, some sequences with none."""
    room = int(c["live"] * c["pages"])
    held = []
    for i in range(c["batch"]):
        n = min(c["width"], room, (i * 7919 + 3) % (2 * room // c["batch"] + 2))
        held.append(n)
        room -= n
    return held


# ------------------------------------------------------------------ inputs
def _cache(g, pages, kv, page, dim):
    """Pages with codes around the middle, scales near those of values with a deviation of one."""
    c = torch.empty((pages, kv, page // 16, 18 * dim), dtype=torch.uint8, device=DEV)
    for at in range(0, pages, 8192):   # in pieces: a large cache leaves no room for much beside it
        part = c[at:at + 8192]
        a, b = (torch.randint(0, 256, part.shape, device=DEV, generator=g, dtype=torch.uint8) for _ in range(2))
        part.copy_((((a & 15) + (b & 15) + 1) >> 1) | ((((a >> 4) + (b >> 4) + 1) >> 1) << 4))
        for lo in (8 * dim, 17 * dim):
            d = torch.rand(part.shape[:3] + (dim // 2,), device=DEV, generator=g) * 0.15 + 0.2
            d = torch.where(torch.rand(d.shape, device=DEV, generator=g) < 0.5, -d, d)
            part[..., lo:lo + dim] = d.to(torch.bfloat16).to(torch.float16).view(torch.uint8)
    return c


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind, kv, dim, page = TYPES[c["type"]], c["kv_heads"], c["dim"], c["page"]

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    def some(n, of):
        return torch.randperm(of, device=DEV, generator=g)[:n].to(torch.int32)

    if c["op"] == "write":
        k, v = normal(c["tokens"], kv, dim), normal(c["tokens"], kv, dim)
        k *= 1 + 9 * (torch.rand((kv, dim), device=DEV, generator=g) < 0.03).float()   # keys have a few large channels
        pages = c["slots"] // page
        order = some(pages, pages).long()[:, None] * page + torch.arange(page, device=DEV)
        slots = order.flatten().to(torch.int32)   # tokens one after the other in pages anywhere
        first = int(torch.randint(0, c["slots"] - c["tokens"] + 1, (1,), device=DEV, generator=g))
        return dict(case=c, k=k.to(kind), v=v.to(kind), slots=slots[first:first + c["tokens"]].contiguous(), every=slots,
                    cache=torch.zeros((pages, kv, page // 16, 18 * dim), dtype=torch.uint8, device=DEV))
    if c["op"] == "read":
        pages = -(-c["tokens"] // page) + 3
        order = some(pages, pages).long()[:, None] * page + torch.arange(page, device=DEV)
        return dict(case=c, cache=_cache(g, pages, kv, page, dim),
                    slots=order.flatten()[:c["tokens"]].to(torch.int32).contiguous())
    if c["op"] == "attn":
        news, lens = _news(c), _lens(c)
        width = -(-max(lens) // page)
        need = [-(-n // page) for n in lens]
        table = torch.zeros((c["batch"], width), dtype=torch.int32)
        ids = some(sum(need), sum(need)).cpu()
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        starts = [0]
        for n in news:
            starts.append(starts[-1] + n)
        return dict(case=c, q=normal(starts[-1], c["heads"], dim).to(kind), cache=_cache(g, sum(need), kv, page, dim),
                    page_table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                    q_starts=None if c["new"] == 1 else torch.tensor(starts, dtype=torch.int32, device=DEV))
    pool = torch.empty((c["caches"], c["pages"], page, kv, dim), dtype=kind, device=DEV)
    for part in pool:
        part.copy_(normal(*part.shape))
    if c["op"] == "copy":
        ids = some(2 * c["pairs"], c["pages"])
        return dict(case=c, pool=pool, caches=list(pool.unbind()), src=ids[:c["pairs"]].contiguous(),
                    dst=ids[c["pairs"]:].contiguous())
    held = _held(c)
    ids = some(c["pages"], c["pages"]).cpu()
    table = torch.full((c["batch"], c["width"]), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    for b in range(1, c["batch"], 3):   # forks share all but their last page
        n = min(held[b], held[b - 1])
        table[b, :max(0, n - 1)] = table[b - 1, :max(0, n - 1)]
    lens = [max(0, n * page - b % page) for b, n in enumerate(held)]
    return dict(case=c, pool=pool, caches=list(pool.unbind()), page_table=table.to(DEV),
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------- plain forms
def _expand(tile, dim):
    """Tiles [..][18 D] -> keys and values, f32 [..][16][D]."""
    lead = tile.shape[:-1]
    n, blocks = len(lead), dim // 32

    def codes(part, order):   # order: which of the seven axes are token / 8, token % 8 (in parts) and the byte's place
        b = part.reshape(lead + order[0])
        b = b.permute(tuple(range(n)) + tuple(n + i for i in order[1])).reshape(lead + (16, dim // 16, 8))
        return torch.stack([b & 15, b >> 4], dim=-2).flatten(-3).float() - 8

    def scales(part, shape, order):
        s = part.contiguous().view(torch.float16).reshape(lead + shape)
        return s.permute(tuple(range(n)) + tuple(n + i for i in order)).reshape(lead + (16, blocks, 1)).float()

    kq = codes(tile[..., :8 * dim], ((dim // 64, 8, 4, 4, 2, 2), (5, 1, 0, 3, 2, 4)))
    ks = scales(tile[..., 8 * dim:9 * dim], (8, 2, blocks), (1, 0, 2))
    vq = codes(tile[..., 9 * dim:17 * dim], ((dim // 64, 8, 4, 4, 2, 2), (5, 2, 4, 0, 3, 1)))
    vs = scales(tile[..., 17 * dim:], (4, blocks, 2, 2), (2, 0, 3, 1))
    return ((kq.unflatten(-1, (blocks, 32)) * ks).flatten(-2), (vq.unflatten(-1, (blocks, 32)) * vs).flatten(-2))


def _plain_read(cache, slots, kind):
    pages, kv, tiles, size = cache.shape
    k, v = _expand(cache, size // 18)                                  # [pages][kv][tiles][16][D]
    at = slots.long()
    k, v = (x.permute(0, 2, 3, 1, 4).reshape(pages * tiles * 16, kv, -1)[at] for x in (k, v))
    return k.to(kind), v.to(kind)


def _quantize(x):
    """f32 [..][D] -> codes 0 to 15 [..][D] (uint8) and scales float16 [..][D / 32]."""
    b = x.unflatten(-1, (-1, 32))
    most, least = b.amax(-1), b.amin(-1)
    top = torch.where(most >= -least, most, least)
    d = (top / -8).to(torch.bfloat16).float().clamp(-TOP, TOP).to(torch.float16)
    step = d.double()[..., None]   # in 64 bits: a quotient next to a border
    q = torch.where(step == 0, torch.zeros_like(step), b.double() / step)
    return (q.round().clamp(-8, 7) + 8).to(torch.uint8).flatten(-2), d


def _plain_write(s):
    cache, at = s["cache"], s["slots"].long()
    pages, kv, tiles, size = cache.shape
    dim = size // 18
    t = at % 16
    base = ((at // (16 * tiles))[:, None] * kv + torch.arange(kv, device=DEV)) * tiles + (at // 16 % tiles)[:, None]
    base = (base * size)[..., None]
    flat = cache.view(-1)
    i, x, g = torch.arange(dim // 16, device=DEV)[:, None], torch.arange(8, device=DEV), torch.arange(dim // 32, device=DEV)
    block, low, high = (i // 4) * 512 + (i % 4) * 4, t[:, None, None] % 8, t[:, None, None] // 8
    places = {"k": block + (low * 4 + x // 2) * 16 + 2 * (x % 2) + high,
              "v": block + (x * 4 + low // 2) * 16 + 2 * (low % 2) + high + 9 * dim}
    low, high = t[:, None] % 8, t[:, None] // 8
    steps = {"k": 4 * dim + (low * 2 + high) * (dim // 32) + g,
             "v": 17 * dim // 2 + ((low // 2) * (dim // 32) + g) * 4 + 2 * high + low % 2}
    for name in ("k", "v"):
        q, d = _quantize(s[name].float())
        q = q.unflatten(-1, (-1, 2, 8))
        flat[base + places[name].flatten(1)[:, None]] = (q[..., 0, :] | (q[..., 1, :] << 4)).flatten(-2)
        flat.view(torch.float16)[base // 2 + steps[name][:, None]] = d
    k, v = _plain_read(cache, s["every"], s["k"].dtype)
    return {"k": k, "v": v}


def _plain_attn(s):
    c, q = s["case"], s["q"]
    batch, kv, dim = c["batch"], c["kv_heads"], c["dim"]
    group, heads = c["heads"] // kv, c["heads"]
    starts = torch.arange(batch + 1, device=DEV) if s["q_starts"] is None else s["q_starts"].long()
    news, lens = starts[1:] - starts[:-1], s["lens"].long()
    j = torch.arange(c["new"], device=DEV)
    rows = torch.where(j < news[:, None], starts[:-1, None] + j, 0)              # [batch][new]
    k, v = _expand(s["cache"][s["page_table"].long()], dim)                      # [batch][width][kv][tiles][16][D]
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(batch, kv, -1, dim) for x in (k, v))
    qp = q[rows].float().view(batch, c["new"], kv, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, kv, -1, dim)
    score = torch.matmul(qp / math.sqrt(dim), k.transpose(-1, -2)).view(batch, kv, c["new"], group, -1)
    del k
    seen = (lens - news + 1)[:, None] + j
    hidden = torch.arange(score.shape[-1], device=DEV) >= seen[..., None]
    score = score.masked_fill_(hidden[:, None, :, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    del score
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w.view(batch, kv, -1, w.shape[-1]), v).view(batch, kv, c["new"], group, dim)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    out = out.permute(0, 2, 1, 3, 4).reshape(batch, c["new"], heads, dim)
    whose = torch.searchsorted(starts[1:], torch.arange(q.shape[0], device=DEV), right=True)
    return out[whose, torch.arange(q.shape[0], device=DEV) - starts[whose]].to(q.dtype)


def _plain_copy(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return s["pool"]


def _plain_compact(s):
    c, pool, table = s["case"], s["pool"], s["page_table"].long()
    pages, dump = c["pages"], c["pages"]
    used = torch.arange(c["width"], device=DEV) < ((s["lens"].long() + c["page"] - 1) // c["page"])[:, None]
    live = torch.zeros(pages + 1, dtype=torch.int64, device=DEV)
    live[torch.where(used, table, dump).flatten()] = 1
    live = live[:pages]
    n = live.sum()
    at = torch.arange(pages, device=DEV)
    hole, mover = (live == 0) & (at < n), (live == 1) & (at >= n)
    # the k-th hole takes the k-th page that has to move
    source = torch.full((pages + 1,), dump, device=DEV)
    source[torch.where(mover, mover.long().cumsum(0) - 1, dump)] = at
    target = torch.full((pages + 1,), dump, device=DEV)
    target[torch.where(hole, hole.long().cumsum(0) - 1, dump)] = at
    new = torch.where((live == 1) & (at < n), at, -1)
    new = torch.cat([new, new.new_full((1,), -1)])
    source, target = source[:pages], target[:pages]
    moved = torch.arange(pages, device=DEV) < mover.sum()
    new[torch.where(moved, source, dump)] = torch.where(moved, target, -1)
    gather = torch.where(hole, source[(hole.long().cumsum(0) - 1).clamp_min(0)], at)
    pool.copy_(pool[:, gather])
    new = new[:pages]
    out = torch.where(used, new[torch.where(used, table, 0)], -1)
    return {"pool": pool, "table": out.to(torch.int32), "map": new.to(torch.int32), "live": n.view(1).to(torch.int32)}


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "read":
            k, v = _plain_read(s["cache"], s["slots"], TYPES[c["type"]])
            return {"k": k, "v": v}
        return {"write": _plain_write, "attn": _plain_attn, "copy": _plain_copy, "compact": _plain_compact}[c["op"]](s)
    import q4_q8_int8_gb300 as mmq
    if c["op"] == "write":
        mmq.kv4_write(s["k"], s["v"], s["slots"], s["cache"])
        k, v = mmq.kv4_read(s["cache"], s["every"], s["k"].dtype)
        return {"k": k, "v": v}
    if c["op"] == "read":
        k, v = mmq.kv4_read(s["cache"], s["slots"], TYPES[c["type"]])
        return {"k": k, "v": v}
    if c["op"] == "attn":
        return mmq.kv4_attention(s["q"], s["cache"], s["page_table"], s["lens"], q_starts=s["q_starts"])
    if c["op"] == "copy":
        mmq.pages_copy(s["caches"], s["src"], s["dst"])
        return s["pool"]
    table, page_map, live = mmq.pages_compact(s["caches"], s["page_table"], s["lens"], c["page"])
    return {"pool": s["pool"], "table": table, "map": page_map, "live": live}


# -------------------------------------------------------------------- work
def work(case):
    c = case
    kv, dim = c["kv_heads"], c["dim"]
    token = kv * dim * 2                      # values of a token, keys and values
    held = token * 9 // 16                    # bytes of a token in the cache
    if c["op"] == "write":
        return {"bytes": c["tokens"] * (2 * token + held + 4) + c["slots"] * (held + 2 * token + 4),
                "flops": 2 * token * (c["tokens"] + c["slots"])}
    if c["op"] == "read":
        return {"bytes": c["tokens"] * (held + 2 * token + 4), "flops": 2 * token * c["tokens"]}
    if c["op"] == "attn":
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(_news(c), _lens(c)))
        return {"bytes": held * sum(_lens(c)) + 4 * sum(_news(c)) * c["heads"] * dim,
                "flops": 4 * pairs * c["heads"] * dim}
    size = c["page"] * kv * dim * 2
    if c["op"] == "copy":
        return {"bytes": 2 * size * c["pairs"] * c["caches"], "flops": 0}
    # a live page is past the front with the share of free pages
    live = sum(_held(c))
    return {"bytes": 2 * size * c["caches"] * live * (1 - live / c["pages"]) + 8 * live + 4 * c["pages"], "flops": 0}


# ------------------------------------------------------------------ 64 bits
def _values(cache, slots):
    """Keys and values at `slots` in 64 bits, [T][kv][D], each code fetched from its own byte."""
    pages, kv, tiles, size = cache.shape
    dim = size // 18
    flat, at = cache.view(-1), slots.long()[:, None, None]
    t, h, x = at % 16, torch.arange(kv, device=DEV)[:, None], torch.arange(dim, device=DEV)
    tile = size * (((at // (16 * tiles)) * kv + h) * tiles + at // 16 % tiles)
    p, i, g = x % 8, x // 16, x // 32
    out = []
    for name in ("k", "v"):
        if name == "k":
            byte = tile + i // 4 * 512 + (t % 8) * 64 + p // 2 * 16 + i % 4 * 4 + p % 2 * 2 + t // 8
            scale = tile + 8 * dim + 2 * (((t % 8) * 2 + t // 8) * (dim // 32) + g)
        else:
            byte = tile + 9 * dim + i // 4 * 512 + p * 64 + t % 8 // 2 * 16 + i % 4 * 4 + t % 2 * 2 + t // 8
            scale = tile + 17 * dim + 2 * ((t % 8 // 2 * (dim // 32) + g) * 4 + t // 8 * 2 + t % 2)
        code = torch.where(x // 8 % 2 == 1, flat[byte] // 16, flat[byte] % 16).double() - 8
        out.append(code * flat.view(torch.float16)[scale // 2].double())
    return out


def _exact_write(s):
    """Every slot's values: those of the new tokens from the definition, zeros elsewhere."""
    out = {}
    for name in ("k", "v"):
        x = s[name].double()
        b = x.unflatten(-1, (-1, 32))
        size, where = b.abs().max(-1)
        both = (b.amax(-1) == size) & (b.amin(-1) == -size)
        top = torch.where(both, size, b.gather(-1, where[..., None])[..., 0])
        d = torch.clamp((-top / 8).to(torch.bfloat16).double(), -TOP, TOP).to(torch.float16).double()[..., None]
        steps = torch.clamp(torch.round(b / torch.where(d == 0, 1.0, d)), -8, 7) * d
        full = torch.zeros((s["case"]["slots"],) + x.shape[1:], dtype=torch.float64, device=DEV)
        full[s["slots"].long()] = steps.flatten(-2)
        out[name] = full[s["every"].long()]
    return out


def _exact_attn(s):
    c = s["case"]
    kv, dim, page = c["kv_heads"], c["dim"], c["page"]
    group = c["heads"] // kv
    news, lens = _news(c), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(news, lens)):
        ids = s["page_table"][b, :-(-m // page)]
        slots = (ids.long()[:, None] * page + torch.arange(page, device=DEV)).flatten()[:m]
        k, v = _values(s["cache"], slots)
        see = m - n + 1 + torch.arange(n, device=DEV)
        mask = torch.arange(m, device=DEV) >= see[:, None]
        for h in range(kv):
            q = s["q"][at:at + n, h * group:(h + 1) * group].double()
            score = torch.einsum("ngd,md->gnm", q, k[:, h]) * dim ** -0.5
            score.masked_fill_(mask, float("-inf"))
            out[at:at + n, h * group:(h + 1) * group] = torch.einsum("gnm,md->ngd", torch.softmax(score, -1), v[:, h])
            del score
        at += n
    return out


def _exact_compact(s):
    c, page = s["case"], s["case"]["page"]
    table, lens = s["page_table"].tolist(), s["lens"].tolist()
    live = sorted({p for row, n in zip(table, lens) for p in row[:-(-n // page)]})
    n = len(live)
    taken = set(live)
    holes = [p for p in range(n) if p not in taken]
    moves = dict(zip([p for p in live if p >= n], holes))
    where = [moves.get(p, p) if p in taken else -1 for p in range(c["pages"])]
    new = [[where[p] if i < -(-m // page) else -1 for i, p in enumerate(row)] for row, m in zip(table, lens)]
    pool = s["pool"].double()
    for a, b in moves.items():
        pool[:, b] = pool[:, a]
    return {"pool": pool, "table": torch.tensor(new, dtype=torch.int32, device=DEV),
            "map": torch.tensor(where, dtype=torch.int32, device=DEV),
            "live": torch.tensor([n], dtype=torch.int32, device=DEV)}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "read":
        k, v = _values(s["cache"], s["slots"])
        return {"k": k, "v": v}
    if c["op"] == "copy":
        pool = s["pool"].double()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[:, b] = s["pool"][:, a].double()
        return pool
    return {"write": _exact_write, "attn": _exact_attn, "compact": _exact_compact}[c["op"]](s)
