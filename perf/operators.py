"""The decode-layer operators around the quantized GEMMs, as measured: the
cases, their inputs, their plain form in torch, the library's calls and their
values in 64 bits.

  rope   query / key head norms, rotary positions and the cache write, from
         the f32 rows that a fused q/k/v projection leaves
  attn   attention of a batch of sequences that share one long prefix, each
         with its own paged suffix
  moe    a mixture-of-experts FFN on q4_K experts for a few tokens
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence: latency only
        dict(name="rope_decode_1", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             inter=False, norm=True, type="f16"),
        # an odd batch of decode steps, heads as wide as the 7B projections (32 x 128 each), interleaved pairs
        dict(name="rope_batch_77", op="rope", tokens=77, heads=32, kv_heads=32, dim=128, rot=128, axes=1,
             inter=True, norm=False, type="bf16"),
        # a ragged multimodal prefill: time / height / width positions, few kv heads
        dict(name="rope_axes_2047", op="rope", tokens=2047, heads=28, kv_heads=4, dim=128, rot=128, axes=3,
             inter=False, norm=True, type="bf16"),
        # a long prefill chunk
        dict(name="rope_prefill_8192", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             inter=False, norm=True, type="f16"),
        # a few requests on one system prompt: latency
        dict(name="attn_b4_2k", op="attn", batch=4, q_len=1, heads=32, kv_heads=8, dim=128, prefix=2048,
             suffix=128, page=16, type="f16"),
        # an odd batch, as many kv heads as heads, narrow heads, a prefix that ends inside every tile
        dict(name="attn_b33_5001", op="attn", batch=33, q_len=1, heads=32, kv_heads=32, dim=64, prefix=5001,
             suffix=600, page=32, type="bf16"),
        # a long shared document
        dict(name="attn_b64_32k", op="attn", batch=64, q_len=1, heads=32, kv_heads=8, dim=128, prefix=32768,
             suffix=1024, page=64, type="bf16"),
        # a full serving batch: the prefix part is a tensor-core product
        dict(name="attn_b256_16k", op="attn", batch=256, q_len=1, heads=32, kv_heads=8, dim=128, prefix=16384,
             suffix=512, page=16, type="f16"),
        # one token, many small experts: latency
        dict(name="moe_t1_e64", op="moe", tokens=1, model=2048, ffn=768, experts=64, top_k=8, renorm=True,
             residual=True),
        # a few tokens, each expert with about one
        dict(name="moe_t3_e32", op="moe", tokens=3, model=4096, ffn=1536, experts=32, top_k=4, renorm=True,
             residual=True),
        # a small decode batch over many experts
        dict(name="moe_t16_e64", op="moe", tokens=16, model=4096, ffn=2048, experts=64, top_k=6, renorm=False,
             residual=False),
        # a decode batch, few experts as wide as the 7B FFN: every expert is read
        dict(name="moe_t32_e8", op="moe", tokens=32, model=4096, ffn=11008, experts=8, top_k=2, renorm=True,
             residual=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "moe"])
    kind = rng.choice(["f16", "bf16"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        axes = rng.choice([1, 1, 2, 3])
        rot = rng.choice([dim, dim, dim // 2 // 8 * 8])
        most = min(8192, 8192 * 6144 // (6 * kv * dim))
        return dict(op=op, tokens=_log(rng, 1, most), heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, dim=dim, rot=rot,
                    axes=axes, inter=rng.random() < 0.3, norm=rng.random() < 0.7, type=kind)
    if op == "attn":
        dim = rng.choice([64, 128, 128])
        kv = rng.choice([1, 2, 4, 8])
        q_len = rng.choice([1, 1, 1, 2, 5])
        batch = _log(rng, 1, 192)
        return dict(op=op, batch=max(1, batch // q_len), q_len=q_len, heads=kv * rng.choice([1, 3, 4]), kv_heads=kv,
                    dim=dim, prefix=_log(rng, 1, 16384) if rng.random() < 0.9 else 0,
                    suffix=q_len + _log(rng, 1, 512), page=rng.choice([16, 32, 64]), type=kind)
    experts = rng.choice([8, 16, 24, 64])
    ffn = 256 * _log(rng, 1, {8: 40, 16: 20, 24: 12, 64: 6}[experts])
    return dict(op=op, tokens=_log(rng, 1, 32), model=256 * _log(rng, 2, 16), ffn=ffn, experts=experts,
                top_k=rng.choice([1, 2, 4, 8]), renorm=rng.random() < 0.5, residual=rng.random() < 0.5)


def _sections(c):
    """Rotated pairs per axis: about a quarter for the first axis, the rest in equal parts."""
    half, a = c["rot"] // 2, c["axes"]
    if a == 1:
        return [half]
    rest = (half - half // 4) // (a - 1)
    return [half - rest * (a - 1)] + [rest] * (a - 1)


def _lens(c):
    """Tokens in each sequence's own suffix, its new ones among them: ragged, from one step to the longest."""
    span = c["suffix"] - c["q_len"] + 1
    return [c["q_len"] + (i * 7919 + c["suffix"] - c["q_len"]) % span for i in range(c["batch"])]


# ------------------------------------------------------------------ inputs
def _q4k(g, n, k, level):
    """q4_K bytes [n][k/256][144] of weights with no mean: 16 levels around the middle, 6-bit scales, minima near
    7.5 of their scales."""
    sb = k // 256
    sc = torch.randint(16, 64, (n, sb, 8), device=DEV, generator=g, dtype=torch.uint8)
    mn = torch.clamp(sc.to(torch.int16) + torch.randint(-3, 4, sc.shape, device=DEV, generator=g, dtype=torch.int16),
                     0, 63).to(torch.uint8)
    d = ((torch.rand((n, sb, 1), device=DEV, generator=g) + 0.5) * level).to(torch.float16)
    dmin = (d.float() * 7.5).to(torch.float16)
    s = torch.empty((n, sb, 12), device=DEV, dtype=torch.uint8)
    s[..., 0:4] = sc[..., :4] | ((sc[..., 4:] >> 4) << 6)
    s[..., 4:8] = mn[..., :4] | ((mn[..., 4:] >> 4) << 6)
    s[..., 8:12] = (sc[..., 4:] & 15) | ((mn[..., 4:] & 15) << 4)
    q = torch.randint(0, 256, (n, sb, 128), device=DEV, generator=g, dtype=torch.uint8)
    return torch.cat([d.view(torch.uint8), dmin.view(torch.uint8), s, q], dim=2).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=g)

    if c["op"] == "rope":
        t, dim, kind = c["tokens"], c["dim"], TYPES[c["type"]]
        half, limit = c["rot"] // 2, 16384
        qkv = normal(t, (c["heads"] + 2 * c["kv_heads"]) * dim)
        # a few channels of the projections are much larger than the others
        qkv *= 1 + 9 * (torch.rand(qkv.shape[1], device=DEV, generator=g) < 0.02).float()
        angle = torch.arange(limit, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(half, device=DEV, dtype=torch.float64) / half)
        at = int(torch.randint(0, limit - t, (1,), device=DEV, generator=g))
        pos = torch.arange(at, at + t, device=DEV, dtype=torch.int32)
        if c["axes"] > 1:  # time runs on, the others go over a picture's rows and columns
            pos = torch.stack([pos, (pos // 37) % 61, pos % 37][: c["axes"]]).contiguous()
        slots = t + 64
        axis = torch.tensor([a for a, n in enumerate(_sections(c)) for _ in range(n)], device=DEV)
        return dict(case=c, qkv=qkv, axis=axis, cos=angle.cos().float(), sin=angle.sin().float(), positions=pos,
                    slots=torch.randperm(slots, device=DEV, generator=g)[:t].to(torch.int32),
                    k_cache=normal(slots, c["kv_heads"], dim).to(kind), v_cache=normal(slots, c["kv_heads"], dim).to(kind),
                    q_weight=1 + 0.2 * normal(dim) if c["norm"] else None,
                    k_weight=1 + 0.2 * normal(dim) if c["norm"] else None)
    if c["op"] == "attn":
        kind, kv, dim = TYPES[c["type"]], c["kv_heads"], c["dim"]
        width = -(-c["suffix"] // c["page"])
        pages = c["batch"] * width
        return dict(case=c, q=normal(c["batch"] * c["q_len"], c["heads"], dim).to(kind),
                    k_prefix=normal(c["prefix"], kv, dim).to(kind), v_prefix=normal(c["prefix"], kv, dim).to(kind),
                    k_cache=normal(pages, c["page"], kv, dim).to(kind), v_cache=normal(pages, c["page"], kv, dim).to(kind),
                    page_table=torch.randperm(pages, device=DEV, generator=g).view(c["batch"], width).to(torch.int32),
                    lens=torch.tensor(_lens(c), device=DEV, dtype=torch.int32))
    t, k, f, e = c["tokens"], c["model"], c["ffn"], c["experts"]
    x = normal(t, k)
    x *= 1 + 9 * (torch.rand(k, device=DEV, generator=g) < 0.01).float()
    return dict(case=c, x=x, w_router=normal(e, k) / math.sqrt(k),
                w_gu=_q4k(g, e * 2 * f, k, 1.0 / (184 * math.sqrt(k))).view(e, 2 * f, k // 256, 144),
                w_down=_q4k(g, e * k, f, 1.0 / (184 * math.sqrt(f))).view(e, k, f // 256, 144),
                residual=normal(t, k) if c["residual"] else None)


# ------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, rot, inter):
    """x [T][H][D] in f32, cos / sin [T][1][rot/2]: the first rot values of each head turned pair by pair."""
    half = rot // 2
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :half], r[..., half:])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], dim=-1).flatten(-2) if inter else torch.cat([u, v], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    t, hq, hk, dim = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    x = s["qkv"].view(t, hq + 2 * hk, dim)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_weight"]
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_weight"]
    pos = s["positions"].view(c["axes"], t).long()
    row, col = pos[s["axis"]].T, torch.arange(c["rot"] // 2, device=DEV)
    cos, sin = s["cos"][row, col][:, None], s["sin"][row, col][:, None]
    q, k = _rotate(q, cos, sin, c["rot"], c["inter"]), _rotate(k, cos, sin, c["rot"], c["inter"])
    at, kind = s["slots"].long(), s["k_cache"].dtype
    s["k_cache"][at] = k.to(kind)
    s["v_cache"][at] = v.to(kind)
    return {"q": q.to(kind), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    c = s["case"]
    b, n, hk, dim, p = c["batch"], c["q_len"], c["kv_heads"], c["dim"], c["prefix"]
    group = c["heads"] // hk
    q = s["q"].float().view(b, n, hk, group, dim) / math.sqrt(dim)
    kp, vp = s["k_prefix"].float(), s["v_prefix"].float()
    at = s["page_table"].long()
    ks = s["k_cache"][at].float().view(b, -1, hk, dim)
    vs = s["v_cache"][at].float().view(b, -1, hk, dim)
    shared = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(hk, -1, dim), kp.permute(1, 2, 0))
    shared = shared.view(hk, b, n, group, p).permute(1, 2, 0, 3, 4)
    mine = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(b, hk, n * group, dim), ks.permute(0, 2, 3, 1))
    mine = mine.view(b, hk, n, group, -1).permute(0, 2, 1, 3, 4)
    token = torch.arange(ks.shape[1], device=DEV)
    seen = s["lens"].long()[:, None] - n + 1 + torch.arange(n, device=DEV)
    mine = mine.masked_fill(~(token < seen[..., None])[:, :, None, None, :], float("-inf"))
    score = torch.cat([shared, mine], dim=-1)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total == 0, torch.ones_like(total), total)
    a, m = w[..., :p], w[..., p:]
    out = torch.matmul(a.permute(2, 0, 1, 3, 4).reshape(hk, -1, p), vp.permute(1, 0, 2))
    out = out.view(hk, b, n, group, dim).permute(1, 2, 0, 3, 4)
    last = torch.matmul(m.permute(0, 2, 1, 3, 4).reshape(b, hk, n * group, -1), vs.permute(0, 2, 1, 3))
    out = out + last.view(b, hk, n, group, dim).permute(0, 2, 1, 3, 4)
    return out.reshape(b * n, c["heads"], dim).to(s["q"].dtype)


def _plain_weights(w):
    """q4_K bytes [..][sb][144] -> f32 [..][256 sb]."""
    d = w[..., 0:2].contiguous().view(torch.float16).float()
    dmin = w[..., 2:4].contiguous().view(torch.float16).float()
    lo, mid, hi = w[..., 4:8], w[..., 8:12], w[..., 12:16]
    sc = torch.cat([lo & 63, (hi & 15) | ((lo >> 6) << 4)], dim=-1).float() * d
    mn = torch.cat([mid & 63, (hi >> 4) | ((mid >> 6) << 4)], dim=-1).float() * dmin
    q = w[..., 16:].unflatten(-1, (4, 1, 32))
    q = torch.cat([q & 15, q >> 4], dim=-2).flatten(-3, -2).float()
    return (q * sc[..., None] - mn[..., None]).flatten(-3)


def _plain_moe(s):
    c = s["case"]
    x = s["x"]
    p = torch.softmax(x @ s["w_router"].T, dim=-1)
    best, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    best, ids = best[:, :c["top_k"]].contiguous(), ids[:, :c["top_k"]].contiguous()
    if c["renorm"]:
        best = best / best.sum(-1, keepdim=True)
    gu = torch.matmul(x, _plain_weights(s["w_gu"]).transpose(1, 2))
    gate, up = gu[..., 0::2], gu[..., 1::2]
    h = gate / (1 + torch.exp(-gate)) * up
    part = torch.zeros_like(p).scatter_(1, ids, best)
    y = torch.matmul(h * part.T[..., None], _plain_weights(s["w_down"]).transpose(1, 2)).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"]
    return {"out": y, "ids": ids.to(torch.int32), "weights": best}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rope": _plain_rope, "attn": _plain_attn, "moe": _plain_moe}[c["op"]](s)
    import q4_q8_int8_gb300 as mmq
    if c["op"] == "rope":
        q = mmq.qk_norm_rope(s["qkv"], c["heads"], s["cos"], s["sin"], s["positions"], s["slots"], s["k_cache"],
                             s["v_cache"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                             interleaved=c["inter"], sections=_sections(c))
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "attn":
        return mmq.shared_prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], s["k_cache"], s["v_cache"],
                                           s["page_table"], s["lens"], q_len=c["q_len"])
    out, ids, weights = mmq.q4K_moe(s["x"], s["w_router"], s["w_gu"], s["w_down"], c["top_k"],
                                    renormalize=c["renorm"], residual=s["residual"])
    return {"out": out, "ids": ids, "weights": weights}


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "rope":
        values = c["tokens"] * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        table = c["tokens"] * c["rot"] // 2 * 8
        return {"bytes": values * 6 + table + 4 * c["tokens"] * (c["axes"] + 1), "flops": 6 * values}
    if c["op"] == "attn":
        mine = sum(_lens(c))
        token = 4 * c["kv_heads"] * c["dim"]
        rows = c["batch"] * c["q_len"] * c["heads"]
        pairs = rows * c["prefix"] + c["heads"] * c["q_len"] * mine
        return {"bytes": (c["prefix"] + mine) * token + 4 * rows * c["dim"], "flops": 4 * pairs * c["dim"]}
    t, k, f, e = c["tokens"], c["model"], c["ffn"], c["experts"]
    busy = e * (1 - (1 - c["top_k"] / e) ** t)
    weights = busy * 3 * k * f * 0.5625
    return {"bytes": weights + 4 * e * k + 4 * t * k * (3 if c["residual"] else 2),
            "flops": 2 * t * c["top_k"] * 3 * k * f + 2 * t * e * k}


# ------------------------------------------------------------------ 64 bits
def _exact_rope(s):
    c = s["case"]
    t, hq, hk, dim, half = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    x = s["qkv"].double().view(t, -1, dim).clone()
    if c["norm"]:
        for lo, n, w in ((0, hq, s["q_weight"]), (hq, hk, s["k_weight"])):
            part = x[:, lo:lo + n]
            part *= w.double() / torch.sqrt(part.square().sum(-1, keepdim=True) / dim + EPS)
    pos = s["positions"].view(c["axes"], t).long()
    first = 0
    turned = x[:, :hq + hk]
    was = turned.clone()
    for axis, n in enumerate(_sections(c)):
        for j in range(first, first + n):
            a, b = (2 * j, 2 * j + 1) if c["inter"] else (j, j + half)
            z = torch.complex(was[..., a], was[..., b])
            z = z * torch.complex(s["cos"][pos[axis], j].double(), s["sin"][pos[axis], j].double())[:, None]
            turned[..., a], turned[..., b] = z.real, z.imag
        first += n
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache[s["slots"].long()] = x[:, hq:hq + hk]
    v_cache[s["slots"].long()] = x[:, hq + hk:]
    return {"q": x[:, :hq], "k_cache": k_cache, "v_cache": v_cache}


def _exact_attn(s):
    c = s["case"]
    b, n, hk, dim, page = c["batch"], c["q_len"], c["kv_heads"], c["dim"], c["page"]
    group, lens = c["heads"] // hk, s["lens"].tolist()
    out = torch.zeros((b * n, c["heads"], dim), dtype=torch.float64, device=DEV)
    q = s["q"].double()
    for h in range(hk):
        mine = q[:, h * group:(h + 1) * group].reshape(b * n * group, dim)
        kp, vp = s["k_prefix"][:, h].double(), s["v_prefix"][:, h].double()
        score = mine @ kp.T / math.sqrt(dim)
        top = score.amax(-1) if c["prefix"] else torch.full((b * n * group,), float("-inf"), dtype=torch.float64, device=DEV)
        score = torch.exp(score - top[:, None])
        total, acc = score.sum(-1), score @ vp
        del score
        total, acc, top = total.view(b, n, group), acc.view(b, n, group, dim), top.view(b, n, group)
        for i in range(b):
            ids = s["page_table"][i, :-(-lens[i] // page)].long()
            ks = s["k_cache"][ids, :, h].double().reshape(-1, dim)
            vs = s["v_cache"][ids, :, h].double().reshape(-1, dim)
            for j in range(n):
                see = max(0, lens[i] - n + 1 + j)
                row = q[i * n + j, h * group:(h + 1) * group] @ ks[:see].T / math.sqrt(dim)
                most = torch.maximum(top[i, j], row.amax(-1)) if see else top[i, j]
                if bool(torch.isinf(most).any()):
                    continue
                old, new = torch.exp(top[i, j] - most), torch.exp(row - most[:, None])
                sums = total[i, j] * old + new.sum(-1)
                out[i * n + j, h * group:(h + 1) * group] = (acc[i, j] * old[:, None] + new @ vs[:see]) / sums[:, None]
    return out


def _exact_weights(w):
    """q4_K bytes [n][sb][144] -> f64 [n][256 sb], from the words of the block's head."""
    n, sb = w.shape[:2]
    head = w[..., :16].contiguous()
    halves = head[..., :4].contiguous().view(torch.float16).double()
    bits = head[..., 4:].long()
    out = torch.empty((n, sb, 8, 32), dtype=torch.float64, device=w.device)
    for j in range(8):
        if j < 4:
            sc, mn = bits[..., j] % 64, bits[..., j + 4] % 64
        else:
            sc = bits[..., j + 4] % 16 + 16 * (bits[..., j - 4] // 64)
            mn = bits[..., j + 4] // 16 + 16 * (bits[..., j] // 64)
        byte = w[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        v = (byte // 16 if j % 2 else byte % 16).double()
        out[..., j, :] = (halves[..., 0] * sc)[..., None] * v - (halves[..., 1] * mn)[..., None]
    return out.view(n, sb * 256)


def _exact_moe(s):
    c = s["case"]
    x = s["x"].double()
    logit = x @ s["w_router"].double().T
    p = torch.exp(logit - torch.logsumexp(logit, dim=-1, keepdim=True))
    ids = torch.argsort(-p, dim=-1, stable=True)[:, :c["top_k"]]
    weights = p.gather(1, ids)
    if c["renorm"]:
        weights = weights / weights.sum(-1, keepdim=True)
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double().clone()
    for e in range(c["experts"]):
        token, place = torch.nonzero(ids == e, as_tuple=True)
        if not token.numel():
            continue
        gu = x[token] @ _exact_weights(s["w_gu"][e]).T
        gate, up = gu[:, 0::2], gu[:, 1::2]
        h = gate * torch.sigmoid(gate) * up
        y.index_add_(0, token, weights[token, place][:, None] * (h @ _exact_weights(s["w_down"][e]).T))
    return {"out": y, "ids": ids.to(torch.int32), "weights": weights}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "moe": _exact_moe}[case["op"]](s)
