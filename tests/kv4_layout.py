"""The 4-bit cache's layout, byte by byte, and its quantization in 64 bits, apart from the library's code."""
import torch


def places(slots, kv_heads, page_size, D):
    """For each slot, head and dimension: (byte of the key's code, of its scale, of the value's code, of its scale) and
    whether the code is the upper nibble."""
    s = slots.long()[:, None, None]
    h = torch.arange(kv_heads, device=s.device)[:, None]
    x = torch.arange(D, device=s.device)
    page, place = s // page_size, s % page_size
    tile = 18 * D * ((page * kv_heads + h) * (page_size // 16) + place // 16)
    t = place % 16
    r, upper = t % 8, t // 8
    block16, x8, block32 = x // 16, x % 8, x // 32
    word = (block16 // 4) * 512 + (block16 % 4) * 4          # of the lanes' words
    k = tile + word + (4 * r + x8 // 2) * 16 + upper + 2 * (x8 % 2)
    ks = tile + 8 * D + 2 * ((2 * r + upper) * (D // 32) + block32)
    v = tile + 9 * D + word + (4 * x8 + r // 2) * 16 + upper + 2 * (t % 2)
    vs = tile + 17 * D + 2 * (((r // 2) * (D // 32) + block32) * 4 + 2 * upper + t % 2)
    return k, ks, v, vs, (x // 8 % 2 == 1).expand_as(k)


def codes_and_scales(cache, slots):
    """(key codes, key scales, value codes, value scales), [T][kv_heads][D] each, scales in 64 bits."""
    pages, kv_heads, tiles, size = cache.shape
    k, ks, v, vs, high = places(slots, kv_heads, 16 * tiles, size // 18)
    flat = cache.reshape(-1)
    code = lambda at: torch.where(high, flat[at] >> 4, flat[at] & 15).to(torch.int64)  # noqa: E731
    scale = lambda at: flat.view(torch.float16)[at // 2].double()  # noqa: E731
    return code(k), scale(ks), code(v), scale(vs)


def values(cache, slots):
    """Keys and values in 64 bits, [T][kv_heads][D]."""
    kq, ks, vq, vs = codes_and_scales(cache, slots)
    return (kq - 8) * ks, (vq - 8) * vs


def quantize(x):
    """x [..][D] -> (codes 0..15, scales in 64 bits for each value)."""
    b = x.double().unflatten(-1, (-1, 32))
    most, least = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
    top = torch.where(most >= -least, most, least)
    finite = torch.isfinite(b).all(-1, keepdim=True)
    d = (top.float() / -8).to(torch.bfloat16).double().clamp(-8160, 8160).to(torch.float16).double()
    d = torch.where(finite, d, torch.full_like(d, float("nan")))
    q = torch.where((d == 0) | d.isnan(), torch.zeros_like(b), b / d)
    return (q.round().clamp(-8, 7) + 8).long().flatten(-2), d.expand_as(b).flatten(-2)
