"""One decode step of a mixture-of-experts decoder layer for a batch of
sequences that share a long prompt, on q4_K weights throughout:

    norm -> q8_1 -> q/k/v projection        quantize_q8_1, q4K_gemm
    head norms, rotary positions, cache     qk_norm_rope
    attention: shared prompt + own suffix   shared_prefix_attention
    q8_1 -> output projection, residual     quantize_q8_1, q4K_gemm
    norm -> routed experts, residual        q4K_moe

Run as a script it builds a layer with random weights, takes a few steps and
prints the time of one (the whole step, and replayed from a CUDA graph).
"""
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import q4_q8_int8_gb300 as mmq

EPS = 1e-6


def random_q4K(rows, inner, generator, std):
    """q4_K bytes [rows][inner/256][144] (CUDA) of weights with no mean and about this deviation."""
    sb = inner // 256
    raw = torch.randint(0, 256, (rows, sb, 144), device="cuda", dtype=torch.uint8, generator=generator)
    # d sc (v - 7.5): random six-bit scales sc (rms 36.5), the same bits as minima, and 16 levels (rms 4.6)
    d = torch.full((rows, sb, 1), std / 168, device="cuda").half()
    raw[..., 0:2] = d.view(torch.uint8)
    raw[..., 2:4] = (d.float() * 7.5).half().view(torch.uint8)
    raw[..., 8:12] = raw[..., 4:8]
    raw[..., 12:16] = (raw[..., 12:16] & 15) * 17
    return raw


class Layer:
    """Weights, rotary tables and caches of one layer."""

    def __init__(self, hidden=2048, heads=16, kv_heads=4, dim=128, ffn=768, experts=32, top_k=4, prompt=4096, batch=16,
                 new=64, page=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.top_k = hidden, heads, kv_heads, dim, top_k
        self.w_qkv = random_q4K((heads + 2 * kv_heads) * dim, hidden, g, hidden ** -0.5)
        self.w_o = random_q4K(hidden, heads * dim, g, (heads * dim) ** -0.5)
        self.w_gu = random_q4K(experts * 2 * ffn, hidden, g, hidden ** -0.5).view(experts, 2 * ffn, hidden // 256, 144)
        self.w_down = random_q4K(experts * hidden, ffn, g, ffn ** -0.5).view(experts, hidden, ffn // 256, 144)
        self.w_router = torch.randn((experts, hidden), device="cuda", generator=g) * hidden ** -0.5
        self.norm_attn, self.norm_ffn = (1 + 0.1 * torch.randn(hidden, device="cuda", generator=g) for _ in range(2))
        self.q_weight, self.k_weight = (1 + 0.1 * torch.randn(dim, device="cuda", generator=g) for _ in range(2))
        turn = torch.arange(prompt + new, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(dim // 2, device="cuda", dtype=torch.float64) * 2 / dim)
        self.cos, self.sin = turn.cos().float(), turn.sin().float()
        self.prompt = prompt
        self.k_prompt, self.v_prompt = (torch.randn((prompt, kv_heads, dim), device="cuda", generator=g).half()
                                        for _ in range(2))
        width = -(-new // page)
        self.page = page
        self.page_table = torch.arange(batch * width, device="cuda", dtype=torch.int32).view(batch, width)
        self.k_cache, self.v_cache = (torch.zeros((batch * width, page, kv_heads, dim), device="cuda").half()
                                      for _ in range(2))


def rms_norm(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def decode_step(layer, x, lens, keep=None):
    """x float32 [batch][hidden], one new token per sequence, the one at place lens[b] of its own suffix (int32 [batch]).
    Returns the layer's output [batch][hidden] and the chosen experts; `keep`: a dict that receives what the steps
    hand on."""
    batch = x.shape[0]
    positions = lens + layer.prompt
    rows = torch.arange(batch, device=x.device)
    slots = layer.page_table[rows, (lens // layer.page).long()] * layer.page + lens % layer.page
    qkv = mmq.q4K_gemm(mmq.quantize_q8_1(rms_norm(x, layer.norm_attn)), layer.w_qkv, layer.w_qkv.shape[0])
    q = mmq.qk_norm_rope(qkv, layer.heads, layer.cos, layer.sin, positions, slots, layer.k_cache, layer.v_cache,
                         q_weight=layer.q_weight, k_weight=layer.k_weight, eps=EPS)
    seen = torch.empty(q.shape, device=x.device)     # float32, as the next prepass reads it
    mmq.shared_prefix_attention(q, layer.k_prompt, layer.v_prompt, layer.k_cache, layer.v_cache, layer.page_table,
                                lens + 1, out=seen)
    x = x + mmq.q4K_gemm(mmq.quantize_q8_1(seen.view(batch, -1)), layer.w_o, layer.hidden)
    z = rms_norm(x, layer.norm_ffn)
    out, ids, _ = mmq.q4K_moe(z, layer.w_router, layer.w_gu, layer.w_down, layer.top_k, residual=x)
    if keep is not None:
        keep.update(qkv=qkv, q=q, slots=slots, seen=seen, x=x, z=z)
    return out, ids


def main():
    batch = 16
    layer = Layer(batch=batch)
    x = torch.randn((batch, layer.hidden), device="cuda")
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    for _ in range(5):
        y, ids = decode_step(layer, x, lens)
        lens += 1
    torch.cuda.synchronize()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(50):
        decode_step(layer, x, lens)
    end.record()
    torch.cuda.synchronize()
    print(f"one step, batch {batch}, prompt {layer.prompt}: {start.elapsed_time(end) * 20:.1f} us")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode_step(layer, x, lens)
    graph.replay()
    torch.cuda.synchronize()
    start.record()
    for _ in range(50):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"the same from a CUDA graph: {start.elapsed_time(end) * 20:.1f} us")
    if mmq.status() != mmq.MMQ_OK:
        raise RuntimeError("device status")


if __name__ == "__main__":
    main()
