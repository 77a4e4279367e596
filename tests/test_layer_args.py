"""Refusals of the operators between the projections, before any device work."""
import ctypes

import pytest

import q4_q8_int8_gb300 as mmq
from q4_q8_int8_gb300 import build as mmq_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    mmq_build.build()
    return mmq.load_library()


def rope(**change):
    p = mmq.mmq_qk_norm_rope_t(0x10000, 0x20000, 0x30000, 0x40000, None, None, 0x50000, 0x60000, 0x70000, 0x80000,
                               6 * 64, 3, 100, 10, 4, 1, 64, 64, (ctypes.c_int32 * 4)(32), 0, mmq.MMQ_TYPE_F16, 1e-6)
    for k, v in change.items():
        setattr(p, k, (ctypes.c_int32 * 4)(*v) if k == "sections" else v)
    return mmq.mmq_qk_norm_rope(p, None)


@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(q=None), dict(k_cache=None), dict(v_cache=None), dict(positions=None), dict(slots=None),
    dict(cos_table=None), dict(sin_table=None), dict(tokens=-1), dict(tokens=2 ** 31), dict(n_slots=-1),
    dict(heads=0), dict(kv_heads=0), dict(head_dim=60), dict(head_dim=264), dict(head_dim=8), dict(rot=72),
    dict(rot=60), dict(rot=-8), dict(ld=6 * 64 - 4), dict(ld=6 * 64 + 2), dict(type=mmq.MMQ_TYPE_F32), dict(type=-1),
    dict(sections=(31,)), dict(sections=(33, -1)), dict(sections=(16, 8, 4, 8)), dict(table_rows=-1)])
def test_rope_refuses_arguments(change):
    assert rope(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("name,by", [("qkv", 8), ("q", 8), ("k_cache", 2), ("v_cache", 8), ("q_weight", 4),
                                     ("k_weight", 8), ("cos_table", 4), ("sin_table", 4), ("positions", 2), ("slots", 1)])
def test_rope_refuses_alignment(name, by):
    assert rope(**{name: 0x90000 + by}) == mmq.MMQ_ERR_ALIGN


def test_null_structs():
    assert mmq.load_library().mmq_qk_norm_rope(None, None) == mmq.MMQ_ERR_ARG
    assert mmq.load_library().mmq_shared_prefix_attention(None, None, 0, None) == mmq.MMQ_ERR_ARG
    assert mmq.load_library().mmq_shared_prefix_attention_workspace(None) == 0
    assert mmq.load_library().mmq_q4K_moe(None, None, 0, None) == mmq.MMQ_ERR_ARG
    assert mmq.load_library().mmq_q4K_moe_workspace(None) == 0


def attn(workspace=0x100, ws_bytes=1 << 40, **change):
    f = dict(q=0x10000, out=0x20000, k_prefix=0x30000, v_prefix=0x40000, k_cache=0x50000, v_cache=0x60000,
             page_table=0x70000, lens=0x80000, q_stride=512, prefix=100, prefix_token_stride=128,
             prefix_head_stride=64, n_pages=8, table_width=2, batch=4, q_len=1, heads=8, kv_heads=2, head_dim=64,
             page_size=16, type=mmq.MMQ_TYPE_F16, out_type=mmq.MMQ_TYPE_F16, scale=0.125)
    f.update(change)
    return mmq.mmq_shared_prefix_attention(mmq.mmq_shared_prefix_attention_t(**f), workspace, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(out=None), dict(k_prefix=None), dict(v_prefix=None), dict(k_cache=None), dict(v_cache=None),
    dict(page_table=None), dict(lens=None), dict(workspace=None), dict(batch=-1), dict(q_len=0), dict(heads=0),
    dict(heads=7), dict(kv_heads=0), dict(kv_heads=3), dict(head_dim=32), dict(head_dim=96), dict(head_dim=256),
    dict(page_size=0), dict(page_size=12), dict(page_size=1 << 21), dict(prefix=-1), dict(n_pages=-1),
    dict(table_width=-1), dict(table_width=1 << 30), dict(type=2), dict(out_type=1), dict(out_type=3), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride=504), dict(q_stride=516),
    dict(prefix_token_stride=60), dict(prefix_token_stride=132), dict(prefix_head_stride=32),
    dict(prefix_head_stride=68), dict(batch=1 << 30)])
def test_attention_refuses_arguments(change):
    assert attn(**change) == mmq.MMQ_ERR_ARG
    p = {k: v for k, v in change.items() if isinstance(v, (int, float)) and k != "workspace"}
    if p:   # a size it refuses has no workspace either
        assert mmq.mmq_shared_prefix_attention_workspace(mmq.mmq_shared_prefix_attention_t(**p)) == 0


@pytest.mark.parametrize("name,by", [("q", 8), ("out", 4), ("k_prefix", 2), ("v_prefix", 8), ("k_cache", 4),
                                     ("v_cache", 2), ("page_table", 2), ("lens", 1), ("workspace", 128)])
def test_attention_refuses_alignment(name, by):
    assert attn(**{name: 0x90000 + by}) == mmq.MMQ_ERR_ALIGN


def moe(workspace=0x100, ws_bytes=1 << 40, **change):
    f = dict(x=0x10000, w_router=0x20000, w_gu=0x30000, w_down=0x40000, residual=None, out=0x50000, ids=0x60000,
             weights=0x70000, tokens=4, model=512, ffn=256, experts=8, top_k=2, renormalize=1)
    f.update(change)
    return mmq.mmq_q4K_moe(mmq.mmq_q4K_moe_t(**f), workspace, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(w_router=None), dict(w_gu=None), dict(w_down=None), dict(out=None), dict(ids=None),
    dict(weights=None), dict(workspace=None), dict(tokens=-1), dict(tokens=65), dict(model=0), dict(model=384),
    dict(ffn=0), dict(ffn=300), dict(experts=0), dict(experts=257), dict(top_k=0), dict(top_k=9),
    dict(top_k=17, experts=64), dict(tokens=64, top_k=9, experts=16), dict(model=1 << 21), dict(ffn=1 << 21)])
def test_moe_refuses_arguments(change):
    assert moe(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("name,by", [("x", 8), ("w_router", 4), ("w_gu", 1), ("w_down", 8), ("residual", 4), ("out", 8),
                                     ("ids", 2), ("weights", 1), ("workspace", 128)])
def test_moe_refuses_alignment(name, by):
    assert moe(**{name: 0x90000 + by}) == mmq.MMQ_ERR_ALIGN
