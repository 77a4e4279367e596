"""Refusals of the 4-bit cache's entry points, before any device work."""
import ctypes

import pytest

import q4_q8_int8_gb300 as mmq
from q4_q8_int8_gb300 import build as mmq_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    mmq_build.build()
    return mmq.load_library()


def write(**change):
    f = dict(k=0x10000, v=0x20000, cache=0x30000, slots=0x40000, k_token_stride=512, k_head_stride=64,
             v_token_stride=512, v_head_stride=64, tokens=3, n_slots=64, kv_heads=2, head_dim=64, page_size=16,
             type=mmq.MMQ_TYPE_F16)
    f.update(change)
    return mmq.mmq_kv4_write(mmq.mmq_kv4_write_t(**f), None)


def read(**change):
    f = dict(cache=0x30000, slots=0x40000, k=0x10000, v=0x20000, tokens=3, n_slots=64, kv_heads=2, head_dim=64,
             page_size=16, type=mmq.MMQ_TYPE_F16)
    f.update(change)
    return mmq.mmq_kv4_read(mmq.mmq_kv4_read_t(**f), None)


BOTH = [dict(k=None), dict(v=None), dict(cache=None), dict(slots=None), dict(tokens=-1), dict(tokens=2 ** 31 - 1),
        dict(n_slots=-16), dict(n_slots=2 ** 31), dict(n_slots=40, page_size=32), dict(kv_heads=0), dict(kv_heads=65536),
        dict(head_dim=32), dict(head_dim=96), dict(head_dim=256), dict(page_size=8), dict(page_size=0), dict(page_size=48),
        dict(page_size=1 << 21), dict(type=3), dict(type=-1)]


@pytest.mark.parametrize("change", BOTH + [dict(k_token_stride=-8), dict(k_head_stride=60), dict(v_token_stride=4),
                                           dict(v_head_stride=1 << 39)])
def test_write_refuses_arguments(change):
    assert write(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("change", BOTH)
def test_read_refuses_arguments(change):
    assert read(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("name,by", [("k", 8), ("v", 4), ("cache", 8), ("slots", 2)])
def test_slots_calls_refuse_alignment(call, name, by):
    assert call(**{name: 0x90000 + by}) == mmq.MMQ_ERR_ALIGN


def attn(workspace=0x100, ws_bytes=1 << 40, **change):
    f = dict(q=0x10000, out=0x20000, cache=0x30000, page_table=0x40000, lens=0x50000, q_starts=0x60000, q_stride=512,
             tokens=5, n_pages=8, table_width=2, batch=4, heads=8, kv_heads=2, head_dim=64, page_size=16,
             type=mmq.MMQ_TYPE_F16, out_type=mmq.MMQ_TYPE_F16, scale=0.125)
    f.update(change)
    return mmq.mmq_kv4_attention(mmq.mmq_kv4_attention_t(**f), workspace, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(out=None), dict(cache=None), dict(page_table=None), dict(lens=None), dict(workspace=None),
    dict(q_starts=None), dict(q_starts=None, batch=0), dict(batch=-1), dict(batch=(1 << 20) + 1), dict(tokens=-1),
    dict(tokens=1 << 30), dict(heads=0), dict(heads=7), dict(heads=65536, kv_heads=1), dict(kv_heads=0), dict(kv_heads=3),
    dict(head_dim=32), dict(head_dim=256), dict(page_size=8), dict(page_size=24), dict(page_size=1 << 21),
    dict(n_pages=-1), dict(n_pages=1 << 31), dict(table_width=-1), dict(table_width=1 << 28), dict(type=2),
    dict(out_type=1), dict(out_type=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(q_stride=504), dict(q_stride=516), dict(q_stride=1 << 39)])
def test_attention_refuses_arguments(change):
    assert attn(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("name,by", [("q", 8), ("out", 4), ("cache", 8), ("page_table", 2), ("lens", 1), ("q_starts", 2),
                                     ("workspace", 128)])
def test_attention_refuses_alignment(name, by):
    assert attn(**{name: 0x90000 + by}) == mmq.MMQ_ERR_ALIGN


def test_null_structs():
    lib = mmq.load_library()
    assert lib.mmq_kv4_write(None, None) == lib.mmq_kv4_read(None, None) == mmq.MMQ_ERR_ARG
    assert lib.mmq_kv4_attention(None, None, 0, None) == mmq.MMQ_ERR_ARG and lib.mmq_kv4_attention_workspace(None) == 0


def test_page_bytes():
    assert mmq.mmq_kv4_page_bytes(8, 128, 16) == 8 * 18 * 128 and mmq.mmq_kv4_page_bytes(2, 64, 64) == 2 * 4 * 18 * 64
    assert not any((mmq.mmq_kv4_page_bytes(0, 128, 16), mmq.mmq_kv4_page_bytes(8, 96, 16), mmq.mmq_kv4_page_bytes(8, 64, 12)))


def pointers(*at):
    return (ctypes.c_void_p * len(at))(*at)


def copy(caches=(0x10000, 0x20000), **change):
    f = dict(caches=None if caches is None else pointers(*caches), src=0x30000, dst=0x40000, pairs=3, n_pages=10,
             page_bytes=64, n_caches=2 if caches is None else len(caches))
    f.update(change)
    return mmq.mmq_pages_copy(mmq.mmq_pages_copy_t(**f), None)


@pytest.mark.parametrize("change", [
    dict(caches=None), dict(caches=(0x10000, None)), dict(caches=()), dict(caches=(0x10000,) * 257), dict(src=None),
    dict(dst=None), dict(pairs=-1), dict(pairs=2 ** 31), dict(n_pages=-1), dict(n_pages=2 ** 31), dict(page_bytes=0),
    dict(page_bytes=24), dict(page_bytes=-16), dict(page_bytes=2 ** 32 + 16), dict(n_caches=-1)])
def test_copy_refuses_arguments(change):
    assert copy(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("change", [dict(caches=(0x10000, 0x20008)), dict(src=0x30002), dict(dst=0x40001)])
def test_copy_refuses_alignment(change):
    assert copy(**change) == mmq.MMQ_ERR_ALIGN


def compact(caches=(0x10000,), workspace=0x100, ws_bytes=1 << 30, **change):
    f = dict(caches=None if caches is None else pointers(*caches), page_table=0x20000, lens=0x30000, table_out=0x40000,
             page_map=0x50000, live=0x60000, n_pages=10, page_bytes=64, table_width=4, batch=3,
             n_caches=1 if caches is None else len(caches), page_size=16)
    f.update(change)
    return mmq.mmq_pages_compact(mmq.mmq_pages_compact_t(**f), workspace, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(caches=None), dict(caches=(None,)), dict(caches=(0x10000,) * 257), dict(page_table=None), dict(lens=None),
    dict(table_out=None), dict(page_map=None), dict(live=None), dict(workspace=None), dict(n_pages=-1),
    dict(n_pages=(1 << 20) + 1), dict(page_bytes=40), dict(table_width=-1), dict(table_width=1 << 28), dict(batch=-1),
    dict(batch=(1 << 20) + 1), dict(page_size=0), dict(page_size=12), dict(page_size=1 << 21), dict(n_caches=-1)])
def test_compact_refuses_arguments(change):
    assert compact(**change) == mmq.MMQ_ERR_ARG


@pytest.mark.parametrize("change", [dict(caches=(0x10004,)), dict(page_table=2), dict(lens=1), dict(table_out=0x40002),
                                    dict(page_map=0x50001), dict(live=0x60002), dict(workspace=0x180)])
def test_compact_refuses_alignment(change):
    assert compact(**change) == mmq.MMQ_ERR_ALIGN


def test_pages_null_structs():
    lib = mmq.load_library()
    assert lib.mmq_pages_copy(None, None) == lib.mmq_pages_compact(None, None, 0, None) == mmq.MMQ_ERR_ARG
    assert lib.mmq_pages_compact_workspace(None) == 0
