"""The 4-bit cache's binding without a GPU (stand-ins for tensors and library): what it refuses before the library is
called, what it passes on, and where a call with stream= allocates."""
import types

import pytest

import q4_q8_int8_gb300 as mmq
from tests.test_streams import Tensor, world  # noqa: F401

torch = pytest.importorskip("torch")
f16, f32, i32, u8 = torch.float16, torch.float32, torch.int32, torch.uint8


def cache(pages=8, kv=2, tiles=1, D=64, **more):
    return Tensor((pages, kv, tiles, 18 * D), u8, **more)


def write(k=None, v=None, slots=None, cache_=None, **more):
    k = Tensor((3, 2, 64), f16) if k is None else k
    mmq.kv4_write(k, Tensor((3, 2, 64), f16) if v is None else v, Tensor(3, i32) if slots is None else slots,
                  cache() if cache_ is None else cache_, **more)


def read(cache_=None, slots=None, **more):
    return mmq.kv4_read(cache() if cache_ is None else cache_, Tensor(3, i32) if slots is None else slots, **more)


def attend(q=None, cache_=None, table=None, lens=None, q_starts=None, **more):
    return mmq.kv4_attention(Tensor((3, 4, 64), f16) if q is None else q, cache() if cache_ is None else cache_,
                             Tensor((3, 2), i32) if table is None else table, Tensor(3, i32) if lens is None else lens,
                             q_starts=q_starts, **more)


CALLS = pytest.mark.parametrize("call", [write, read, attend], ids=lambda c: c.__name__)


@pytest.fixture(autouse=True)
def messages(monkeypatch):
    monkeypatch.setattr(mmq, "strerror", lambda code: "refused")


def refused(world, call, **more):  # noqa: F811
    with pytest.raises(mmq.MMQError) as e:
        call(**more)
    assert e.value.code == mmq.MMQ_ERR_ARG
    assert not [name for name, _ in world.lib.calls if name != "mmq_strerror" and not name.endswith(("workspace", "bytes"))]


@CALLS
def test_devices(world, call, monkeypatch):  # noqa: F811
    refused(world, call, stream=types.SimpleNamespace(cuda_stream=5, device_index=1))
    call(stream=world.side)
    world.lib.calls.clear()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    refused(world, call)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(Tensor, "get_device", lambda self: -1)
    refused(world, call)


@pytest.mark.parametrize("call,blocks", [(write, 0), (read, 2), (attend, 2)], ids=["write", "read", "attend"])
def test_allocations_are_the_given_streams(world, call, blocks):  # noqa: F811
    call(stream=world.side)
    assert world.blocks == [world.side] * blocks and world.lib.calls[-1][1][-1] == 77
    world.blocks.clear()
    call()
    assert world.blocks == [None] * blocks and world.lib.calls[-1][1][-1] == 1


@pytest.mark.parametrize("change", [
    dict(k=Tensor((3, 2, 64), torch.float64), v=Tensor((3, 2, 64), torch.float64)), dict(v=Tensor((3, 2, 64), f32)),
    dict(v=Tensor((3, 128), f16)), dict(v=Tensor((4, 2, 64), f16)), dict(k=Tensor((3, 2, 64), f16, stride=(128, 64, 2))),
    dict(v=Tensor((3, 2, 64), f16, stride=(128, 64, 2))), dict(slots=Tensor(4, i32)), dict(slots=Tensor(3, torch.int64)),
    dict(slots=Tensor(3, i32, stride=(2,))), dict(cache_=cache(kv=3)), dict(cache_=cache(D=128)),
    dict(cache_=Tensor((8, 2, 1, 18 * 64), torch.int8)), dict(cache_=cache(stride=(1, 2, 3, 4)))])
def test_write_refuses(world, change):  # noqa: F811
    refused(world, write, **change)


@pytest.mark.parametrize("change", [
    dict(slots=Tensor(3, torch.int64)), dict(slots=Tensor(3, i32, stride=(2,))), dict(dtype=torch.float64),
    dict(cache_=Tensor((8, 2, 1, 1153), u8)), dict(cache_=cache(stride=(1, 2, 3, 4))),
    dict(out=(Tensor((3, 2, 64), f16), Tensor((3, 2, 64), f32))), dict(out=(Tensor((3, 2, 64), f16), Tensor((2, 2, 64), f16))),
    dict(out=(Tensor((3, 2, 64), f16), Tensor((3, 2, 64), f16, stride=(256, 64, 1)))),
    dict(out=(Tensor((3, 2, 64), f16), Tensor((3, 2, 64), f16)), dtype=f32)])
def test_read_refuses(world, change):  # noqa: F811
    refused(world, read, **change)


@pytest.mark.parametrize("change", [
    dict(q=Tensor((3, 4, 64), f32)), dict(q=Tensor((3, 4, 64), f16, stride=(256, 32, 1))), dict(cache_=cache(D=128)),
    dict(cache_=cache(stride=(1, 2, 3, 4))), dict(table=Tensor((3, 2), torch.int64)), dict(lens=Tensor(2, i32)),
    dict(table=Tensor((2, 2), i32), lens=Tensor(2, i32)), dict(q_starts=Tensor(3, i32)), dict(q_starts=Tensor(4, torch.int64)),
    dict(out=Tensor((3, 4, 64), torch.bfloat16)), dict(out=Tensor((3, 4, 128), f16)),
    dict(workspace=Tensor(1 << 20, u8, stride=(0,)))])
def test_attention_refuses(world, change):  # noqa: F811
    refused(world, attend, **change)


def test_what_is_passed_on(world):  # noqa: F811
    write(k=Tensor((3, 2, 64), f16, stride=(1024, 128, 1)), cache_=cache(pages=5, tiles=4))
    p = world.lib.calls[-1][1][0]
    assert (p.k_token_stride, p.k_head_stride, p.v_token_stride, p.v_head_stride) == (1024, 128, 128, 64)
    assert (p.tokens, p.n_slots, p.kv_heads, p.head_dim, p.page_size, p.type) == (3, 5 * 64, 2, 64, 64, mmq.MMQ_TYPE_F16)
    one = Tensor((1, 1, 64), f16, stride=(7, 9, 1))    # strides of one entry do not matter
    write(k=one, v=one, slots=Tensor(1, i32), cache_=cache(kv=1))
    p = world.lib.calls[-1][1][0]
    assert (p.k_token_stride, p.k_head_stride) == (64, 64)
    attend(q=Tensor((7, 4, 64), f16, stride=(999 * 8, 64, 1)), q_starts=Tensor(4, i32), scale=0.5)
    p = world.lib.calls[-1][1][0]
    assert (p.tokens, p.batch, p.q_stride, p.scale, bool(p.q_starts)) == (7, 3, 999 * 8, 0.5, True)
    attend()
    assert not world.lib.calls[-1][1][0].q_starts


def copy(caches=None, src=None, dst=None, **more):
    caches = [Tensor((8, 64), u8), Tensor((8, 64), u8)] if caches is None else caches
    mmq.pages_copy(caches, Tensor(3, i32) if src is None else src, Tensor(3, i32) if dst is None else dst, **more)


def compact(caches=None, table=None, lens=None, **more):
    caches = [Tensor((8, 64), u8), Tensor((8, 64), u8)] if caches is None else caches
    mmq.pages_compact(caches, Tensor((3, 2), i32) if table is None else table, Tensor(3, i32) if lens is None else lens, 16, **more)


@pytest.mark.parametrize("call", [copy, compact])
def test_pages_devices(world, call, monkeypatch):  # noqa: F811
    test_devices(world, call, monkeypatch)


@pytest.mark.parametrize("call", [copy, compact])
@pytest.mark.parametrize("caches", [
    [Tensor((8, 64), u8), Tensor((9, 64), u8)], [Tensor((8, 64), u8), Tensor((8, 64), f16)],
    [Tensor((8, 64), u8, stride=(128, 1))], [Tensor((8, 64), u8)] * 257])
def test_caches_that_are_not_alike(world, call, caches):  # noqa: F811
    refused(world, call, caches=caches)


@pytest.mark.parametrize("change", [dict(src=Tensor(3, torch.int64)), dict(dst=Tensor(2, i32)), dict(dst=Tensor(3, i32, stride=(2,)))])
def test_copy_refuses(world, change):  # noqa: F811
    refused(world, copy, **change)


@pytest.mark.parametrize("change", [
    dict(table=Tensor((3, 2), torch.int64)), dict(lens=Tensor(2, i32)), dict(lens=Tensor(3, torch.int64)), dict(pages=9),
    dict(caches=[]), dict(table_out=Tensor((3, 2), torch.int64)), dict(table_out=Tensor((2, 3), i32)),
    dict(workspace=Tensor(1 << 20, u8, stride=(2,)))])
def test_compact_refuses(world, change):  # noqa: F811
    refused(world, compact, **change)


def test_pages_allocations_and_what_is_passed_on(world):  # noqa: F811
    compact(stream=world.side)
    assert world.blocks == [world.side] * 4 and world.lib.calls[-1][1][-1] == 77
    p = world.lib.calls[-1][1][0]
    assert (p.n_pages, p.page_bytes, p.table_width, p.batch, p.n_caches, p.page_size) == (8, 64, 2, 3, 2, 16)
    compact(caches=[], pages=5)
    p = world.lib.calls[-1][1][0]
    assert (p.n_pages, p.n_caches) == (5, 0) and not p.caches
    copy(caches=[Tensor((8, 16, 4), torch.float32)])
    p = world.lib.calls[-1][1][0]
    assert (p.pairs, p.n_pages, p.page_bytes, p.n_caches) == (3, 8, 256, 1)
