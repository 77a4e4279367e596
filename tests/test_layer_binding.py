"""Refusals of the layer operators' binding, before the library is called;
without a GPU (stand-ins for tensors and library)."""
import types

import pytest

import q4_q8_int8_gb300 as mmq
from tests.test_streams import Tensor, attention, moe, rope, world  # noqa: F401

torch = pytest.importorskip("torch")
CALLS = pytest.mark.parametrize("call", [rope, attention, moe], ids=lambda c: c.__name__)


def refused(world, call, **more):  # noqa: F811
    with pytest.raises(mmq.MMQError) as e:
        call(**more)
    assert e.value.code == mmq.MMQ_ERR_ARG
    assert not [name for name, _ in world.lib.calls if name != "mmq_strerror" and not name.endswith("workspace")]


@pytest.fixture(autouse=True)
def messages(monkeypatch):
    monkeypatch.setattr(mmq, "strerror", lambda code: "refused")


@CALLS
def test_tensors_on_another_device_than_the_current(world, call, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    refused(world, call)


@CALLS
def test_a_stream_of_another_device(world, call):  # noqa: F811
    refused(world, call, stream=types.SimpleNamespace(cuda_stream=5, device_index=1))
    call(stream=world.side)


@CALLS
def test_tensors_on_the_host(world, call, monkeypatch):  # noqa: F811
    monkeypatch.setattr(Tensor, "get_device", lambda self: -1)
    refused(world, call)


def host_gemm(**more):
    mmq.q4K_gemm_host(Tensor((4, 256), torch.float32), Tensor(512 * 144, torch.uint8), 512, **more)


@pytest.mark.parametrize("call", [attention, moe, host_gemm], ids=lambda c: c.__name__)
def test_a_workspace_that_is_not_contiguous(world, call):  # noqa: F811
    """Its values reach past its storage (expanded), or lie between another's (strided)."""
    for stride in ((0,), (2,)):
        refused(world, call, workspace=Tensor(1 << 20, torch.uint8, stride=stride))
    call(workspace=Tensor(1 << 20, torch.uint8))


f16, i32 = torch.float16, torch.int32


def attend(q, k_prefix, v_prefix, kv, D):
    T = q.shape[0]
    mmq.shared_prefix_attention(q, k_prefix, v_prefix, Tensor((8, 16, kv, D), f16), Tensor((8, 16, kv, D), f16),
                                Tensor((T, 2), i32), Tensor(T, i32))


@pytest.mark.parametrize("q,k,v", [
    (((3, 4, 64), None), ((50, 1, 64), (64, 50 * 64, 1)), ((50, 1, 64), None)),       # one kv head: no step from head to head
    (((3, 4, 64), None), ((1, 2, 64), (999, 64, 1)), ((1, 2, 64), (128, 64, 1))),     # one key: none from token to token
    (((3, 1, 64), (512, 8, 1)), ((50, 1, 64), None), ((50, 1, 64), None)),            # one head
])
def test_strides_of_a_single_entry_do_not_matter(world, q, k, v):  # noqa: F811
    attend(Tensor(q[0], f16, stride=q[1]), Tensor(k[0], f16, stride=k[1]), Tensor(v[0], f16, stride=v[1]), k[0][1], 64)
    p = next(args[0] for name, args in world.lib.calls if name == "mmq_shared_prefix_attention")
    assert (p.prefix_token_stride, p.prefix_head_stride) == ((k[0][1] * 64 if k[0][0] == 1 else 64), 64)


@pytest.mark.parametrize("q,k,v", [
    (((3, 4, 64), (256, 32, 1)), ((50, 2, 64), None), ((50, 2, 64), None)),
    (((3, 4, 64), None), ((50, 2, 64), (128, 64, 1)), ((50, 2, 64), (256, 64, 1))),
    (((3, 4, 64), None), ((50, 2, 64), (128, 64, 1)), ((50, 2, 64), (128, 128, 1))),
    (((3, 4, 64), None), ((50, 2, 64), (128, 64, 1)), ((50, 2, 64), (128, 64, 2))),
    (((3, 4, 64), None), ((50, 2, 64), None), ((50, 128), None)),
])
def test_strides_that_differ_are_refused(world, q, k, v):  # noqa: F811
    with pytest.raises(mmq.MMQError):
        attend(Tensor(q[0], f16, stride=q[1]), Tensor(k[0], f16, stride=k[1]), Tensor(v[0], f16, stride=v[1]), 2, 64)
    assert not world.lib.calls
