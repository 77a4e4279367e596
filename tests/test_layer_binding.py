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
