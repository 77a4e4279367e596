"""Memory that a call with stream= allocates comes from that stream's pool.

The current stream's pool may hand out a block that work queued on the current
stream still uses (the workspace of the call before, say), and the given stream
does not wait for that work.  Shown without a GPU: stand-ins for the tensors,
the library and the allocator, which notes the stream each block is for.
"""
import contextlib
import types

import pytest

import q4_q8_int8_gb300 as mmq

torch = pytest.importorskip("torch")


class Tensor:
    """What the binding asks of a CUDA tensor; no memory."""
    made = 0

    def __init__(self, shape, dtype, stride=None):
        self.shape = torch.Size(shape if isinstance(shape, (tuple, list)) else (shape,))
        self.dtype, self.device = dtype, "cuda:0"
        Tensor.made += 1
        self.at = Tensor.made << 32
        steps, n = [], 1
        for d in reversed(self.shape):
            steps.insert(0, n)
            n *= d
        self.steps, self.n = stride or tuple(steps), n
        self.contiguous = stride is None

    def get_device(self):
        return 0

    def stride(self, i=None):
        return self.steps if i is None else self.steps[i]

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.n

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self.at

    def record_stream(self, stream):
        pass


class Library:
    """Every entry point: a size where one is asked for, else success."""
    calls = None

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith(("workspace", "bytes")) else 0
        return entry


@pytest.fixture
def world(monkeypatch):
    """(streams that blocks were allocated for, the library's calls)."""
    now, blocks, lib = [None], [], Library()

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s
        yield
        now[0] = before

    def empty(shape, dtype=None, device=None, pin_memory=False):
        if not pin_memory:
            blocks.append(now[0])
        return Tensor(shape, dtype)

    current = types.SimpleNamespace(cuda_stream=1, device_index=0, synchronize=lambda: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(mmq, "_lib", lib)
    monkeypatch.setattr(mmq, "load_library", lambda *a: lib)
    return types.SimpleNamespace(blocks=blocks, lib=lib, side=types.SimpleNamespace(
        cuda_stream=77, device_index=0, synchronize=lambda: None))


f16, f32, i32, u8 = torch.float16, torch.float32, torch.int32, torch.uint8


def rope(**more):
    mmq.qk_norm_rope(Tensor((3, 6 * 64), f32), 4, Tensor((9, 32), f32), Tensor((9, 32), f32), Tensor(3, i32),
                     Tensor(3, i32), Tensor((8, 1, 64), f16), Tensor((8, 1, 64), f16), **more)


def attention(**more):
    mmq.shared_prefix_attention(Tensor((3, 4, 64), f16), Tensor((50, 2, 64), f16), Tensor((50, 2, 64), f16),
                                Tensor((8, 16, 2, 64), f16), Tensor((8, 16, 2, 64), f16), Tensor((3, 2), i32),
                                Tensor(3, i32), **more)


def moe(**more):
    mmq.q4K_moe(Tensor((3, 512), f32), Tensor((8, 512), f32), Tensor((8, 512, 2, 144), u8), Tensor((8, 512, 1, 144), u8), 2,
                **more)


OPERATORS = [(rope, 1), (attention, 2), (moe, 4)]


@pytest.mark.parametrize("call,blocks", OPERATORS, ids=lambda v: getattr(v, "__name__", None))
def test_layer_operators_allocate_on_the_given_stream(world, call, blocks):
    call(stream=world.side)
    assert world.blocks == [world.side] * blocks
    name, args = world.lib.calls[-1]
    assert args[-1] == 77
    world.blocks.clear()
    call()
    assert world.blocks == [None] * blocks
    assert world.lib.calls[-1][1][-1] == 1


def q8(M, K):
    return Tensor((M, K), torch.int8), Tensor((M, K // 32), f32), Tensor((M, K // 32), i32)


W = 512 * 256 // 256 * 144      # bytes of a q4_K matrix, 512 x 256
GEMMS = [
    ("quantize_q8_1", lambda **m: mmq.quantize_q8_1(Tensor((4, 256), f32), **m), 3),
    ("quantize_q8_1_tcop", lambda **m: mmq.quantize_q8_1_tcop(Tensor((4, 256), f32), **m), 4),
    ("q4K_gemm_tcop", lambda **m: mmq.q4K_gemm_tcop(Tensor(4096, u8), Tensor(W, u8), 4, 512, 256, **m), 1),
    ("q4K_gemm", lambda **m: mmq.q4K_gemm(q8(4, 256), Tensor(W, u8), 512, **m), 1),
    ("q4K_gemm_host", lambda **m: mmq.q4K_gemm_host(Tensor((4, 256), f32), Tensor(W, u8), 512, **m), 1),
    ("q4K_gemm_q8_1", lambda **m: mmq.q4K_gemm_q8_1(q8(4, 256), Tensor(W, u8), 512, **m), 4),
    ("q4K_block_dots", lambda **m: mmq.q4K_block_dots(q8(4, 256), Tensor(W, u8), 512, **m), 1),
    ("q4K_scaled_block_dots", lambda **m: mmq.q4K_scaled_block_dots(q8(4, 256), Tensor(W, u8), 512, **m), 1),
    ("interleave_rows_q4K", lambda **m: mmq.interleave_rows_q4K(Tensor(W, u8), Tensor(W, u8), 512, 256, **m), 1),
    ("q4K_gemm_swiglu_q8_1", lambda **m: mmq.q4K_gemm_swiglu_q8_1(q8(4, 256), Tensor(W, u8), 256, with_h=True, **m), 4),
    ("repack_q6K", lambda **m: mmq.repack_q6K(Tensor(512 * 210, u8), 512, 256, **m), 1),
    ("q6K_gemm", lambda **m: mmq.q6K_gemm(q8(4, 256), Tensor(512 * 224, u8), 512, **m), 1),
    ("q6K_block_dots", lambda **m: mmq.q6K_block_dots(q8(4, 256), Tensor(512 * 224, u8), 512, **m), 1),
    ("q6K_scaled_block_dots", lambda **m: mmq.q6K_scaled_block_dots(q8(4, 256), Tensor(512 * 224, u8), 512, **m), 1),
    ("dequantize_q4K_f16", lambda **m: mmq.dequantize_q4K_f16(Tensor(W, u8), 512, 256, **m), 1),
    ("convert_f16", lambda **m: mmq.convert_f16(Tensor((4, 256), f32), **m), 1),
    ("gemm_f16", lambda **m: mmq.gemm_f16(Tensor((4, 256), f16), Tensor((512, 256), f16), **m), 1),
]


@pytest.mark.parametrize("call,blocks", [g[1:] for g in GEMMS], ids=[g[0] for g in GEMMS])
def test_projections_allocate_on_the_given_stream(world, call, blocks):
    call(stream=world.side)
    assert world.blocks == [world.side] * blocks
    assert world.lib.calls[-1][1][-1].value == 77
    world.blocks.clear()
    call()
    assert world.blocks == [None] * blocks
    assert world.lib.calls[-1][1][-1].value == 1
