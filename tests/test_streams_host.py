"""Which stream's memory a call takes what the caller leaves to it to allocate from,
without a GPU: the library, the allocator and the streams are stand-ins."""
import types

import pytest
import torch

from block_scaled_fp4_mxfp4_gb300 import build as libbuild

libbuild.build()
from block_scaled_fp4_mxfp4_gb300 import mxfp4 as mx  # noqa: E402


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


CALLER, SIDE = Stream(11), Stream(22)


class Tensor(torch.Tensor):
    """Host memory that says it is on a GPU, and for which streams it was recorded."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.recorded = getattr(self, "recorded", ()) + (stream,)


class World:
    """Allocations and launches, each with the stream it was made on."""

    def __init__(self):
        self.stack, self.allocated, self.launched = [CALLER], [], []

    def make(self, shape, dtype=None, device=None):
        t = torch.zeros(shape, dtype=dtype).as_subclass(Tensor)
        self.allocated.append((self.stack[-1], t))
        return t

    def stream(self, s):
        world = self

        class Context:
            def __enter__(self):
                world.stack.append(s)

            def __exit__(self, *exc):
                world.stack.pop()
        return Context()

    def call(self, name):
        def run(*args):
            if name.endswith("_bytes"):
                return 640
            s = args[-1]
            self.launched.append(getattr(s, "value", s))
            return 0
        return run


@pytest.fixture
def world(monkeypatch):
    w = World()
    fake = types.SimpleNamespace(**{n: getattr(torch, n) for n in (
        "bfloat16", "float16", "float32", "float64", "uint8", "int32", "Tensor")})
    fake.empty = fake.zeros = w.make
    fake.cuda = types.SimpleNamespace(stream=w.stream, current_stream=lambda device=None: w.stack[-1])
    monkeypatch.setattr(mx, "torch", fake)
    monkeypatch.setattr(mx, "_raw_stream", lambda device: w.stack[-1].cuda_stream)

    class Lib:
        def __getattr__(self, name):
            return w.call(name)
    monkeypatch.setattr(mx, "_lib", Lib())
    return w


def t(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype).as_subclass(Tensor)


def group(n, act):
    a = t(4, 64, dtype=torch.bfloat16) if act else t(4, 32)
    return [dict(a=a, sfa=t(512), b=t(8, 32), sfb=t(512), c=t(4, 8, dtype=torch.float16), k=64) for _ in range(n)]


bf = dict(dtype=torch.bfloat16)
CALLS = {
    "mxfp4_quantize": lambda s: mx.mxfp4_quantize(t(4, 64, **bf), stream=s),
    "nvfp4_quantize": lambda s: mx.nvfp4_quantize(t(4, 64, **bf), stream=s),
    "mxfp4_rmsnorm_quantize": lambda s: mx.mxfp4_rmsnorm_quantize(t(4, 64, **bf), t(64, **bf), stream=s, stats=True),
    "mxfp4_gemm_a4w4": lambda s: mx.mxfp4_gemm_a4w4(t(4, 32), t(512), t(8, 32), t(512), 64, stream=s),
    "mxfp4_gemm_a4w4_ex": lambda s: mx.mxfp4_gemm_a4w4_ex(t(4, 32), t(512), t(8, 32), t(512), 64, stream=s),
    "mxfp4_quant_gemm_fused": lambda s: mx.mxfp4_quant_gemm_fused(t(4, 64, **bf), t(8, 32), t(512), stream=s),
    "nvfp4_quant_gemm_fused": lambda s: mx.nvfp4_quant_gemm_fused(t(4, 64, **bf), t(8, 32), t(512), stream=s),
    "mxfp4_group_gemm": lambda s: mx.mxfp4_group_gemm(group(17, False), stream=s),
    "nvfp4_group_gemm": lambda s: mx.nvfp4_group_gemm(group(17, False), stream=s),
    "nvfp4_group_quant_gemm": lambda s: mx.nvfp4_group_quant_gemm(group(2, True), stream=s),
    "mxfp8_add_rmsnorm_quantize": lambda s: mx.mxfp8_add_rmsnorm_quantize(
        t(4, 64, **bf), t(64, **bf), residual=t(4, 64, **bf), want_y=True, stream=s),
    "moe_route": lambda s: mx.moe_route(t(4, 16, dtype=torch.float32), 2, stream=s),
    "mxfp4_moe_experts": lambda s: mx.mxfp4_moe_experts(
        t(4, 128), t(512), t(4, 2, dtype=torch.int32), t(4, 2, dtype=torch.float32), t(3, 256, 64), t(3 * 1024),
        t(3, 128, 64), t(3 * 512), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_belongs_to_the_stream_it_runs_on(world, name):
    """Otherwise a workspace that the call drops, or an output that the caller drops, is given to work of the current
    stream while the kernels on `stream` still use it; and a buffer fresh from the current stream is written while that
    stream's work still reads it."""
    result = CALLS[name](SIDE)
    assert world.launched and set(world.launched) == {SIDE.cuda_stream}
    assert world.allocated
    for stream, _ in world.allocated:
        assert stream is SIDE
    # outputs are for the caller too: they are kept from reuse until the caller's stream is past its use of them
    made = {a.data_ptr() for _, a in world.allocated if hasattr(a, "recorded")}
    outs = result if isinstance(result, (tuple, list)) else [result]
    given = {g.data_ptr() for g in outs}
    assert made <= given
    if "group" not in name:
        assert made == given
    for _, a in world.allocated:
        assert getattr(a, "recorded", (CALLER,)) == (CALLER,)


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_is_the_default(world, name):
    CALLS[name](None)
    assert set(world.launched) == {CALLER.cuda_stream}
    for stream, a in world.allocated:
        assert stream is CALLER and not hasattr(a, "recorded")
