"""Calls given a stream other than the current one, with outputs and workspace left to the call: the current stream
allocates and fills memory of the same sizes right after each call, while the call's kernels still wait behind other
work on their stream, and results are as without `stream`."""
import pytest
import torch

import moe_ref
from block_scaled_fp4_mxfp4_gb300 import workloads as wl
from gpu_util import dev_bf16

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def moe_experts(T, k, E, H, I):
    gen = torch.Generator(device="cuda").manual_seed(T)
    xq, xs, _ = moe_ref.random_mxfp8(gen, T, H, "cuda")
    w13, s13, _ = zip(*(moe_ref.random_mxfp4(gen, 2 * I, H, "cuda") for _ in range(E)))
    w2, s2, _ = zip(*(moe_ref.random_mxfp4(gen, H, I, "cuda") for _ in range(E)))
    ids = torch.randint(0, E, (T, k), generator=gen, device="cuda").to(torch.int32)
    w = torch.rand((T, k), generator=gen, device="cuda")
    a = [xq, xs, ids, w] + [torch.stack(m) for m in (w13, s13, w2, s2)]
    need = mx.moe_experts_workspace_bytes(T, k, E, H, I)
    return lambda **kw: mx.mxfp4_moe_experts(*a, **kw), [need, T * H * 2]


def norm(M, K):
    x, res, w = (dev_bf16(wl.gen_bf16(7, i, m, K)) for i, m in enumerate((M, M, 1)))
    return (lambda **kw: mx.mxfp8_add_rmsnorm_quantize(x, w[0], residual=res, want_y=True, **kw),
            [2 * M * K, 2 * M * K, M * K, mx.sf_bytes(M, K, 32)])


def route(T, E, k):
    z = torch.randn((T, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    return lambda **kw: mx.moe_route(z, k, **kw), [4 * T * k, 4 * T * k]


def gemm(M, N, K):
    a, b = dev_bf16(wl.gen_bf16(8, 1, M, K)), dev_bf16(wl.gen_bf16(8, 2, N, K))
    qb, sb = mx.mxfp4_quantize(b)
    return lambda **kw: mx.mxfp4_quant_gemm_fused(a, qb, sb, **kw), [mx.workspace_bytes(M, N, K), 2 * M * N]


def quantize(M, K):
    a = dev_bf16(wl.gen_bf16(9, 1, M, K))
    return lambda **kw: mx.nvfp4_quantize(a, **kw), [M * K // 2, mx.sf_bytes(M, K, 16)]


@pytest.mark.parametrize("make", [
    lambda: moe_experts(40, 3, 8, 512, 256), lambda: moe_experts(400, 3, 4, 512, 256), lambda: norm(300, 2112),
    lambda: route(3000, 64, 6), lambda: gemm(16, 512, 4096), lambda: gemm(300, 512, 1024), lambda: quantize(256, 1024),
], ids=["experts_small", "experts_large", "norm", "route", "gemm_decode", "gemm", "quantize"])
def test_a_call_on_another_stream_keeps_its_memory(make):
    call, sizes = make()
    want = call()
    want = want if isinstance(want, tuple) else (want,)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    results = []
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)            # some 10 ms
        results.append(call(stream=side))
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0
    for got in results:
        for g, w in zip(got if isinstance(got, tuple) else (got,), want):
            if g is not None:
                assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
