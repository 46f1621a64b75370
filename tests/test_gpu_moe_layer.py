"""The mixture-of-experts layer as a user runs it: its three calls chained, captured
into a graph, and each step checked against its definition on the step's own
inputs; and the kernels' way out of a wait that runs out."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from block_scaled_fp4_mxfp4_gb300 import moe_layer  # noqa: E402


@pytest.mark.parametrize("T", [1, 37, 400])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_layer_is_its_steps(T, score):
    E, H, I, k = 8, 256, 128, 3
    bias = torch.linspace(-0.02, 0.02, E, device="cuda")
    layer = moe_layer.random_layer(E, H, I, k, T, seed=T, score=score, bias=bias, groups=4, topk_groups=3)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    res = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    out, h = layer(x, res)
    q, sf, h2, y = mx.mxfp8_add_rmsnorm_quantize(x, layer.norm, layer.eps, residual=res, want_y=True)
    assert torch.equal(h, h2)
    ids, w = mx.moe_route(y @ layer.router.T, k, bias=bias, **layer.how)
    ri, _ = moe_ref.route(y @ layer.router.T, k, score, bias, 4, 3, 2, True, 1.0)
    assert torch.equal(ids.cpu(), ri)
    values = moe_ref.e4m3_values(q) * torch.exp2(
        sf[moe_ref.blocked_index(T, H // 32, "cuda")].double() - 127).repeat_interleave(32, 1)
    deq = lambda c, s, N, K: moe_ref.e2m1_values(c) * torch.exp2(  # noqa: E731
        s[:, moe_ref.blocked_index(N, K // 32, "cuda")].double() - 127).repeat_interleave(32, 2)
    ref, bound = moe_ref.experts(values, ids, w, deq(layer.w13, layer.s13, 2 * I, H), deq(layer.w2, layer.s2, H, I))
    assert float(((out.double() - ref).abs() / bound).max()) <= 1.0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _ = layer(x, res)
    x.add_(res)
    graph.replay()
    fresh, _ = layer(x, res)
    torch.cuda.synchronize()
    assert torch.equal(captured, fresh) and mx.get_device_error() == 0


def test_layer_without_a_residual_and_fewer_tokens_than_it_has_room_for():
    layer = moe_layer.random_layer(4, 128, 128, 2, 64)
    x = torch.randn((5, 128), device="cuda").bfloat16()
    out, h = layer(x)
    assert h is x and out.shape == (5, 128)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0


@pytest.mark.parametrize("T,E", [(6, 4), (300, 2)])
def test_waits_that_run_out_end_the_call_and_are_reported(T, E):
    """A limit of one nanosecond makes waits of the products give up: the call ends, the code says so, and the next call
    is right. Small tiles and large ones."""
    layer = moe_layer.random_layer(E, 512, 256, 2, T)
    x = torch.randn((T, 512), device="cuda").bfloat16()
    want, _ = layer(x)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0
    old = mx.set_wait_limit_ns(1)
    try:
        layer(x)
        torch.cuda.synchronize()
    finally:
        mx.set_wait_limit_ns(0)
    assert old == 2_000_000_000
    assert 48 < mx.get_device_error() < 64
    again, _ = layer(x)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0 and torch.equal(again, want)
