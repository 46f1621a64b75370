"""The mixture-of-experts calls allocate no device memory: with outputs and workspace given, neither torch's allocator
nor the device's free memory changes over calls after the first (at which CUDA loads the kernels)."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def layer_calls(T, k, E, H, I):
    gen = torch.Generator(device="cuda").manual_seed(T)
    e = lambda *s, d=torch.uint8: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    x = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    res = torch.randn((T, H), device="cuda", generator=gen).bfloat16()
    g = torch.ones(H, device="cuda").bfloat16()
    q, sf, h, y = e(T, H), e(mx.sf_bytes(T, H, 32)), e(T, H, d=torch.bfloat16), e(T, H, d=torch.bfloat16)
    z = torch.randn((T, E), device="cuda", generator=gen)
    ids, w = e(T, k, d=torch.int32), e(T, k, d=torch.float32)
    w13, s13, _ = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, 2 * I, H, "cuda") for _ in range(E))))
    w2, s2, _ = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, H, I, "cuda") for _ in range(E))))
    out, ws = e(T, H, d=torch.bfloat16), mx.moe_experts_workspace(T, k, E, H, I)

    def run():
        mx.mxfp8_add_rmsnorm_quantize(x, g, 1e-6, residual=res, H=h, Y=y, Aq=q, A_sf=sf)
        mx.moe_route(z, k, ids=ids, weights=w)
        mx.mxfp4_moe_experts(q, sf, ids, w, w13, s13, w2, s2, out=out, workspace=ws)
    return run


@pytest.mark.parametrize("T,k,E,H,I", [(3, 2, 8, 256, 128), (400, 3, 4, 256, 128), (6000, 2, 8, 128, 128)])
def test_no_device_memory_is_allocated(T, k, E, H, I):
    run = layer_calls(T, k, E, H, I)
    run()
    torch.cuda.synchronize()
    held, requests = torch.cuda.memory_allocated(), torch.cuda.memory_stats()["allocation.all.allocated"]
    free = torch.cuda.mem_get_info()[0]
    for _ in range(5):
        run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == requests
    assert torch.cuda.mem_get_info()[0] == free
    assert mx.get_device_error() == 0
