"""The calls around a layer's attention allocate no device memory: with outputs and workspace given, neither torch's
allocator nor the device's free memory changes over calls after the first (at which CUDA loads the kernels)."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def calls(T):
    gen = torch.Generator(device="cuda").manual_seed(T)
    rn = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    K, N, R, L, E, H, I, k = 256, 128, 16, 3, 4, 256, 128, 2
    base, x, a, b = rn(T, N).bfloat16(), rn(T, K).bfloat16(), rn(L, R, K).bfloat16(), rn(L, N, R).bfloat16()
    ids = torch.randint(-1, L, (T,), device="cuda", generator=gen).to(torch.int32)
    c, ws = torch.empty_like(base), mx.lora_workspace(T, K, R, L)
    q, kk = rn(T, 4, 64).bfloat16(), rn(T, 1, 64).bfloat16()
    qo, ko, w = torch.empty_like(q), torch.empty_like(kk), rn(64).bfloat16()
    table, pos = rn(100, 64), torch.randint(0, 100, (T,), device="cuda")
    w13, s13, _ = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, 2 * I, H, "cuda") for _ in range(E))))
    w2, s2, _ = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, H, I, "cuda") for _ in range(E))))
    t = min(T, 16)
    h, out = torch.empty_like(x[:t]), torch.empty_like(x[:t])
    idx, wt = torch.empty((t, k), dtype=torch.int32, device="cuda"), torch.empty((t, k), device="cuda")
    norm, router, lws = rn(H).bfloat16(), rn(E, H).bfloat16(), mx.moe_layer_workspace(t, k, E, H, I)

    def run():
        mx.lora_add(base, x, a, b, ids, C=c, workspace=ws)
        mx.qk_norm_rope(q, kk, table, pos, w, w, q_out=qo, k_out=ko)
        mx.mxfp4_moe_layer(x[:t], norm, router, w13, s13, w2, s2, k, residual=x[:t], H=h, out=out, ids=idx, weights=wt,
                           workspace=lws)
    return run


@pytest.mark.parametrize("T", [3, 40, 500])
def test_no_device_memory_is_allocated(T):
    run = calls(T)
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
