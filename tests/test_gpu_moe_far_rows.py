"""Activation rows whose offsets pass 32 bits, in bytes and in units of 16 of them."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def test_rows_of_activations_far_apart():
    T, H, I, apart = 257, 256, 128, 1 << 28                    # 69 GB, of which 66 KB are touched
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(1)
    xq, xs, _ = moe_ref.random_mxfp8(gen, T, H, "cuda")
    far = torch.empty((T, apart), dtype=torch.uint8, device="cuda")[:, :H]
    far.copy_(xq)
    for E in (16, 4):                                          # small tiles, large tiles
        w13, s13, _ = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, 2 * I, H, "cuda") for _ in range(E))))
        w2, s2, _ = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, H, I, "cuda") for _ in range(E))))
        ids = torch.randint(0, E, (T, 1), generator=gen, device="cuda").to(torch.int32)
        w = torch.rand((T, 1), generator=gen, device="cuda")
        want = mx.mxfp4_moe_experts(xq, xs, ids, w, w13, s13, w2, s2)
        got = mx.mxfp4_moe_experts(far, xs, ids, w, w13, s13, w2, s2)
        torch.cuda.synchronize()
        assert mx.get_device_error() == 0 and torch.equal(got, want)
    del far
    torch.cuda.empty_cache()
