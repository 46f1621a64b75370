"""The weighted sum over a token's experts takes the products as the tensor cores
accumulate them, in fp32, and rounds once.

The operands are made so that every step is exact: a token is one unit, so its
gate is one element of G, 96, where silu is the identity in fp32 (exp(-96) vanishes
beside 1) and its activations are 96 times the E2M1 values of U, which E4M3 holds.
A product row is then a sum of multiples of 24 up to 2^15 of them: 15 bits, which
fp32 holds and bf16 (8 bits) or fp16 (11) do not. The weights are small multiples
of 1/4, of both signs. So the sum is exact in fp32, and the result is that of 64
bits rounded once, bit for bit."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def operands(T, k, E, H, I, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = lambda *s: torch.randint(0, 256, s, generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)  # noqa: E731
    sf = lambda n, K, b: torch.full((n, mx.sf_bytes(K[0], K[1], 32)), b, dtype=torch.uint8, device="cuda")  # noqa: E731
    at = torch.randint(0, H, (T,), generator=gen, device="cuda")
    xq = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    xq[torch.arange(T, device="cuda"), at] = 0x38                                # 1.0
    xs = torch.full((mx.sf_bytes(T, H, 32),), 127, dtype=torch.uint8, device="cuda")
    w13 = torch.cat([torch.full((E, I, H // 2), 0x77, dtype=torch.uint8, device="cuda"), codes(E, I, H // 2)], 1)
    s13 = sf(E, (2 * I, H), 127)
    g_rows = moe_ref.blocked_index(2 * I, H // 32, "cuda")[:I].reshape(-1)
    s13[:, g_rows] = 131                                                         # 6 * 2^4 = 96
    w2, s2 = codes(E, H, I // 2), sf(E, (H, I), 127)
    ids = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)]).to(torch.int32)
    w = (torch.randint(1, 8, (T, k), generator=gen, device="cuda") *
         (1 - 2 * torch.randint(0, 2, (T, k), generator=gen, device="cuda"))).float() / 4
    act = 96 * moe_ref.e2m1_values(w13[:, I:])                                   # [E, I, H]: of a unit at column h
    v2 = moe_ref.e2m1_values(w2)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        ref.index_add_(0, tok, (act[e][:, at[tok]].T @ v2[e].T) * w[tok, slot].double()[:, None])
    return (xq, xs, ids, w, w13, s13, w2, s2), ref


@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 128, 128), (5, 3, 4, 256, 128), (50, 4, 8, 384, 256),
                                       (300, 2, 2, 256, 128), (700, 3, 4, 384, 256)])
def test_sum_over_experts_is_rounded_once(T, k, E, H, I):
    a, ref = operands(T, k, E, H, I, T + E)
    # the inputs are what the docstring says: the sum in fp32 is exact, and the products need more than bf16 or fp16
    assert torch.equal(ref.float().double(), ref) and not torch.equal(ref.half().double(), ref)
    out = mx.mxfp4_moe_experts(*a)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0
    assert torch.equal(out, ref.bfloat16())
