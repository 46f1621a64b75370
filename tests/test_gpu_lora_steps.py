"""Adapters of long batches whose blocks take many steps of channels (the rings of B and base wrap, an accumulator is used
again), and of pools in which a batch uses few of the adapters that are held."""
import pytest
import torch

import layer_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from test_gpu_lora import case, check  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,R,L", [
    # steps of 64 channels a block: (N / 64) / blocks, with the blocks of a tile that make the waves of 304 shortest
    (4096, 264, 2120, 40, 3), (4096, 72, 4168, 64, 2), (6000, 136, 1096, 24, 7), (9001, 64, 2056, 8, 5),
])
def test_many_steps_of_channels(T, K, N, R, L, dtype):
    args = case(T, K, N, R, L, dtype, ragged=True)
    base, x, a, b, ids, scales, ranks = args
    order = torch.argsort(ids, stable=True)          # prompts, one after another
    ids.copy_(ids[order])
    c = mx.lora_add(*args)
    check(c, layer_ref.lora(*args))
    assert torch.equal(c[ids < 0], base[ids < 0])
    inplace = base.clone()
    mx.lora_add(inplace, x, a, b, ids, scales, ranks, C=inplace)
    assert torch.equal(inplace, c)
    # mixed ids, the same tokens: the same rows
    mix = torch.randperm(T, device="cuda")
    mixed = mx.lora_add(base[mix].contiguous(), x[mix].contiguous(), a, b, ids[mix].contiguous(), scales, ranks)
    assert torch.equal(mixed, c[mix])


@pytest.mark.parametrize("T,K,N,R,L,used", [
    (1, 512, 264, 16, 4096, [4095]), (64, 1032, 520, 32, 64, [17]), (64, 264, 136, 16, 4096, [2000]), (65, 264, 136, 16, 4096, [0]),
    (700, 264, 136, 72, 512, [5, 511]), (4096, 520, 264, 16, 4096, [4095]), (4096, 264, 2120, 64, 512, [0, 7, 300, 511]),
    (10000, 72, 264, 8, 4096, [1, 4000]),
])
def test_few_of_the_adapters_that_are_held(T, K, N, R, L, used):
    """The result is that of a pool which holds nothing else, within the arithmetic's bound."""
    base, x, a, b, _, scales, ranks = case(T, K, N, R, L, ragged=True)
    ids = torch.tensor(used, dtype=torch.int32, device="cuda")[torch.arange(T, device="cuda") * len(used) // T]
    ranks[used] = torch.tensor([R, max(1, R - 3), 1, R], dtype=torch.int32, device="cuda")[:len(used)]
    c = mx.lora_add(base, x, a, b, ids, scales, ranks)
    own = torch.arange(len(used), dtype=torch.int32, device="cuda")[torch.arange(T, device="cuda") * len(used) // T]
    small = (base, x, a[used].contiguous(), b[used].contiguous(), own, scales[used].contiguous(), ranks[used].contiguous())
    ref = layer_ref.lora(*small)
    check(c, ref)
    check(mx.lora_add(*small), ref)


@pytest.mark.parametrize("T", [1, 16, 333, 4096])
def test_the_same_bits_every_time(T):
    args = case(T, 1024, 520, 32, 9, ragged=True)
    want = mx.lora_add(*args)
    for _ in range(20):
        assert torch.equal(mx.lora_add(*args), want)
