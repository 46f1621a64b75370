"""Batches so long that a warp takes several rounds of heads, queries and keys of a token among them: the ring of heads
on their way wraps, beside and in place."""
import pytest
import torch

import layer_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from test_gpu_qk_norm_rope import check, make, rope_table  # noqa: E402


@pytest.mark.parametrize("T,Hq,Hk,D,rot,interleaved,norm,dtype", [
    # rounds a warp takes on 152 SMs: T * ceil(heads / G) / (72 * 152), G = 8, 4 or 2 heads side by side
    (6000, 70, 33, 64, 64, False, True, torch.float16), (6000, 70, 33, 56, 24, True, False, torch.bfloat16),
    (4096, 61, 9, 128, 128, False, True, torch.bfloat16), (4100, 40, 30, 96, 32, True, True, torch.float16),
    (4096, 25, 4, 192, 64, True, True, torch.bfloat16), (4099, 23, 7, 256, 128, False, False, torch.bfloat16),
])
def test_several_rounds_of_heads(T, Hq, Hk, D, rot, interleaved, norm, dtype):
    q, k, (wq, wk), gen = make(T, Hq, Hk, D, dtype)
    if not norm:
        wq = wk = None
    table = rope_table(5000, rot)
    pos = torch.randint(0, 5000, (T,), device="cuda", generator=gen)
    qo, ko = mx.qk_norm_rope(q, k, table, pos, wq, wk, 1e-6, interleaved)
    for t0 in range(0, T, 1024):
        s = slice(t0, t0 + 1024)
        check(qo[s], layer_ref.head_norm_rope(q[s], wq, table, pos[s], 1e-6, interleaved))
        check(ko[s], layer_ref.head_norm_rope(k[s], wk, table, pos[s], 1e-6, interleaved))
    values = q._base[:, (Hq + Hk) * D:].clone()
    mx.qk_norm_rope(q, k, table, pos, wq, wk, 1e-6, interleaved, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(q._base[:, (Hq + Hk) * D:], values)


def test_few_tokens_are_the_first_of_many():
    """A token's heads are the same bits whether its warps take one round or several."""
    q, k, (wq, wk), _ = make(8000, 64, 8, 128, torch.bfloat16)
    table, pos = rope_table(8000, 128), torch.arange(8000, device="cuda")
    many = mx.qk_norm_rope(q, k, table, pos, wq, wk)
    few = mx.qk_norm_rope(q[:50], k[:50], table, pos[:50], wq, wk)
    last = mx.qk_norm_rope(q[-50:], k[-50:], table, pos[-50:], wq, wk)
    assert all(torch.equal(a[:50], b) for a, b in zip(many, few))
    assert all(torch.equal(a[-50:], b) for a, b in zip(many, last))
