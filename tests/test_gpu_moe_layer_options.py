"""What a mixture-of-experts layer can be told: how a group of experts is ranked, and whose workspace it uses."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from block_scaled_fp4_mxfp4_gb300 import moe_layer  # noqa: E402


@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_ranked_by_their_best_expert_or_two(group_top):
    E, H, I, k, T = 16, 256, 128, 3, 60
    bias = torch.linspace(0.3, -0.3, E, device="cuda")
    layer = moe_layer.random_layer(E, H, I, k, T, seed=1, score="sigmoid", bias=bias, groups=4, topk_groups=2,
                                   group_top=group_top)
    x = torch.randn((T, H), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).bfloat16()
    out, _ = layer(x)
    q, sf, _, y = mx.mxfp8_add_rmsnorm_quantize(x, layer.norm, layer.eps, want_y=True)
    logits = y @ layer.router.T
    ids, w = moe_ref.route(logits, k, "sigmoid", bias, 4, 2, group_top, True, 1.0)
    other, _ = moe_ref.route(logits, k, "sigmoid", bias, 4, 2, 3 - group_top, True, 1.0)
    assert not torch.equal(ids, other)
    ours = mx.moe_route(logits, k, "sigmoid", bias, 4, 2, group_top)
    assert torch.equal(ours[0].cpu(), ids)
    want = mx.mxfp4_moe_experts(q, sf, *ours, layer.w13, layer.s13, layer.w2, layer.s2)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and mx.get_device_error() == 0


def test_layers_share_a_workspace():
    args = (8, 256, 128, 2, 300)
    alone = [moe_layer.random_layer(*args, seed=i) for i in range(3)]
    first = moe_layer.random_layer(*args, seed=0)
    shared = [first] + [moe_layer.random_layer(*args, seed=i, workspace=first.workspace) for i in (1, 2)]
    assert all(l.workspace is first.workspace for l in shared)
    for T in (300, 7):
        x = torch.randn((T, 256), device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)).bfloat16()

        def run(layers):
            h, out = x, None
            for l in layers:
                out, h = l(h, out)
            return out, h
        for a, b in zip(run(alone), run(shared)):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0


def test_a_workspace_that_is_too_small_is_refused():
    small = moe_layer.random_layer(4, 128, 128, 2, 10)
    with pytest.raises(ValueError):
        moe_layer.random_layer(4, 128, 128, 2, 1000, workspace=small.workspace)
