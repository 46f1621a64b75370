"""Layers that run one after another share both workspaces: that of the chain of calls, and that of the calls of few tokens."""
import pytest
import torch

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from block_scaled_fp4_mxfp4_gb300 import moe_layer  # noqa: E402


def test_layers_share_the_workspace_of_few_tokens():
    how = dict(E=8, H=512, I=256, k=2, max_tokens=20, few_tokens=16)
    first = moe_layer.random_layer(seed=1, **how)
    apart = moe_layer.random_layer(seed=2, **how)
    shared = moe_layer.random_layer(seed=2, workspace=first.workspace, few_workspace=first.few_workspace, **how)
    assert shared.few_workspace is first.few_workspace and shared.workspace is first.workspace
    gen = torch.Generator(device="cuda").manual_seed(0)
    for T in (1, 16, 20, 7):
        x = torch.randn((T, 512), device="cuda", generator=gen).bfloat16()
        want = apart(*first(x))
        got = shared(*first(x))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # one made for more tokens serves fewer; one that is too small is refused
    assert moe_layer.random_layer(seed=2, **dict(how, few_tokens=3), few_workspace=first.few_workspace).few_tokens == 3
    with pytest.raises(ValueError):
        moe_layer.random_layer(seed=2, few_workspace=first.few_workspace[:-1], **how)
    assert moe_layer.random_layer(seed=2, **dict(how, few_tokens=0)).few_workspace is None
    assert mx.get_device_error() == 0
