"""Values next to the end of fp32 inside the adapters and the layer of few tokens: what is held in parts (two bf16, digits)
is good to what the parts can hold."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from test_gpu_moe_few import call, make  # noqa: E402
from test_gpu_moe_few_products import layer_sum, open_codes, worst  # noqa: E402


@pytest.mark.parametrize("T", [1, 16, 40, 70, 300, 4000])
@pytest.mark.parametrize("power", [0, -60, -110, -120, -124])
def test_low_parts_of_small_products_are_kept(T, power):
    """u = 2^power (1 + 2^-9): the second bf16 is 2^(power - 9), 2^-133 at the least. base takes the first one away."""
    x = torch.zeros((T, 64), device="cuda")
    x[:, 0], x[:, 1] = 2.0 ** -60, 2.0 ** -69
    a = torch.zeros((1, 8, 64), device="cuda")
    a[0, 3, :2] = 2.0 ** (power + 60)
    b = torch.zeros((1, 64, 8), device="cuda")
    b[0, :, 3] = 2.0 ** 100
    base = torch.full((T, 64), -2.0 ** (power + 100), device="cuda").bfloat16()
    c = mx.lora_add(base, x.bfloat16(), a.bfloat16(), b.bfloat16(), torch.zeros(T, dtype=torch.int32, device="cuda"))
    assert bool((c.double() == 2.0 ** (power + 91)).all())


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 256, 384), (16, 1, 1, 384, 1024), (6, 12, 3, 512, 128)])
@pytest.mark.parametrize("power", [-50, -56, -60, -64, -68])
def test_activations_of_small_rows(T, E, k, H, I, power):
    """Rows far below eps: y is about 2^(power + 10), an activation about the square of that. Its value enters to 2^-127."""
    s = make(T, E, H, I, seed=8)
    s["x"], s["res"] = s["x"] * 2.0 ** power, s["res"] * 2.0 ** power
    out, _, ids, w = call(s, k)
    _, y = moe_ref.add_rmsnorm(s["x"], s["res"], s["weight"], 1e-6)
    ref, bound = layer_sum(*open_codes(y, 4 * 2.0 ** -24 * y.abs()), ids, w, *s["v"])
    sizes = s["v"][1].abs().sum(-1)                                     # [E, H]
    bound += 2.0 ** -127 * (sizes[ids.long()] * w.double()[..., None]).sum(1) + 2.0 ** -134     # bf16's half step
    assert worst(out, ref, bound) <= 1.0
