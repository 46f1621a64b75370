"""Elements of a head that nothing turns: an infinity, a NaN or a negative zero there reaches no other element, whichever
vectors a lane holds side by side."""
import pytest
import torch

import layer_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from test_gpu_qk_norm_rope import make, rope_table  # noqa: E402


def check(got, want):
    """As for finite heads; infinities of the definition are met exactly."""
    z, bound = want
    assert torch.equal(torch.isnan(got), torch.isnan(z))
    far = torch.isinf(z)
    assert torch.equal(got[far].double(), z[far])
    rest = torch.isfinite(z)
    assert bool(((got.double() - z).abs()[rest] <= bound[rest]).all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 32), (40, 16), (96, 48), (128, 32), (192, 64), (256, 0), (256, 16)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_one_element_reaches_only_those_it_turns_with(value, D, rot, interleaved, norm):
    """Token i has the value in element i of one of its heads."""
    q, k, (wq, _), _ = make(D, 3, 2, D, torch.bfloat16)
    q = q.clone()
    at = torch.arange(D, device="cuda")
    q[at, at % 3, at] = value
    table, pos = (rope_table(300, rot), at + 1) if rot else (None, None)
    w = wq if norm else None
    got, gotk = mx.qk_norm_rope(q, k, table, pos, w, w, 1e-6, interleaved)
    want, wantk = (layer_ref.head_norm_rope(x, w, table, pos, 1e-6, interleaved) for x in (q, k))
    check(got, want)
    check(gotk, wantk)
    if not norm:
        # all but the element, and what it turns with, is what it is without it
        assert int((~torch.isfinite(got)).sum()) == (D if not rot else D + rot)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 0), (192, 64), (72, 16)])
def test_what_nothing_turns_keeps_its_bits_without_a_norm(D, rot, interleaved, dtype):
    q, k, _, _ = make(9, 5, 1, D, dtype)
    q = torch.where(torch.rand_like(q, dtype=torch.float32) < 0.3, torch.tensor(-0.0, device="cuda"), q.float()).to(dtype)
    table, pos = (rope_table(30, rot), torch.arange(9, device="cuda")) if rot else (None, None)
    got, _ = mx.qk_norm_rope(q, k, table, pos, interleaved=interleaved)
    assert torch.equal(got[..., rot:].view(torch.int16), q[..., rot:].view(torch.int16))
