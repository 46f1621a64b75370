"""The router's logits in the layer of few tokens, where the sums that make them lose most."""
import pytest
import torch

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from test_gpu_moe_few import call, make  # noqa: E402


def test_small_terms_after_large_ones_in_the_routers_products():
    """In every 16 channels a term of +-c and 15 far smaller ones, which an addition to it would lose. A product passes three
    additions in a chain of four, two that join the chains and two that join four lanes: seven of 2^-24 of the sum of
    sizes at most. Sums of 64 channels are then added in two floats."""
    H, E = 1024, 4
    s = make(2, E, H, 128)
    s["x"].fill_(1.0)
    s["weight"].fill_(1.0)
    c = 2.0 ** 14
    below = 1 - 2.0 ** -8                        # the largest bf16 below a power of two, relative to it
    row = torch.empty(H // 16, 16, device="cuda")
    row[0::2, 0], row[0::2, 1:] = c, c * below * 2.0 ** -24          # half a unit behind c, not quite
    row[1::2, 0], row[1::2, 1:] = -c, c * below * 2.0 ** -25         # the same before -c
    s["router"][0], s["router"][1] = row.flatten(), row.flip(1).flatten()
    s["router"][2], s["router"][3] = -row.flatten(), row.roll(5, 1).flatten()
    router = s["router"].double()
    z = router.sum(1)
    out, h, ids, w = call(s, E, residual=False, eps=0.0, score="sigmoid", renormalize=False)
    got = torch.zeros((2, E), dtype=torch.float64, device="cuda").scatter_(1, ids.long(), w.double())
    bound = (7 * 2.0 ** -24 * router.abs().sum(1) + 5 * 2.0 ** -24 * z.abs()) / 4 + 2.0 ** -21
    assert bool(((got - torch.sigmoid(z)).abs() <= bound).all()), (got, torch.sigmoid(z), bound)
