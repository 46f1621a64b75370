"""The sum of the layer of few tokens against 64 bits in every row: products stay in fp32 up to the weighted sum, which is
rounded once, and a code of y that fp32 leaves open costs a step of that code alone."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from test_gpu_moe_few import call, make  # noqa: E402

UNIT = 2.0 ** -23


def open_codes(y, err):
    """How far E4M3 codes of y may be off whose fp32 value is within `err` of y: a step next to a midpoint, two where
    the block may take the other scale."""
    q, e = moe_ref.mxfp8(y)
    s = torch.exp2(e.double()).repeat_interleave(32, 1)
    v, ev = (y / s).abs(), err / s
    step = moe_ref.e4m3_step(v)
    flip = ((v / step - torch.floor(v / step) - 0.5).abs() * step <= ev)
    top = y.abs().reshape(y.shape[0], -1, 32).amax(-1)
    worst = err.reshape(y.shape[0], -1, 32).amax(-1)
    s2 = torch.exp2(e.double())
    either = (torch.minimum((top - 448 * s2).abs(), (top - 224 * s2).abs()) <= worst).repeat_interleave(32, 1)
    return q, torch.where(flip | either, 2 * step * s, torch.zeros_like(s))


def layer_sum(x, ex, ids, w, w13, w2, exact=False):
    """(out, bound) in float64: x [T, H] with errors ex; fp32 sums on the tensor cores (exact: those of product 1 lose
    nothing), one rounding to bf16 at the end."""
    T, H = x.shape
    I = w13.shape[1] // 2
    out, bound, sizes = (torch.zeros((T, H), dtype=torch.float64, device=x.device) for _ in range(3))
    # an accumulator of each of six digits takes an addition for 64 elements, digits' sizes are up to 2.2 times the
    # value's, and the six are added: each addition off by a unit at most, whichever way it rounds
    n1, n2 = 0 if exact else 2.2 * (H // 64 + 6), 2.2 * (I // 64 + 6)
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0:
                continue
            a, aa = w13[e] @ x[t], w13[e].abs() @ x[t].abs()
            ea = n1 * UNIT * aa + w13[e].abs() @ ex[t]
            g, u, eg, eu = a[:I], a[I:], ea[:I], ea[I:]
            silu = g / (1 + torch.exp(-g))
            act = silu * u
            # |silu'| <= 1.1; exponential, quotient and product
            err = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (6 + 1.2 * g.abs()) * UNIT * act.abs()
            q, eq = (m[0] for m in open_codes(act[None], err[None]))
            y = w2[e] @ q
            ey = w2[e].abs() @ eq + n2 * UNIT * (w2[e].abs() @ (q.abs() + eq))
            wt = float(w[t, j])
            out[t] += wt * y
            bound[t] += abs(wt) * ey
            sizes[t] += abs(wt) * (y.abs() + ey)
    bound += ids.shape[1] * UNIT * sizes
    return out, bound + torch.finfo(torch.bfloat16).eps / 2 * (out.abs() + bound)


SIZES = pytest.mark.parametrize("T,E,k,H,I", [
    (1, 4, 2, 128, 128), (1, 32, 8, 2048, 768), (2, 4, 4, 384, 256), (2, 64, 6, 7168, 256), (5, 40, 6, 640, 384),
    (16, 2, 2, 512, 256), (16, 128, 8, 256, 128), (9, 3, 2, 1152, 2048), (7, 256, 32, 256, 128),
])


def worst(out, ref, bound):
    assert mx.get_device_error() == 0
    return float(((out.double() - ref).abs() / bound).max())


@SIZES
@pytest.mark.parametrize("residual", [True, False])
def test_every_row_against_64_bits(T, E, k, H, I, residual):
    s = make(T, E, H, I, seed=5)
    out, h, ids, w = call(s, k, residual, scale=1.5)
    h2, y = moe_ref.add_rmsnorm(s["x"], s["res"] if residual else None, s["weight"], 1e-6)
    assert torch.equal(h, h2)
    # y: r (three roundings and 2^-40) and a product of its own
    ref, bound = layer_sum(*open_codes(y, 4 * 2.0 ** -24 * y.abs()), ids, w, *s["v"])
    assert worst(out, ref, bound) <= 1.0


@SIZES
def test_every_row_where_the_first_product_is_exact(T, E, k, H, I):
    """Rows of ones and minus ones: y is the row itself, and a sum of products a whole number of 2^-10, below 2^12: fp32 has
    it exactly in any order. Then few codes of the activations are open, and the bound is next to the one rounding."""
    s = make(T, E, H, I, seed=6)
    s["x"] = torch.where(s["x"].float() < 0, -1.0, 1.0).bfloat16()
    s["weight"].fill_(1.0)
    out, _, ids, w = call(s, k, residual=False, eps=0.0)
    y = s["x"].double()
    v13, v2 = s["v"]
    assert float(v13.abs().sum(-1).max()) < 2.0 ** 12 and bool((v13 * 1024 == torch.round(v13 * 1024)).all())
    ref, bound = layer_sum(y, torch.zeros_like(y), ids, w, v13, v2, exact=True)
    assert worst(out, ref, bound) <= 1.0
    tight = bound <= 2.0 ** -8 * ref.abs() + 2.0 ** -9 * ref.abs().amax(1, keepdim=True)
    assert float(tight.double().mean()) >= 0.5
