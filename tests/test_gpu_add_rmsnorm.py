"""Residual sum + RMSNorm + MXFP8 quantization against its definition in 64 bits.

Tolerances. The fp32 sum of squares has at most 64 additions in a row in a thread
and 10 across the block, each off by 2^-24 of the sum; the root halves that; the
division, rsqrt (2 units) and two products add 6: less than 64 * 2^-24 = 2^-18 of y.
The stored y adds half a step of its type, the E4M3 codes half a step of theirs
(2^-4 of the value, 2^-10 of the scale among subnormals). The scale is that of a
maximum within 2^-18 of the exact one."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")

D = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def check(x, res, w, eps, Aq, sf, H, Y, finite=None):
    M, K = x.shape
    h, y = moe_ref.add_rmsnorm(x, res, w, eps)
    rows = torch.ones(M, dtype=torch.bool, device=x.device) if finite is None else finite
    if H is not None:
        assert torch.equal(H[rows], h[rows])
    if Y is not None:
        err = (Y.double() - y).abs()[rows]
        assert bool((err <= (HALF[x.dtype] * (1 + D) + D) * y.abs()[rows] + TINY[x.dtype]).all())
    C = K // 32
    bytes_ = sf[moe_ref.blocked_index(M, C, x.device)]
    s = torch.exp2(bytes_.double() - 127)
    top = y.reshape(M, C, 32).abs().amax(-1)
    assert bool((top * (1 - D) <= 448 * s)[rows].all())
    assert bool(((top * (1 + D) > 224 * s) | (bytes_ == 0))[rows].all())
    sv = s.repeat_interleave(32, 1)
    got = moe_ref.e4m3_values(Aq.contiguous()) * sv
    err = (got - y).abs()[rows]
    assert bool((err <= (2.0 ** -4 * y.abs() * (1 + D) + D * y.abs() + 2.0 ** -10 * sv)[rows]).all())
    pad = torch.ones_like(sf, dtype=torch.bool)
    pad[moe_ref.blocked_index(M, C, x.device).reshape(-1)] = False
    assert bool((sf[pad] == 0x7F).all())


def inputs(M, K, dtype, seed=0, res=True, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    amp = torch.where(torch.rand(K, device="cuda", generator=gen) < 0.02, 30.0, 1.0)
    def rows(v):
        b = torch.zeros((M, K + pad), dtype=dtype, device="cuda")
        b[:, :K] = v.to(dtype)
        return b[:, :K]
    return rows(r(M, K) * amp), rows(r(M, K) * amp) if res else None, (1 + 0.3 * r(K)).to(dtype)


@pytest.mark.parametrize("M,K", [(1, 32), (1, 7168), (3, 96), (5, 2112), (127, 160), (128, 256), (129, 1024), (300, 7168),
                                 (2, 8192), (2, 8224), (3, 32768), (2, 33024), (1, 65536)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_norm_matches_its_definition(M, K, dtype):
    x, res, w = inputs(M, K, dtype, seed=M * K)
    Aq, sf, H, Y = mx.mxfp8_add_rmsnorm_quantize(x, w, 1e-6, residual=res, want_y=True)
    check(x, res, w, 1e-6, Aq, sf, H, Y)
    Aq2, sf2, H2, Y2 = mx.mxfp8_add_rmsnorm_quantize(H, w, 1e-6)
    assert H2 is None and Y2 is None
    assert torch.equal(Aq, Aq2) and torch.equal(sf, sf2)      # the norm is of the rounded sum


@pytest.mark.parametrize("M,K,pad", [(33, 288, 8), (64, 7168, 64), (2, 33024, 16)])
def test_norm_strides_and_in_place(M, K, pad):
    x, res, w = inputs(M, K, torch.bfloat16, seed=7, pad=pad)
    want = mx.mxfp8_add_rmsnorm_quantize(x.contiguous(), w, 1e-5, residual=res.contiguous(), want_y=True)
    Y = torch.full((M, K + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    Aq = torch.full((M, K + pad), 77, dtype=torch.uint8, device="cuda")
    keep = res.clone()
    got = mx.mxfp8_add_rmsnorm_quantize(x, w, 1e-5, residual=res, H=res, Y=Y[:, :K], Aq=Aq[:, :K])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert bool((Y[:, K:] == 5.0).all()) and bool((Aq[:, K:] == 77).all())
    xi = x.clone()
    assert torch.equal(mx.mxfp8_add_rmsnorm_quantize(xi, w, 1e-5, residual=keep, H=xi)[2], want[2])
    check(x, keep, w, 1e-5, got[0], got[1], got[2], got[3])


def test_norm_zero_rows_zero_eps_and_extremes():
    x, _, w = inputs(9, 512, torch.bfloat16, seed=3)
    x[0] = 0                                  # r is finite, y = 0
    x[1] = 0
    x[1, 5] = 2.0 ** -120                     # squares underflow in fp32: with eps = 0 the mean is 0
    x[2] *= 2.0 ** 50
    x[3] *= 2.0 ** -40
    Aq, sf, _, Y = mx.mxfp8_add_rmsnorm_quantize(x, w, 0.0, want_y=True)
    rows = torch.ones(9, dtype=torch.bool, device="cuda")
    rows[1] = False
    check(x, None, w, 0.0, Aq, sf, None, Y, rows)
    assert not Aq[:2].any() and not Y[:2].any()
    assert bool((sf[moe_ref.blocked_index(9, 16, "cuda")][:2] == 0).all())
    check(x, None, w, 1e-3, *mx.mxfp8_add_rmsnorm_quantize(x, w, 1e-3, want_y=True)[:2], None, None)


def test_norm_nan_and_inf_stay_in_their_row():
    x, res, w = inputs(4, 256, torch.float16, seed=4)
    x[1, 40] = float("nan")
    x[2, 200] = float("inf")
    Aq, sf, H, Y = mx.mxfp8_add_rmsnorm_quantize(x, w, 1e-6, residual=res, want_y=True)
    good = torch.tensor([True, False, False, True], device="cuda")
    check(x, res, w, 1e-6, Aq, sf, H, Y, good)
    s = sf[moe_ref.blocked_index(4, 8, "cuda")]
    assert bool((s[1] == 0xFF).all())         # NaN spreads over its row
    assert int(s[2, 6]) == 0xFF               # inf * 0 in its own block


def test_norm_other_stream_empty_batch_and_graph():
    x, res, w = inputs(40, 512, torch.bfloat16, seed=5)
    want = mx.mxfp8_add_rmsnorm_quantize(x, w, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mx.mxfp8_add_rmsnorm_quantize(x, w, residual=res)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e = mx.mxfp8_add_rmsnorm_quantize(x[:0], w, residual=res[:0])
    assert e[0].shape == (0, 512) and e[1].numel() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mx.mxfp8_add_rmsnorm_quantize(x, w, residual=res)
    x.mul_(2)
    g.replay()
    fresh = mx.mxfp8_add_rmsnorm_quantize(x, w, residual=res)
    torch.cuda.synchronize()
    assert torch.equal(out[0], fresh[0]) and torch.equal(out[2], fresh[2])


def test_norm_python_refusals():
    x, res, w = inputs(4, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        mx.mxfp8_add_rmsnorm_quantize(x.float(), w)
    with pytest.raises(ValueError):
        mx.mxfp8_add_rmsnorm_quantize(x, w[:32])
    with pytest.raises(ValueError):
        mx.mxfp8_add_rmsnorm_quantize(x, w, residual=res.half())
    with pytest.raises(ValueError):
        mx.mxfp8_add_rmsnorm_quantize(x, w, residual=res[:2])
    with pytest.raises(ValueError):
        mx.mxfp8_add_rmsnorm_quantize(x.t(), w)
    with pytest.raises(mx.Mxfp4Error):
        mx.mxfp8_add_rmsnorm_quantize(x[:1].expand(4, 64), w)     # rows that overlap
