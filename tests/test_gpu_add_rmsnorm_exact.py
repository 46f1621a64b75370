"""The codes and scales of mxfp8_add_rmsnorm_quantize are those of its definition in 64 bits, where fp32 arithmetic
would take the neighbour: no tolerance but for values that lie within 2^-40 of a rounding midpoint, or maxima that close
to the border between two scales."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")

TYPES = [torch.bfloat16, torch.float16]


def definition(x, res, w, eps):
    """(y / scale, exponents, codes as multiples of the scale), float64."""
    h, y = moe_ref.add_rmsnorm(x, res, w, eps)
    q, e = moe_ref.mxfp8(y)
    s = torch.exp2(e.double()).repeat_interleave(32, 1)
    return y / s, e, q / s


def check(x, res, w, eps):
    M, K = x.shape
    Aq, sf, _, _ = mx.mxfp8_add_rmsnorm_quantize(x, w, eps, residual=res)
    v, e, q = definition(x, res, w, eps)
    bytes_ = sf[moe_ref.blocked_index(M, K // 32, x.device)]
    assert torch.equal(bytes_.int(), e.int() + 127)
    got = moe_ref.e4m3_values(Aq)
    wrong = got != q
    step = moe_ref.e4m3_step(v)
    on = ((v.abs() / step - torch.floor(v.abs() / step) - 0.5) * step).abs() <= 2.0 ** -40 * v.abs()
    assert not bool((wrong & ~on).any()), (int((wrong & ~on).sum()), v[wrong][:4], got[wrong][:4], q[wrong][:4])
    return v, e


def near_one(dtype, side):
    """A row of ones, but for one element, and an eps, for which r is 1 to fp32 and lies on `side` of it."""
    if side == 0:
        return torch.ones(7168, device="cuda", dtype=dtype), 0.0
    if side < 0:                                        # 1 - 2^-26
        return torch.ones(7168, device="cuda", dtype=dtype), 2.0 ** -25
    x = torch.ones(65536 if dtype == torch.bfloat16 else 8192, device="cuda", dtype=dtype)
    x[70] -= 2.0 ** (-8 if dtype == torch.bfloat16 else -11)          # 1 + 2^-24
    return x, 0.0


def r_of(x, eps):
    return float(1 / torch.sqrt(x.double().square().mean() + eps))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("side", [-1, 0, 1])
@pytest.mark.parametrize("subnormal", [False, True])
def test_values_on_either_side_of_a_midpoint(dtype, side, subnormal):
    """y = r w with w a midpoint of E4M3 and r = 1 to fp32."""
    x, eps = near_one(dtype, side)
    K = x.numel()
    r = r_of(x, eps)
    assert (r > 1) - (r < 1) == side and torch.tensor(r, dtype=torch.float64).float() == 1.0
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = torch.randint(0, 8, (K,), device="cuda", generator=gen)
    if subnormal:
        w = (n + 0.5) * 2.0 ** -9
    else:
        w = (1 + (n + 0.5) / 8) * torch.exp2(torch.randint(-6, 8, (K,), device="cuda", generator=gen).float())
    w = w * (1 - 2 * torch.randint(0, 2, (K,), device="cuda", generator=gen))
    w[::32] = 256.0                                     # of every block the maximum: its scale is 1
    v, e = check(torch.stack([x, -x, x]), None, w.to(dtype), eps)
    assert not e.any()
    if side == 0:
        assert torch.equal(v[0], w.to(dtype).double())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("side", [-1, 0, 1])
def test_maxima_on_either_side_of_the_border_between_scales(dtype, side):
    x, eps = near_one(dtype, side)
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.rand(x.numel(), device="cuda", generator=gen) * 100
    w[5::32] = 448.0
    _, e = check(torch.stack([x, x]), None, w.to(dtype), eps)
    keep = torch.ones_like(e, dtype=torch.bool)
    keep[:, 70 // 32] = False
    assert bool((e == (1 if side > 0 else 0))[keep].all())


def rows(M, K, dtype, seed, amp, res=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x = (r(M, K) * amp(gen, M, K)).to(dtype)
    return x, (r(M, K) * amp(gen, M, K)).to(dtype) if res else None, (1 + 0.3 * r(K)).to(dtype)


def plain(gen, M, K):
    return 1.0


def one_channel(gen, M, K):
    a = torch.ones(K, device="cuda")
    a[17 % K] = 1000.0
    return a


def some_channels(gen, M, K):
    return torch.where(torch.rand(K, device="cuda", generator=gen) < 0.01, 20.0, 1.0)


def one_value_a_row(gen, M, K):
    a = torch.ones((M, K), device="cuda")
    a[torch.arange(M, device="cuda"), torch.randint(0, K, (M,), device="cuda", generator=gen)] = 700.0
    return a


def one_value_a_block(gen, M, K):
    a = torch.full((M, K // 32, 32), 2.0 ** -5, device="cuda")
    a[..., 3] = 2.0 ** 10
    return a.reshape(M, K)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("amp", [plain, one_channel, some_channels, one_value_a_row, one_value_a_block])
@pytest.mark.parametrize("M,K", [(4096, 7168), (300000, 32), (3001, 2112), (200, 33024)])
def test_codes_and_scales_are_those_of_64_bits(M, K, amp, dtype):
    """Some 6 to 29 million codes a case. What fp32 gets wrong is about one in a million, more where one channel has most
    of a row's squares, or where a block has an outlier and its other values are subnormal codes."""
    x, res, w = rows(M, K, dtype, M + K, amp, res=amp is some_channels)
    check(x, res, w, 1e-6)


@pytest.mark.parametrize("M,K", [(5, 256), (7, 7168), (400, 2112), (400, 7168), (6, 33024)])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_whose_squares_leave_fp32(M, K, res, in_place):
    """bf16 holds values whose squares, or the sum of them, are beyond fp32: rows of 2^45 to 2^120, among ordinary ones,
    and ordinary rows with one such value."""
    x, r, w = rows(M, K, torch.bfloat16, M * K, some_channels, res)
    up = torch.exp2(torch.tensor([0.0, 45, 50, 62, 64, 100, 118], device="cuda"))[torch.arange(M, device="cuda") % 7]
    x = (x.float() * up[:, None]).to(torch.bfloat16)
    x[::5, 11] = 2.0 ** 127
    if res:
        r = (r.float() * up[:, None]).to(torch.bfloat16)
    h, y = moe_ref.add_rmsnorm(x, r, w, 1e-6)
    assert bool(torch.isfinite(h).all()) and bool((h.float().square().sum(-1) == torch.inf).any())
    check(x, r, w, 1e-6)
    given = x.clone()
    Aq, sf, H, Y = mx.mxfp8_add_rmsnorm_quantize(given, w, 1e-6, residual=r, H=given if in_place else None, want_y=True)
    plain = mx.mxfp8_add_rmsnorm_quantize(x, w, 1e-6, residual=r)
    assert torch.equal(Aq, plain[0]) and torch.equal(sf, plain[1])
    if H is not None:
        assert torch.equal(H, h)
    # y: three fp32 roundings, then half a step of bf16 (2^-134: of its smallest values)
    assert bool(((Y.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -21) * y.abs() + 2.0 ** -134).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eps", [1e25, 1e34, 3e38])
def test_an_eps_beyond_the_squares(dtype, eps):
    x, _, w = rows(9, 7168, dtype, 3, plain)
    eps = float(torch.tensor(eps))
    check(x, None, w, eps)


@pytest.mark.parametrize("M,K", [(6, 256), (9, 7168), (400, 2112), (400, 7168), (6, 33024)])
@pytest.mark.parametrize("eps", [0.0, 1e-38])
def test_rows_whose_squares_nearly_vanish(M, K, eps):
    """Sums of squares far below one, among them subnormal ones and such that lose most of their squares in fp32."""
    x, _, w = rows(M, K, torch.bfloat16, M * K, some_channels)
    down = torch.exp2(torch.tensor([0.0, -45, -55, -60, -66, -70], device="cuda"))[torch.arange(M, device="cuda") % 6]
    x = (x.float() * down[:, None]).to(torch.bfloat16)
    x[::6, 3] = 2.0 ** -70                                     # an ordinary row with such a value
    assert bool((x.float().square().sum(-1) > 0).all())
    check(x, None, w, eps)
    H = torch.zeros_like(x)
    q, sf, _, Y = mx.mxfp8_add_rmsnorm_quantize(x, w, eps, residual=torch.zeros_like(x), H=H, want_y=True)
    assert torch.equal(H, x)
    plain = mx.mxfp8_add_rmsnorm_quantize(x, w, eps)
    assert torch.equal(q, plain[0]) and torch.equal(sf, plain[1])
    _, y = moe_ref.add_rmsnorm(x, None, w, eps)
    assert bool(((Y.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -21) * y.abs() + 2.0 ** -134).all())
