"""Norm and rotation of queries and keys against their definition in 64 bits: head sizes, rotated parts, both layouts,
strides of a joint projection, positions far out and out of range, rows whose squares leave fp32."""
import pytest
import torch

import layer_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def rope_table(P, rot, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))
    angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()


def make(T, Hq, Hk, D, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + T + D)
    qkv = torch.randn((T, (Hq + 2 * Hk) * D), device="cuda", generator=gen).to(dtype)
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    w = [(1 + 0.3 * torch.randn(D, device="cuda", generator=gen)).to(dtype) for _ in range(2)]
    return q, k, w, gen


def check(got, want):
    z, bound = want
    nan = torch.isnan(z)
    assert torch.equal(torch.isnan(got), nan)
    worst = float(((got.double() - z).abs() / bound)[~nan].max()) if bool((~nan).any()) else 0.0
    assert worst <= 1.0, worst


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [
    (1, 1, 1, 8, 0), (1, 4, 1, 64, 64), (7, 3, 2, 64, 32), (16, 32, 8, 128, 128), (5, 5, 3, 96, 48), (33, 24, 1, 192, 64),
    (19, 7, 7, 256, 256), (2, 2, 1, 40, 16), (2000, 13, 5, 128, 128), (1111, 64, 8, 64, 64), (600, 9, 2, 256, 32),
])
def test_against_the_definition(T, Hq, Hk, D, rot, interleaved, dtype):
    q, k, (wq, wk), gen = make(T, Hq, Hk, D, dtype)
    table = rope_table(4096, rot) if rot else None
    pos = torch.randint(0, 4096, (T,), device="cuda", generator=gen).to(torch.int32 if T % 2 else torch.int64)
    for a, b in ((wq, wk), (None, None), (wq, None)):
        qo, ko = mx.qk_norm_rope(q, k, table, pos, a, b, 1e-6, interleaved)
        check(qo, layer_ref.head_norm_rope(q, a, table, pos, 1e-6, interleaved))
        check(ko, layer_ref.head_norm_rope(k, b, table, pos, 1e-6, interleaved))
    # in place, through the strides of the joint projection: the same bits, and values untouched
    joint = q._base if q._base is not None else q
    values = joint[:, (Hq + Hk) * D:].clone()
    qo, ko = mx.qk_norm_rope(q, k, table, pos, wq, wk, 1e-6, interleaved)
    mx.qk_norm_rope(q, k, table, pos, wq, wk, 1e-6, interleaved, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(joint[:, (Hq + Hk) * D:], values)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_at_and_beyond_the_ends_of_the_table(interleaved):
    q, k, (wq, wk), _ = make(6, 4, 2, 64, torch.bfloat16)
    table = rope_table(100, 32)
    pos = torch.tensor([0, 99, 100, -1, 2 ** 40, -2 ** 63], device="cuda")
    qo, ko = mx.qk_norm_rope(q, k, table, pos, wq, wk, 1e-6, interleaved)
    check(qo, layer_ref.head_norm_rope(q, wq, table, pos, 1e-6, interleaved))
    check(ko, layer_ref.head_norm_rope(k, wk, table, pos, 1e-6, interleaved))
    assert bool(torch.isnan(qo[2:]).all()) and not bool(torch.isnan(qo[:2]).any())


def test_a_long_table_and_transposed_heads():
    """A table of more than 2^31 bytes, and tensors that lie head by head."""
    P, rot, T, H, D = (1 << 22) + 77, 128, 37, 6, 128
    table = torch.zeros((P, rot), device="cuda")
    table[P - T:] = rope_table(T, rot)
    x = torch.randn((H, T, D), device="cuda").bfloat16()
    pos = torch.arange(P - T, P, device="cuda")
    out = torch.empty_like(x)
    q = x.transpose(0, 1)
    mx.qk_norm_rope(q, q[:, :0], table, pos, None, None, q_out=out.transpose(0, 1))
    check(out.transpose(0, 1), layer_ref.head_norm_rope(q, None, table, pos, 0.0, False))


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-6])
def test_rows_whose_squares_leave_fp32(eps):
    """Heads of 1e30, 1e-30, the largest and smallest values, zeros, one value among zeros: normalized all the same."""
    D = 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((9, 1, D), device="cuda", generator=gen)
    scale = torch.tensor([1.0, 1e30, 1e-30, 2.0 ** 125, 2.0 ** -130, 0.0, 1e18, 1e-13, 1.0], device="cuda")
    x = (x * scale[:, None, None]).bfloat16()
    x[8] = 0
    x[8, 0, 5] = 2.0 ** -60
    w = torch.ones(D, device="cuda").bfloat16()
    table, pos = rope_table(64, D), torch.arange(9, device="cuda")
    qo, _ = mx.qk_norm_rope(x, x[:, :0], table, pos, w, None, eps)
    z, bound = layer_ref.head_norm_rope(x, w, table, pos, eps, False)
    check(qo, (z, bound))


def test_infinities_and_nan_stay_in_their_heads():
    q, k, (wq, wk), _ = make(3, 4, 2, 64, torch.bfloat16)
    table, pos = rope_table(10, 64), torch.arange(3, device="cuda")
    want, wantk = mx.qk_norm_rope(q, k, table, pos, wq, wk)
    q2 = q.clone()
    q2[1, 2, 3] = float("nan")
    q2[2, 0, 4] = float("inf")
    got, gotk = mx.qk_norm_rope(q2, k, table, pos, wq, wk)
    assert torch.equal(gotk, wantk)
    assert bool(torch.isnan(got[1, 2]).all())
    at = [4, 36]
    assert bool(torch.isnan(got[2, 0, at]).all())
    rest = torch.ones(64, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert not got[2, 0, rest].any()
    got[1, 2], got[2, 0] = want[1, 2], want[2, 0]
    assert torch.equal(got, want)


def test_streams_and_graphs():
    q, k, (wq, wk), _ = make(50, 8, 2, 128, torch.float16)
    table, pos = rope_table(500, 128), torch.arange(50, device="cuda")
    want, wantk = mx.qk_norm_rope(q, k, table, pos, wq, wk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = mx.qk_norm_rope(q, k, table, pos, wq, wk, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, want) and torch.equal(b, wantk)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = mx.qk_norm_rope(q, k, table, pos, wq, wk)
    pos.add_(400)
    g.replay()
    want, wantk = mx.qk_norm_rope(q, k, table, pos, wq, wk)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, wantk)


def test_zero_tokens_and_refusals_of_the_binding():
    q, k, (wq, wk), _ = make(4, 2, 1, 64, torch.bfloat16)
    table, pos = rope_table(10, 64), torch.arange(4, device="cuda")
    qo, ko = mx.qk_norm_rope(q[:0], k[:0], table, pos[:0], wq, wk)
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)
    for args in ((q.float(), k, table, pos), (q, k.half(), table, pos), (q, k[:3], table, pos), (q, k, table, None),
                 (q, k, table.double(), pos), (q, k, table, pos.float()), (q, k, table, pos[:3]),
                 (q, k, table, pos, wq[:32]), (q, k, table, pos, wq.float()), (q, k[..., :32], table, pos),
                 (q.transpose(1, 2), k, table, pos)):
        with pytest.raises(ValueError):
            mx.qk_norm_rope(*args)
    with pytest.raises(ValueError):
        mx.qk_norm_rope(q, k, table, pos, q_out=q[:, :1])
    with pytest.raises(mx.Mxfp4Error):
        mx.qk_norm_rope(q, k, table[:, :24].contiguous(), pos)
