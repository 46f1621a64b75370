"""Routing against its definition in 64 bits: the ids are equal; the weights may be
off by what fp32 costs: 28 units of 2^-24 for a score (see the kernel's error
bound), up to 30 more for a logit that far below the maximum, k + 2 for the
renormalisation: less than 2^-17 of the value."""
import math

import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def check(z, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=2, renormalize=True, scale=1.0):
    ids, w = mx.moe_route(z, k, score, bias, groups, topk_groups, group_top, renormalize, scale)
    ri, rw = moe_ref.route(z, k, score, bias, groups, topk_groups, group_top, renormalize, scale)
    bad = (ids.cpu() != ri).any(-1).nonzero().flatten()
    assert len(bad) == 0, (bad[:4], ids[bad[:1]], ri[bad[:1]])
    g, nan = w.cpu().double(), torch.isnan(rw)
    assert torch.equal(torch.isnan(g), nan)
    assert bool(((g - rw).abs() <= 2.0 ** -17 * rw.abs() + 1e-37)[~nan].all())
    return ids, w


def logits(T, E, dtype=torch.float32, seed=0, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((T, E), device="cuda", generator=gen) * spread).to(dtype)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (5, 31, 3), (4, 32, 32), (7, 33, 2), (64, 60, 5), (33, 128, 8),
                                   (50, 129, 6), (40, 256, 8), (9, 511, 10), (6, 512, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_route_matches_its_definition(T, E, k, score, dtype):
    z = logits(T, E, dtype, seed=T * E + k)
    bias = torch.randn(E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(E)) * 0.1
    check(z, k, score)
    check(z, k, score, bias, renormalize=False, scale=2.5)


@pytest.mark.parametrize("E,groups,topk_groups,k", [(256, 8, 4, 8), (64, 8, 3, 6), (60, 4, 2, 5), (96, 32, 5, 4),
                                                    (512, 512, 40, 32), (512, 64, 64, 9), (48, 3, 1, 16), (8, 8, 1, 1)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(E, groups, topk_groups, k, group_top, score):
    z = logits(24, E, seed=E + groups)
    bias = torch.randn(E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(E)) * 0.05
    check(z, k, score, bias, groups, topk_groups, group_top, True, 2.5)
    check(z, k, score, None, groups, topk_groups, group_top, False)


def test_route_equal_scores_take_the_lower_index():
    z = torch.zeros((3, 40), device="cuda")
    z[1, 20:] = 1.0
    z[2] = logits(1, 40)[0].round()
    for score in ("softmax", "sigmoid"):
        check(z, 7, score)
        check(z, 7, score, torch.zeros(40, device="cuda"))
        check(z, 7, score, None, 8, 3, 2)
    assert mx.moe_route(z, 3)[0][0].tolist() == [0, 1, 2]


@pytest.mark.parametrize("E", [24, 64, 128, 256, 512])
def test_route_many_equal_keys_of_neighbours(E):
    """Three values only, so runs of experts tie within and across the lanes of a warp."""
    z = logits(12, E, seed=E).round().clamp(-1, 1)
    z[0] = 1.0
    z[1, : E // 2] = -math.inf
    for score in ("softmax", "sigmoid"):
        for k in (1, 9, 20):
            check(z, k, score)
            check(z, k, score, torch.ones(E, device="cuda"))
            check(z, min(k, 2 * (E // 8)), score, None, 8, 2, 2)


def test_route_scores_below_the_normal_range():
    """Sigmoids of logits below -87 are subnormal or zero in fp32."""
    z = -86.5 - logits(20, 64, seed=3, spread=1.0).abs() * 2
    z[10:] -= 30
    for bias in (None, torch.zeros(64, device="cuda")):
        for args in ((), (8, 3, 2), (16, 2, 1)):
            ids, _ = mx.moe_route(z, 6, "sigmoid", bias, *args, renormalize=False)
            ri, _ = moe_ref.route(z, 6, "sigmoid", bias, *((args or (1, 1, 2))), False, 1.0)
            assert torch.equal(ids.cpu(), ri)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scores_closer_than_fp32(score):
    """Sums s + bias that fp32 cannot order: neighbours a few 2^-28 apart."""
    E = 96
    z = logits(64, E, seed=9, spread=0.5)
    s = torch.softmax(z.double(), -1) if score == "softmax" else torch.sigmoid(z.double())
    bias = (0.5 - s[0] + torch.arange(E, device="cuda").double() * 2.0 ** -28).float()
    check(z, 8, score, bias)
    check(z, 8, score, bias, 12, 5, 2)
    check(z[:1].expand(64, E).contiguous(), 8, score, bias, 12, 5, 1)


def test_route_saturated_scores_rank_by_logit():
    z = torch.tensor([[50.0, 60.0, 55.0, 1e30, -1e30, 40.0]], device="cuda")
    assert check(z, 4, "sigmoid", renormalize=False)[0].tolist() == [[3, 1, 2, 0]]
    check(z, 6, "softmax", renormalize=False)


def test_route_masked_experts():
    z = logits(6, 40, seed=2)
    z[:, ::3] = -math.inf
    z[1] = -math.inf                       # nothing left
    z[2, 1:] = -math.inf                   # one left
    z[2, 0] = 0.5
    bias = torch.rand(40, device="cuda") * 5
    for score in ("softmax", "sigmoid"):
        for ren in (True, False):
            ids, w = check(z, 6, score, None, renormalize=ren)
            assert ids[1].tolist() == [-1] * 6 and not w[1].any()
            assert ids[2].tolist() == [0] + [-1] * 5
            ids, _ = check(z, 6, score, bias, renormalize=ren)
            assert not bool(((ids % 3 == 0) & (ids > 0)).any())
            check(z, 6, score, bias, 5, 2, 2, ren)


def test_route_nan_and_infinity():
    z = logits(5, 33, seed=3)
    z[0, 7] = math.nan
    z[2, 9] = math.inf
    z[3, :] = math.nan
    z[4, :20] = -math.inf
    z[4, 25] = math.nan
    bias = torch.zeros(33, device="cuda")
    for score in ("softmax", "sigmoid"):
        check(z, 4, score)
        check(z, 4, score, bias)
        check(z, 4, score, bias, 3, 2, 2)


def test_route_strides_streams_graph_and_large_batch():
    z = logits(2000, 128, torch.bfloat16, seed=6)
    wide = torch.zeros((2000, 131), dtype=torch.bfloat16, device="cuda")
    wide[:, :128] = z
    want = mx.moe_route(z, 8)
    got = mx.moe_route(wide[:, :128], 8)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert mx.moe_route(z[:0], 8)[0].shape == (0, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mx.moe_route(z, 8)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mx.moe_route(z, 8)
    z.neg_()
    g.replay()
    fresh = mx.moe_route(z, 8)
    torch.cuda.synchronize()
    assert torch.equal(out[0], fresh[0]) and torch.equal(out[1], fresh[1])
    big = logits(40000, 64, seed=8)
    ids, w = mx.moe_route(big, 4, "sigmoid")
    pick = torch.topk(big, 4, -1)
    assert torch.equal(torch.gather(big, 1, ids.long()), pick[0])
    assert bool(((w.sum(-1) - 1).abs() < 2.0 ** -20).all())


def test_route_python_refusals():
    z = logits(4, 16)
    with pytest.raises(ValueError):
        mx.moe_route(z.double(), 2)
    with pytest.raises(ValueError):
        mx.moe_route(z, 2, score="tanh")
    with pytest.raises(ValueError):
        mx.moe_route(z, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        mx.moe_route(z, 2, ids=torch.zeros((4, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(mx.Mxfp4Error):
        mx.moe_route(z, 17)
    with pytest.raises(mx.Mxfp4Error):
        mx.moe_route(z[:1].expand(4, 16), 2)          # rows that overlap
