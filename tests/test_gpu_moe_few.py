"""The mixture-of-experts layer of a few tokens: its choice against the definition in 64 bits, its sum against the
products of the experts it chose, sizes that end inside tiles, every routing option, in place, streams, graphs, and the way
out of a wait that runs out."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")

UNIT = 2.0 ** -23


def make(T, E, H, I, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + T + E)
    rn = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    w13, s13, v13 = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, 2 * I, H, "cuda") for _ in range(E))))
    w2, s2, v2 = (torch.stack(m) for m in zip(*(moe_ref.random_mxfp4(gen, H, I, "cuda") for _ in range(E))))
    return dict(x=rn(T, H).bfloat16(), res=(2 * rn(T, H)).bfloat16(), weight=(1 + 0.2 * rn(H)).bfloat16(),
                router=(1.5 * rn(E, H) * H ** -0.5).bfloat16(), bias=0.05 * rn(E), w=(w13, s13, w2, s2), v=(v13, v2))


def call(s, k, residual=True, **kw):
    return mx.mxfp4_moe_layer(s["x"], s["weight"], s["router"], *s["w"], k, residual=s["res"] if residual else None, **kw)


def check(s, got, k, residual=True, eps=1e-6, bias=None, score="softmax", groups=1, topk_groups=1, group_top=2,
          renormalize=True, scale=1.0):
    out, h, ids, w = got
    h2, y = moe_ref.add_rmsnorm(s["x"], s["res"] if residual else None, s["weight"], eps)
    assert torch.equal(h, h2)
    ri, rw = moe_ref.route(y @ s["router"].double().T, k, score, bias, groups, topk_groups, group_top, renormalize, scale)
    assert torch.equal(ids.cpu(), ri)
    # scores in fp32: the logits' error and a few units of the exponential, sum and quotient
    assert float((w.double().cpu() - rw).abs().max()) <= 2.0 ** -18 * scale
    # MXFP8 of y in fp32: the other neighbour only where y's error (4 units) reaches the midpoint
    q, e = moe_ref.mxfp8(y)
    sc = torch.exp2(e.double()).repeat_interleave(32, 1)
    v = (y / sc).abs()
    step = moe_ref.e4m3_step(v)
    near = ((v / step - torch.floor(v / step) - 0.5).abs() * step <= 4 * UNIT * v)
    top = y.abs().reshape(y.shape[0], -1, 32).amax(-1)
    s2 = torch.exp2(e.double())
    near |= (torch.minimum((top - 448 * s2).abs(), (top - 224 * s2).abs()) <= 4 * UNIT * top).repeat_interleave(32, 1)
    v13, v2 = s["v"]
    ref, bound = moe_ref.experts(q, ids, w, v13, v2)
    rows = ~near.any(1)
    assert int(rows.sum()) >= 1 or y.shape[0] < 3
    worst = float(((out.double() - ref).abs() / bound)[rows].max()) if bool(rows.any()) else 0.0
    assert worst <= 1.0, worst
    assert mx.get_device_error() == 0


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (2, 4, 4, 384, 256), (5, 40, 6, 640, 384), (8, 6, 3, 256, 640),
    (9, 3, 2, 1152, 128), (16, 2, 2, 512, 256), (16, 128, 8, 256, 128), (7, 512, 32, 128, 128), (16, 511, 7, 128, 128),
    (3, 33, 5, 2048, 768),
])
@pytest.mark.parametrize("residual", [True, False])
def test_against_the_definition(T, E, k, H, I, residual):
    s = make(T, E, H, I)
    check(s, call(s, k, residual), k, residual)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("how", [
    dict(bias=True), dict(groups=4, topk_groups=2), dict(groups=8, topk_groups=3, group_top=1, bias=True),
    dict(renormalize=False, scale=2.5), dict(groups=24, topk_groups=6), dict(groups=2, topk_groups=1, bias=True, scale=0.5),
])
def test_routing_options(score, how):
    s = make(11, 24, 256, 128)
    how = dict(how, score=score)
    if how.get("bias"):
        how["bias"] = s["bias"]
    check(s, call(s, 3, **how), 3, **how)


@pytest.mark.parametrize("T", [1, 6, 16])
def test_popular_experts_and_repeated_calls(T):
    """All tokens on the same experts, and the same bits every time, whichever block takes which unit."""
    s = make(T, 16, 512, 256)
    s["bias"] = torch.zeros(16, device="cuda")
    s["bias"][3], s["bias"][11] = 8.0, 9.0
    got = call(s, 2, bias=s["bias"])
    assert got[2].tolist() == [[11, 3]] * T
    check(s, got, 2, bias=s["bias"])
    ws = mx.moe_layer_workspace(16, 2, 16, 512, 256).fill_(0xFF)
    for _ in range(20):
        again = call(s, 2, bias=s["bias"], workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_rows_do_not_depend_on_one_another():
    s = make(9, 12, 256, 256)
    want = call(s, 3)
    for t in (0, 8):
        one = dict(s, x=s["x"][t:t + 1], res=s["res"][t:t + 1])
        got = call(one, 3)
        assert all(torch.equal(a, b[t:t + 1]) for a, b in zip(got, want))
    bad = dict(s, x=s["x"].clone())
    bad["x"][4, 17] = float("nan")
    bad["x"][5, 0] = float("inf")
    got = call(bad, 3)
    keep = [t for t in range(9) if t not in (4, 5)]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, want))
    assert not bool(torch.isfinite(got[0][4]).any()) and not bool(torch.isfinite(got[0][5]).any())
    assert int(got[2].min()) >= 0 and int(got[2].max()) < 12
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0


def test_bias_of_the_lowest_value():
    """Experts masked by fp32's lowest value go before those masked by -inf, in groups too, whose sums pass fp32."""
    s = make(4, 8, 256, 128)
    low, none = torch.finfo(torch.float32).min, float("-inf")
    _, y = moe_ref.add_rmsnorm(s["x"], s["res"], s["weight"], 1e-6)
    z = y @ s["router"].double().T
    for bias, k, groups, topk in (([none, none, low, low, none, none, none, none], 2, 4, 1),
                                  ([none, none, low, low, 0.0, none, none, none], 3, 4, 2),
                                  ([none, none, none, none, none, none, none, low], 3, 1, 1)):
        b = torch.tensor(bias, device="cuda")
        for score in ("softmax", "sigmoid"):
            _, _, ids, w = call(s, k, bias=b, groups=groups, topk_groups=topk, score=score)
            ri, rw = moe_ref.route(z, k, score, b, groups, topk, 2, True, 1.0)
            # lowest + score: equal in fp32, so the lower index comes first
            assert torch.equal(ids.cpu().sort(-1)[0], ri.sort(-1)[0])
            assert float((w.double().cpu().sum(-1) - rw.sum(-1)).abs().max()) <= 2.0 ** -18
    assert mx.get_device_error() == 0


def test_zero_rows():
    s = make(3, 4, 256, 128)
    s["x"][1], s["res"][1] = 0, 0
    for eps in (1e-6, 0.0):
        out, h, ids, w = call(s, 2, eps=eps)
        assert not out[1].any() and ids[1].tolist() == [0, 1] and w[1].tolist() == [0.5, 0.5]
        check(s, (out, h, ids, w), 2, eps=eps)


@pytest.mark.parametrize("power", [47, -48])
def test_large_and_small_magnitudes(power):
    s = make(5, 6, 1024, 128)
    s["x"], s["res"] = s["x"] * 2.0 ** power, s["res"] * 2.0 ** power
    s["x"][2], s["res"][2] = 2.0 ** 49 if power > 0 else 2.0 ** -60, 0
    check(s, call(s, 3, eps=0.0), 3, eps=0.0)


def test_zero_row_with_an_eps_below_the_normal_numbers():
    s = make(3, 4, 256, 128)
    s["x"][1], s["res"][1] = 0, 0
    out, _, ids, w = call(s, 2, eps=1e-44)
    assert not out[1].any() and ids[1].tolist() == [0, 1] and w[1].tolist() == [0.5, 0.5]


def test_in_place_and_strides():
    T, H = 6, 384
    s = make(T, 8, H, 128)
    want = call(s, 2)
    wide = torch.full((T, 3 * H + 16), 5.0, device="cuda").bfloat16()
    x, r, o = wide[:, 8:8 + H], wide[:, 8 + H:8 + 2 * H], wide[:, 16 + 2 * H:]
    for target in (x, r):
        x.copy_(s["x"])
        r.copy_(s["res"])
        got = mx.mxfp4_moe_layer(x, s["weight"], s["router"], *s["w"], 2, residual=r, H=target, out=o)
        assert got[1] is target and all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((wide[:, :8] == 5.0).all()) and bool((wide[:, 8 + 2 * H:16 + 2 * H] == 5.0).all())
    # the result in the place of x
    x.copy_(s["x"])
    r.copy_(s["res"])
    got = mx.mxfp4_moe_layer(x, s["weight"], s["router"], *s["w"], 2, residual=r, out=x)
    assert torch.equal(x, want[0]) and torch.equal(got[1], want[1])


def test_streams_and_graphs():
    s = make(4, 10, 512, 256)
    want = call(s, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(s, 3, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = call(s, 3, workspace=mx.moe_layer_workspace(4, 3, 10, 512, 256))
        graphs.append((g, o))
    s["x"].copy_(s["x"].flip(0))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    fresh = call(s, 3)
    torch.cuda.synchronize()
    for _, o in graphs:
        assert all(torch.equal(a, b) for a, b in zip(o, fresh))
    assert mx.get_device_error() == 0


def test_two_graphs_that_share_a_workspace():
    """Layers that run one after another may share one: what a replay leaves there does not matter to the next."""
    s = [make(3, 10, 512, 256, seed=1), make(16, 24, 256, 384, seed=2)]
    size = max(mx.moe_layer_workspace_bytes(3, 3, 10, 512, 256), mx.moe_layer_workspace_bytes(16, 3, 24, 256, 384))
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    want = [call(x, 3) for x in s]
    graphs = []
    for x in s:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = call(x, 3, workspace=ws)
        graphs.append((g, o))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graphs[i][0].replay()
        assert all(torch.equal(a, b) for a, b in zip(graphs[i][1], want[i]))
    assert mx.get_device_error() == 0


def test_two_streams_at_once():
    """Calls of two streams share the SMs: units wait only for units that some block already has."""
    s = [make(16, 64, 1024, 512, seed=i) for i in range(2)]
    want = [call(x, 4) for x in s]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(call(s[i], 4, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
    assert mx.get_device_error() == 0


def test_waits_that_run_out_end_the_call_and_are_reported():
    s = make(6, 8, 1024, 512)
    want = call(s, 2)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0
    mx.set_wait_limit_ns(1)
    try:
        call(s, 2)
        torch.cuda.synchronize()
    finally:
        mx.set_wait_limit_ns(0)
    assert 64 < mx.get_device_error() < 80
    again = call(s, 2)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0 and all(torch.equal(a, b) for a, b in zip(again, want))


def test_zero_tokens_and_refusals_of_the_binding():
    s = make(2, 4, 256, 128)
    none = dict(s, x=s["x"][:0], res=s["res"][:0])
    out, h, ids, w = call(none, 2)
    assert out.shape == (0, 256) and ids.shape == (0, 2)
    for key, value in (("x", s["x"].half()), ("weight", s["weight"][:128]), ("router", s["router"][:3]),
                       ("router", s["router"].float()), ("res", s["res"][:1])):
        with pytest.raises(ValueError):
            call(dict(s, **{key: value}), 2)
    with pytest.raises(ValueError):
        call(s, 2, score="tanh")
    with pytest.raises(mx.Mxfp4Error):
        call(s, 5)
    with pytest.raises(mx.Mxfp4Error):
        call(dict(s, x=torch.zeros((17, 256), device="cuda").bfloat16()), 2, residual=False)
    with pytest.raises(mx.Mxfp4Error):
        call(s, 2, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("seed", range(4))
def test_experts_whose_tokens_take_several_units(seed):
    """More than four tokens of an expert are several units of work: all blocks agree on which tokens are whose, call after
    call, and a token's result is that of its call alone."""
    s = make(11, 24, 256, 128, seed=seed)
    how = dict(groups=2, topk_groups=1, bias=s["bias"], scale=0.5)
    alone = [call(dict(s, x=s["x"][t:t + 1], res=s["res"][t:t + 1]), 3, **how) for t in range(11)]
    assert int(torch.bincount(torch.cat([a[2] for a in alone]).flatten().long()).max()) > 4
    for _ in range(40):
        got = call(s, 3, **how)
        assert all(torch.equal(g, torch.cat(parts)) for g, parts in zip(got, zip(*alone)))
