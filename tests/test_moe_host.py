"""The mixture-of-experts entry points without a GPU: exported symbols, sizes,
refusals, and the 64-bit definitions the GPU tests compare with."""
import pytest
import torch

import moe_ref
from block_scaled_fp4_mxfp4_gb300 import build as libbuild

libbuild.build()
from block_scaled_fp4_mxfp4_gb300 import mxfp4 as mx  # noqa: E402

L = mx.lib()
OK, INVALID, SHAPE, MISALIGNED, WORKSPACE, NO_DEVICE = 0, 1, 2, 3, 4, 7


def test_every_declared_symbol_is_exported():
    names = mx.declared_symbols(mx.MOE_HEADER_PATH)
    assert sorted(names) == ["moe_route", "mxfp4_moe_experts", "mxfp4_moe_experts_workspace_bytes",
                             "mxfp8_add_rmsnorm_quantize"]
    for n in names:
        assert hasattr(L, n), n


def norm(**kw):
    a = dict(X=16, ldx=64, res=16, ldr=64, w=16, dtype=0, eps=1e-6, M=4, K=64, H=16, ldh=64, Y=16, ldy=64, Aq=16,
             ldq=64, sf=16)
    a.update(kw)
    return L.mxfp8_add_rmsnorm_quantize(a["X"], a["ldx"], a["res"], a["ldr"], a["w"], a["dtype"], a["eps"], a["M"],
                                        a["K"], a["H"], a["ldh"], a["Y"], a["ldy"], a["Aq"], a["ldq"], a["sf"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(M=0, X=None, w=None, Aq=None, sf=None), OK),
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(K=48), SHAPE), (dict(dtype=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(X=None), INVALID), (dict(w=None), INVALID), (dict(Aq=None), INVALID), (dict(sf=None), INVALID),
    (dict(ldx=32), INVALID), (dict(ldr=32), INVALID), (dict(ldh=32), INVALID), (dict(ldy=32), INVALID),
    (dict(ldq=32), INVALID), (dict(ldx=68), MISALIGNED), (dict(ldr=68), MISALIGNED), (dict(ldh=68), MISALIGNED),
    (dict(ldy=68), MISALIGNED), (dict(ldq=68), MISALIGNED), (dict(X=24), MISALIGNED), (dict(res=24), MISALIGNED),
    (dict(w=24), MISALIGNED), (dict(H=24), MISALIGNED), (dict(Y=24), MISALIGNED), (dict(Aq=20), MISALIGNED),
    (dict(sf=18), MISALIGNED),
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


def route(**kw):
    a = dict(z=16, dtype=2, ldl=64, T=4, E=64, bias=16, score=0, groups=1, topk_groups=1, group_top=2, k=8, renorm=1,
             scale=1.0, ids=16, w=16)
    a.update(kw)
    return L.moe_route(a["z"], a["dtype"], a["ldl"], a["T"], a["E"], a["bias"], a["score"], a["groups"],
                       a["topk_groups"], a["group_top"], a["k"], a["renorm"], a["scale"], a["ids"], a["w"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), OK), (dict(T=0, z=None, ids=None, w=None), OK), (dict(T=-1), INVALID), (dict(dtype=3), INVALID),
    (dict(score=2), INVALID), (dict(ldl=63), INVALID), (dict(E=0), INVALID), (dict(groups=0), INVALID),
    (dict(topk_groups=2), INVALID), (dict(groups=8, topk_groups=0), INVALID), (dict(group_top=3), INVALID),
    (dict(k=0), INVALID), (dict(scale=float("nan")), INVALID), (dict(groups=5), SHAPE), (dict(k=33), SHAPE),
    (dict(groups=16, topk_groups=1, k=5), SHAPE), (dict(E=513, ldl=513), SHAPE), (dict(z=None), INVALID),
    (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(z=18), MISALIGNED), (dict(bias=18), MISALIGNED),
    (dict(ids=18), MISALIGNED), (dict(w=18), MISALIGNED), (dict(dtype=0, z=17), MISALIGNED),
])
def test_route_refusals(kw, want):
    assert route(**kw) == want


def experts(**kw):
    a = dict(x=256, ldx=256, xs=256, ids=256, w=256, w13=256, s13=256, w2=256, s2=256, out=256, ldo=256, T=4, k=2, E=8,
             H=256, I=128, ws=256, wsb=1 << 40)
    a.update(kw)
    return L.mxfp4_moe_experts(a["x"], a["ldx"], a["xs"], a["ids"], a["w"], a["w13"], a["s13"], a["w2"], a["s2"],
                               a["out"], a["ldo"], a["T"], a["k"], a["E"], a["H"], a["I"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(H=0), INVALID),
    (dict(I=0), INVALID), (dict(k=33), SHAPE), (dict(E=513), SHAPE), (dict(H=192), SHAPE), (dict(I=64), SHAPE),
    (dict(T=1 << 30), SHAPE), (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(ids=None), INVALID),
    (dict(w=None), INVALID), (dict(w13=None), INVALID), (dict(s13=None), INVALID), (dict(w2=None), INVALID),
    (dict(s2=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ldx=128), INVALID),
    (dict(ldo=128), INVALID), (dict(ldx=264), MISALIGNED), (dict(ldo=260), MISALIGNED), (dict(x=264), MISALIGNED),
    (dict(w13=272), MISALIGNED), (dict(w2=272), MISALIGNED), (dict(s13=264), MISALIGNED), (dict(xs=264), MISALIGNED),
    (dict(out=264), MISALIGNED), (dict(ws=128), MISALIGNED), (dict(ids=258), MISALIGNED), (dict(wsb=0), WORKSPACE),
])
def test_experts_refusals(kw, want):
    assert experts(**kw) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU answer")
def test_valid_calls_without_gpu_report_no_device():
    assert norm() == route() == experts() == NO_DEVICE


def test_workspace_grows_with_tokens():
    f = mx.moe_experts_workspace_bytes
    sizes = [f(T, 8, 64, 2048, 768) for T in (1, 2, 7, 64, 255, 256, 257, 1000, 1024, 1025, 4096, 9999)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert f(0, 8, 64, 2048, 768) == 0 and f(4, 8, 64, 2000, 768) == 0
    # at least the activations between the products and the rows before they are summed
    assert f(100, 4, 16, 512, 256) >= 400 * (256 + 256 // 32 + 2 * 512)


def test_reference_mxfp8_is_the_type_of_torch():
    gen = torch.Generator().manual_seed(1)
    y = torch.randn((64, 256), generator=gen, dtype=torch.float64) * torch.exp2(torch.randn((64, 1), generator=gen) * 20)
    y[3] = 0
    y[4, :32] = 448.0 * 2.0 ** 5            # the border: exact, with the smaller scale
    q, e = moe_ref.mxfp8(y)
    s = torch.exp2(e.double()).repeat_interleave(32, 1)
    assert torch.equal(q, (y / s).float().to(torch.float8_e4m3fn).double() * s)
    assert int(e[4, 0]) == 5 and bool((e[3] == -127).all())
    top = y.reshape(64, 8, 32).abs().amax(-1)
    assert bool((top <= 448 * torch.exp2(e.double())).all())
    assert bool(((top > 224 * torch.exp2(e.double())) | (top == 0)).all())


def test_reference_route_on_a_row_by_hand():
    z = torch.tensor([[0.0, 2.0, 2.0, -float("inf"), 1.0, -1.0]])
    ids, w = moe_ref.route(z, 4, "softmax", None, 1, 1, 1, True, 2.0)
    assert ids.tolist() == [[1, 2, 4, 0]]
    assert abs(float(w.sum()) - 2.0) < 1e-12 and abs(float(w[0, 0] / w[0, 3]) - 7.38905609893065) < 1e-12
    ids, w = moe_ref.route(z, 3, "sigmoid", torch.tensor([0, 0, 0, 9.0, 0, 9.0]), 2, 1, 2, False, 1.0)
    assert ids.tolist() == [[5, 4, -1]] and float(w[0, 2]) == 0.0
