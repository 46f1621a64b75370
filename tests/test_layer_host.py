"""The entry points of include/mxfp4_layer.h without a GPU: exported symbols, sizes and refusals."""
import pytest
import torch

import layer_ref
from block_scaled_fp4_mxfp4_gb300 import build as libbuild

libbuild.build()
from block_scaled_fp4_mxfp4_gb300 import mxfp4 as mx  # noqa: E402

L = mx.lib()
OK, INVALID, SHAPE, MISALIGNED, WORKSPACE, NO_DEVICE = 0, 1, 2, 3, 4, 7


def test_every_declared_symbol_is_exported():
    names = mx.declared_symbols(mx.LAYER_HEADER_PATH)
    assert {"lora_add", "lora_workspace_bytes", "qk_norm_rope"} <= set(names)
    for n in names:
        assert hasattr(L, n), n


def lora(**kw):
    a = dict(x=16, ldx=64, a=16, b=16, ids=16, scales=16, ranks=16, base=16, ldb=96, dtype=0, c=32, ldc=96, T=4, K=64,
             N=96, R=8, L=3, ws=256, wsb=1 << 40)
    a.update(kw)
    return L.lora_add(a["x"], a["ldx"], a["a"], a["b"], a["ids"], a["scales"], a["ranks"], a["base"], a["ldb"],
                      a["dtype"], a["c"], a["ldc"], a["T"], a["K"], a["N"], a["R"], a["L"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), OK), (dict(T=0, x=None, a=None, b=None, ids=None, base=None, c=None, ws=None), OK), (dict(T=-1), INVALID),
    (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(R=0), INVALID), (dict(L=0), INVALID), (dict(dtype=2), INVALID),
    (dict(K=60), SHAPE), (dict(N=92), SHAPE), (dict(R=12), SHAPE), (dict(R=264), SHAPE), (dict(L=4097), SHAPE),
    (dict(T=1 << 31), SHAPE), (dict(T=(1 << 30) + 1), SHAPE), (dict(K=(1 << 30) + 8, ldx=1 << 31), SHAPE), (dict(N=(1 << 30) + 8), SHAPE),
    (dict(x=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(ids=None), INVALID),
    (dict(base=None), INVALID), (dict(c=None), INVALID), (dict(ws=None), INVALID), (dict(ldx=56), INVALID),
    (dict(ldb=88), INVALID), (dict(ldc=88), INVALID), (dict(c=16, ldc=104), INVALID), (dict(ldx=68), MISALIGNED),
    (dict(ldb=100), MISALIGNED), (dict(ldc=100), MISALIGNED), (dict(x=24), MISALIGNED), (dict(a=24), MISALIGNED),
    (dict(b=24), MISALIGNED), (dict(base=24), MISALIGNED), (dict(c=24), MISALIGNED), (dict(ids=18), MISALIGNED),
    (dict(scales=18), MISALIGNED), (dict(ranks=18), MISALIGNED), (dict(ws=128), MISALIGNED), (dict(wsb=0), WORKSPACE),
])
def test_lora_refusals(kw, want):
    assert lora(**kw) == want


def test_lora_workspace_grows_with_everything():
    f = mx.lora_workspace_bytes
    sizes = [1, 2, 3, 7, 8, 16, 63, 64, 65, 127, 128, 500, 607, 608, 609, 1000, 4096, 19455, 19456, 19457, 70000]
    for Ls in (1, 5, 4096):
        for R in (8, 64, 256):
            for K in (8, 512, 520, 7168, 1 << 20):
                got = [f(T, K, R, Ls) for T in sizes]
                assert got == sorted(got) and got[0] > 0
        for T in sizes:
            assert f(T, 64, 8, Ls) <= f(T, 7168, 8, Ls) <= f(T, 7168, 16, Ls) <= f(T, 7168, 16, 4096)
    assert f(0, 64, 8, 1) == 0 and f(4, 60, 8, 1) == 0 and f(4, 64, 12, 1) == 0 and f(4, 64, 8, 0) == 0


def qk(**kw):
    a = dict(q=16, q_st=256, q_sh=64, k=16, k_st=64, k_sh=64, wq=16, wk=16, table=16, pos=16, pos64=0, dtype=0, eps=1e-6,
             T=4, Hq=4, Hk=1, D=64, rot=64, inter=0, P=10, qo=32, qo_st=256, qo_sh=64, ko=32, ko_st=64, ko_sh=64)
    a.update(kw)
    return L.qk_norm_rope(a["q"], a["q_st"], a["q_sh"], a["k"], a["k_st"], a["k_sh"], a["wq"], a["wk"], a["table"],
                          a["pos"], a["pos64"], a["dtype"], a["eps"], a["T"], a["Hq"], a["Hk"], a["D"], a["rot"],
                          a["inter"], a["P"], a["qo"], a["qo_st"], a["qo_sh"], a["ko"], a["ko_st"], a["ko_sh"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), OK), (dict(Hq=0, Hk=0), OK), (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=-1), INVALID),
    (dict(D=0), INVALID), (dict(rot=-16), INVALID), (dict(rot=80), INVALID), (dict(dtype=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(D=60, rot=16), SHAPE),
    (dict(D=264), SHAPE), (dict(rot=24), SHAPE), (dict(rot=20, inter=1), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(T=1 << 29), SHAPE), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qo=None), INVALID),
    (dict(ko=None), INVALID), (dict(table=None), INVALID), (dict(pos=None), INVALID), (dict(P=0), INVALID),
    (dict(qo_st=0), INVALID), (dict(qo_sh=0), INVALID), (dict(ko_st=-56), INVALID), (dict(Hk=2, ko_sh=56), INVALID),
    (dict(qo=16, qo_st=512), INVALID), (dict(ko=16, ko_sh=8), INVALID), (dict(q_st=260), MISALIGNED),
    (dict(q_sh=68), MISALIGNED), (dict(k_st=68), MISALIGNED), (dict(ko_sh=68), MISALIGNED), (dict(q=24), MISALIGNED),
    (dict(k=24), MISALIGNED), (dict(qo=24), MISALIGNED), (dict(ko=24), MISALIGNED), (dict(wq=24), MISALIGNED),
    (dict(wk=24), MISALIGNED), (dict(table=24), MISALIGNED), (dict(pos=18), MISALIGNED), (dict(pos=20, pos64=1), MISALIGNED),
])
def test_qk_refusals(kw, want):
    assert qk(**kw) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU answer")
def test_valid_calls_without_gpu_report_no_device():
    assert lora() == qk() == qk(Hk=0, k=None, ko=None, k_st=3) == qk(rot=0, table=None, pos=None, P=0) == NO_DEVICE


def test_reference_rotation_keeps_lengths_and_turns_by_the_angle():
    x = torch.randn((3, 2, 16), dtype=torch.float64)
    angle = torch.arange(5, dtype=torch.float64)[:, None] * torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64)
    table = torch.cat([torch.cos(angle), torch.sin(angle)], 1)
    pos = torch.tensor([0, 4, 2])
    for inter in (False, True):
        z, _ = layer_ref.head_norm_rope(x, None, table, pos, 0.0, inter)
        assert torch.allclose(z.norm(dim=-1), x.norm(dim=-1)) and torch.equal(z[0], x[0]) and torch.equal(z[..., 8:], x[..., 8:])
        i, j = (0, 1) if inter else (0, 4)
        turned = torch.complex(x[1, :, i], x[1, :, j]) * torch.polar(torch.tensor(1.0).double(), torch.tensor(4.0).double())
        assert torch.allclose(torch.complex(z[1, :, i], z[1, :, j]), turned)


def test_reference_adapters_are_a_low_rank_update_of_the_weight():
    base = torch.zeros((5, 7), dtype=torch.float32)
    x, a, b = torch.randn(5, 9), torch.randn(2, 3, 9), torch.randn(2, 7, 3)
    ids = torch.tensor([1, 0, -1, 1, 2])
    c, bound = layer_ref.lora(base, x, a, b, ids, torch.tensor([0.5, 2.0]), torch.tensor([3, 1]))
    assert torch.allclose(c[1], 0.5 * (b[0] @ a[0]).double() @ x[1].double(), atol=1e-5)
    assert torch.allclose(c[3], 2.0 * (b[1, :, :1] @ a[1, :1]).double() @ x[3].double(), atol=1e-5)
    assert not c[2].any() and not c[4].any() and bool((bound >= 0).all())


def layer(**kw):
    a = dict(x=256, ldx=256, res=512, ldr=256, w=16, eps=1e-6, router=16, bias=16, score=0, groups=1, topk_groups=1,
             group_top=2, k=2, renorm=1, scale=1.0, w13=32, s13=16, w2=32, s2=16, h=1024, ldh=256, out=2048, ldo=256, ids=16,
             ow=16, T=4, E=8, H=256, I=128, ws=256, wsb=1 << 40)
    a.update(kw)
    return L.mxfp4_moe_layer(a["x"], a["ldx"], a["res"], a["ldr"], a["w"], a["eps"], a["router"], a["bias"], a["score"],
                             a["groups"], a["topk_groups"], a["group_top"], a["k"], a["renorm"], a["scale"], a["w13"],
                             a["s13"], a["w2"], a["s2"], a["h"], a["ldh"], a["out"], a["ldo"], a["ids"], a["ow"], a["T"],
                             a["E"], a["H"], a["I"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(T=17), SHAPE), (dict(k=0), INVALID), (dict(k=9), SHAPE), (dict(E=0), INVALID),
    (dict(E=513), SHAPE), (dict(H=192), SHAPE), (dict(I=64), SHAPE), (dict(H=0), INVALID), (dict(I=0), INVALID),
    (dict(score=2), INVALID), (dict(groups=0), INVALID), (dict(groups=3), SHAPE), (dict(groups=2, topk_groups=3), INVALID),
    (dict(groups=8, topk_groups=1), SHAPE), (dict(group_top=3), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(router=None), INVALID), (dict(w13=None), INVALID), (dict(s13=None), INVALID),
    (dict(w2=None), INVALID), (dict(s2=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(ldx=128), INVALID), (dict(ldr=128), INVALID), (dict(ldh=128), INVALID), (dict(ldo=128), INVALID),
    (dict(h=2048), INVALID), (dict(h=256, ldh=264), INVALID), (dict(h=512, ldh=264), INVALID), (dict(ldx=260), MISALIGNED),
    (dict(ldr=260), MISALIGNED), (dict(ldh=260), MISALIGNED), (dict(ldo=260), MISALIGNED), (dict(x=264), MISALIGNED),
    (dict(res=520), MISALIGNED), (dict(h=1032), MISALIGNED), (dict(out=2056), MISALIGNED), (dict(w=24), MISALIGNED),
    (dict(router=24), MISALIGNED), (dict(bias=18), MISALIGNED), (dict(w13=48), MISALIGNED), (dict(w2=48), MISALIGNED),
    (dict(s13=24), MISALIGNED), (dict(s2=24), MISALIGNED), (dict(ids=18), MISALIGNED), (dict(ow=18), MISALIGNED),
    (dict(ws=128), MISALIGNED), (dict(wsb=0), WORKSPACE),
])
def test_moe_layer_refusals(kw, want):
    assert layer(**kw) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU answer")
def test_valid_moe_layer_calls_without_gpu_report_no_device():
    assert layer() == layer(res=None, bias=None, h=None, ids=None, ow=None) == layer(h=256) == layer(out=256) == NO_DEVICE


def test_moe_layer_workspace_grows_with_tokens():
    f = mx.moe_layer_workspace_bytes
    sizes = [f(T, 8, 64, 2048, 768) for T in range(1, 17)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert f(0, 8, 64, 2048, 768) == 0 and f(17, 8, 64, 2048, 768) == 0 and f(4, 8, 64, 2000, 768) == 0


@pytest.mark.parametrize("code", range(127))
def test_six_digits_are_the_value_of_an_e4m3_code(code):
    """The few-token layer's form of an MXFP8 activation: its magnitude, a whole number of 2^-9, from six E2M1 digits that
    stand 8 apart, as csrc/moe_few.cu makes them."""
    n = int(torch.tensor([code], dtype=torch.uint8).view(torch.float8_e4m3fn).double() * 512)
    assert n < 1 << 18
    digits, rest = [], n
    for _ in range(5):
        d = ((rest + 3) & 7) - 3
        rest = (rest - d) // 8
        digits.append(d)
    digits.append(rest)
    if rest in (5, 7):
        digits[5] = 6
        digits[4] += -8 if rest == 5 else 8
    # an E2M1 code for each, the value of which is half the digit
    levels = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    codes = [abs(d) if abs(d) <= 4 else abs(d) // 2 + 2 for d in digits]
    assert all(2 * levels[c] == abs(d) for c, d in zip(codes, digits))
    assert sum(d * 8 ** i for i, d in enumerate(digits)) == n
    # scales 2^(e - 8 + 3 i) of an activation scale 2^e: half a digit of 8^i in units of 2^-9
    assert sum((1 if d > 0 else -1) * levels[c] * 2.0 ** (3 * i - 8) for i, (c, d) in enumerate(zip(codes, digits))) == n / 512
