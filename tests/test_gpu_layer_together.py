"""A decoder layer's steps around its attention, run one after another as a server does for a batch of requests with
adapters of their own: projection and adapters, norm and rotation of the heads, (plain attention), projection and adapters,
and the mixture-of-experts half for few tokens. Each step is checked against its definition on the step's own inputs, and
the whole is captured and replayed."""
import pytest
import torch

import layer_ref
import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from block_scaled_fp4_mxfp4_gb300 import moe_layer  # noqa: E402
from test_gpu_qk_norm_rope import rope_table  # noqa: E402


class Step:
    """One decoding step of T requests with hidden size H and Hq / Hk heads of D."""

    def __init__(self, T, H=512, Hq=8, Hk=2, D=64, R=16, L=3, few=16):
        gen = torch.Generator(device="cuda").manual_seed(T)
        rn = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
        self.T, self.H, self.Hq, self.Hk, self.D = T, H, Hq, Hk, D
        N = (Hq + 2 * Hk) * D
        self.x, self.res = rn(T, H).bfloat16(), rn(T, H).bfloat16()
        self.wqkv = mx.mxfp4_quantize((rn(N, H) * H ** -0.5).bfloat16())
        self.wo = mx.mxfp4_quantize((rn(H, Hq * D) * (Hq * D) ** -0.5).bfloat16())
        self.qkv_lora = ((rn(L, R, H) * H ** -0.5).bfloat16(), (rn(L, N, R) * R ** -0.5).bfloat16())
        self.o_lora = ((rn(L, R, Hq * D) * (Hq * D) ** -0.5).bfloat16(), (rn(L, H, R) * R ** -0.5).bfloat16())
        self.ids = torch.randint(-1, L, (T,), device="cuda", generator=gen).to(torch.int32)
        self.scales = rn(L)
        self.wq, self.wk = (1 + 0.1 * rn(D)).bfloat16(), (1 + 0.1 * rn(D)).bfloat16()
        self.table, self.pos = rope_table(1000, D), torch.randint(0, 1000, (T,), device="cuda", generator=gen)
        self.layer = moe_layer.random_layer(8, H, 256, 2, max(T, 16), seed=T, few_tokens=few)
        self.lora_ws = mx.lora_workspace(T, max(H, Hq * D), R, L)

    def __call__(self):
        T, Hq, Hk, D = self.T, self.Hq, self.Hk, self.D
        self.qkv0 = mx.mxfp4_quant_gemm_fused(self.x, *self.wqkv)
        self.qkv = mx.lora_add(self.qkv0, self.x, *self.qkv_lora, self.ids, self.scales, workspace=self.lora_ws)
        q, k, v = self.qkv.unflatten(1, (Hq + 2 * Hk, D)).split([Hq, Hk, Hk], 1)
        self.q, self.k = mx.qk_norm_rope(q, k, self.table, self.pos, self.wq, self.wk)
        kk, vv = (t.repeat_interleave(Hq // Hk, 1).transpose(0, 1).float() for t in (self.k, v))
        p = torch.softmax(self.q.transpose(0, 1).float() @ kk.transpose(1, 2) * D ** -0.5, -1)
        self.att = (p @ vv).transpose(0, 1).reshape(T, Hq * D).bfloat16()
        self.o = mx.mxfp4_quant_gemm_fused(self.att, *self.wo)
        mx.lora_add(self.o, self.att, *self.o_lora, self.ids, self.scales, C=self.o, workspace=self.lora_ws)
        self.out, self.h = self.layer(self.o, self.res)
        return self.out, self.h


def within(got, ref):
    want, bound = ref
    assert float(((got.double() - want).abs() / bound).max()) <= 1.0


@pytest.mark.parametrize("T", [1, 5, 16, 100])
def test_the_steps_of_a_layer_one_after_another(T):
    s = Step(T)
    out, h = s()
    within(s.qkv, layer_ref.lora(s.qkv0, s.x, *s.qkv_lora, s.ids, s.scales, None))
    q, k, _ = s.qkv.unflatten(1, (s.Hq + 2 * s.Hk, s.D)).split([s.Hq, s.Hk, s.Hk], 1)
    within(s.q, layer_ref.head_norm_rope(q, s.wq, s.table, s.pos, 1e-6, False))
    within(s.k, layer_ref.head_norm_rope(k, s.wk, s.table, s.pos, 1e-6, False))
    o0 = mx.mxfp4_quant_gemm_fused(s.att, *s.wo)
    within(s.o, layer_ref.lora(o0, s.att, *s.o_lora, s.ids, s.scales, None))
    assert torch.equal(h, moe_ref.add_rmsnorm(s.o, s.res, s.layer.norm, 1e-6)[0])
    if T <= 16:
        same = mx.mxfp4_moe_layer(s.o, s.layer.norm, s.layer.router, s.layer.w13, s.layer.s13, s.layer.w2, s.layer.s2, 2,
                                  residual=s.res)
        assert torch.equal(out, same[0])
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = s()
    s.x.copy_(s.x.flip(0) * 0.5)
    s.ids.copy_(s.ids.roll(1))
    s.pos.copy_(s.pos.flip(0))
    for _ in range(3):
        graph.replay()
    fresh = s()
    torch.cuda.synchronize()
    assert torch.equal(captured[0], fresh[0]) and torch.equal(captured[1], fresh[1])
    assert mx.get_device_error() == 0


def test_layers_of_few_tokens_and_of_many_agree():
    """The one call and the chain of calls, on a router whose scores lie far apart: the same experts, and results that
    differ by no more than two roundings of logits, codes and sums can make."""
    E, H, I, k = 8, 512, 256, 2
    few = moe_layer.random_layer(E, H, I, k, 18, seed=3, few_tokens=16)
    chain = moe_layer.random_layer(E, H, I, k, 18, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(0)
    # a token's first E channels say which experts it takes
    few.router.zero_()
    few.router[:, :E] = torch.eye(E, device="cuda") * 2
    chain.router.copy_(few.router)
    x = torch.randn((9, H), device="cuda", generator=gen).bfloat16()
    x[:, :E] = 0
    for t in range(9):
        x[t, t % E], x[t, (t + 3) % E] = 3, 2
    a, ha = few(x)
    b, hb = chain(x)
    assert torch.equal(ha, hb)
    # E4M3 codes may differ by a step of 2^-3 in few of 512 terms, weights by a bf16 logit of up to 6: 2^-6
    assert float((a.double() - b.double()).norm()) <= 2.0 ** -5 * float(b.double().norm())
    assert torch.equal(few(x.repeat(2, 1))[0], chain(x.repeat(2, 1))[0])     # 18 tokens: the chain
    with pytest.raises(ValueError):
        moe_layer.random_layer(E, H, I, k, 16, few_tokens=17)


def test_no_tokens(monkeypatch):
    """A layer of zero tokens gives empty results, by the call that it would take for one."""
    x = torch.empty((0, 512), device="cuda").bfloat16()
    for few in (16, 0):
        layer = moe_layer.random_layer(8, 512, 256, 2, 16, few_tokens=few)
        if few == 0:
            monkeypatch.setattr(mx, "mxfp4_moe_layer", None)
        out, h = layer(x, x)
        assert out.shape == h.shape == (0, 512) and out.dtype == h.dtype == torch.bfloat16
