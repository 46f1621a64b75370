"""The experts' products against their definition in 64 bits; the tolerance is
derived element by element from the operands (see moe_ref.experts)."""
import math

import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


class Layer:
    def __init__(self, T, k, E, H, I, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.xq, self.xs, self.x = moe_ref.random_mxfp8(gen, T, H, "cuda")
        a = [moe_ref.random_mxfp4(gen, 2 * I, H, "cuda") for _ in range(E)]
        b = [moe_ref.random_mxfp4(gen, H, I, "cuda") for _ in range(E)]
        self.w13, self.s13, self.v13 = (torch.stack([m[i] for m in a]) for i in range(3))
        self.w2, self.s2, self.v2 = (torch.stack([m[i] for m in b]) for i in range(3))
        self.ids = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] if k <= E else
                                torch.randint(0, E, (k,), generator=gen, device="cuda") for _ in range(T)]).to(torch.int32)
        self.w = torch.rand((T, k), generator=gen, device="cuda") + 0.1

    def run(self, **kw):
        return mx.mxfp4_moe_experts(self.xq, self.xs, self.ids, self.w, self.w13, self.s13, self.w2, self.s2, **kw)

    def check(self, out, rows=None, long=False):
        torch.cuda.synchronize()
        assert mx.get_device_error() == 0
        ref, bound = moe_ref.experts(self.x, self.ids, self.w, self.v13, self.v2)
        if long:
            # over long sums the worst case over all roundings says little: beside it, the norm of the error. A product
            # row is off by half a step of bf16, 2^-8, and a sum of k of them with signs by chance has a norm of their
            # absolute values over sqrt(k); the result is rounded once more: 2^-8 (1 + sqrt(k)) <= 2^-6 for k <= 9.
            assert float((out.double() - ref).norm()) <= 2.0 ** -6 * float(ref.norm())
        else:
            # the bound (a worst case over all roundings) is itself small beside the results
            assert float(bound.norm()) <= 0.1 * float(ref.norm()) + 1e-20
        err = (out.double() - ref).abs()
        rows = slice(None) if rows is None else rows
        worst = float((err / bound)[rows].max())
        assert worst <= 1.0, worst
        return ref


@pytest.mark.parametrize("T,k,E,H,I", [
    (1, 1, 1, 128, 128),          # one row, one expert, one stage a product
    (1, 2, 4, 256, 128),
    (3, 2, 4, 128, 384),
    (16, 1, 1, 256, 128),         # exactly one MMA width
    (17, 1, 1, 256, 256),
    (32, 1, 1, 1280, 128),        # a full small tile, more stages than the ring holds
    (33, 1, 3, 384, 256),
    (64, 4, 16, 256, 1408),
    (40, 8, 8, 512, 256),         # every token takes every expert: tiles of 40 rows
    (224, 1, 1, 256, 128),        # exactly one large tile
    (225, 1, 1, 256, 128),        # one row in the second
    (500, 3, 5, 640, 384),
    (129, 5, 7, 2560, 256),
    (3000, 3, 6, 128, 128),       # more choices than one placing block takes
    (700, 1, 512, 128, 128),      # as many experts as there may be
    (2, 32, 2, 128, 128),         # the same expert several times for one token
])
def test_experts_match_their_definition(T, k, E, H, I):
    s = Layer(T, k, E, H, I, seed=T + 10 * k + E)
    s.check(s.run())


@pytest.mark.parametrize("T,k,E,H,I", [(1, 8, 8, 7168, 512), (16, 8, 64, 2048, 768), (200, 6, 64, 1024, 1024),
                                       (600, 4, 8, 4096, 1024), (900, 2, 5, 1280, 1408)])
def test_many_stages_and_units_give_the_same_bits_every_time(T, k, E, H, I):
    """Long pipelines over many units, run again and again: whatever is read before it has landed, or overwritten before
    it was read, changes bits from run to run."""
    s = Layer(T, k, E, H, I, seed=20)
    ws = mx.moe_experts_workspace(T, k, E, H, I)
    first = s.run(workspace=ws).clone()
    s.check(first, long=True)
    differ = sum(not torch.equal(s.run(workspace=ws), first) for _ in range(40))
    torch.cuda.synchronize()
    assert differ == 0 and mx.get_device_error() == 0


def test_choices_left_out():
    s = Layer(50, 4, 8, 256, 128, seed=1)
    s.ids[::2, 1] = -1
    s.ids[3] = -1                                  # a token with no choice
    s.ids[4, 2] = 8                                # beyond the experts
    s.ids[5, 0] = -(1 << 31)
    s.ids[6, 3] = (1 << 31) - 1
    s.ids[s.ids == 5] = -1                         # an expert without tokens
    out = torch.full((50, 256), math.nan, dtype=torch.bfloat16, device="cuda")
    s.check(s.run(out=out))
    assert not out[3].any()
    s.ids[:] = -1
    out.fill_(math.nan)
    s.run(out=out)
    torch.cuda.synchronize()
    assert not out.any() and mx.get_device_error() == 0


@pytest.mark.parametrize("T,E", [(64, 8), (300, 3)])
def test_one_expert_takes_everything(T, E):
    s = Layer(T, 1, E, 256, 256, seed=2)
    s.ids[:] = E - 1
    s.check(s.run())


@pytest.mark.parametrize("T,k,E", [(20, 2, 8), (400, 2, 3)])
def test_workspace_contents_do_not_matter(T, k, E):
    s = Layer(T, k, E, 256, 256, seed=3)
    ws = mx.moe_experts_workspace(T, k, E, 256, 256)
    outs = []
    for fill in (0x00, 0xFF, 0x7F):
        ws.fill_(fill)
        outs.append(s.run(workspace=ws))
    s.check(outs[0])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for _ in range(5):                             # the order of the sorted rows changes nothing
        assert torch.equal(s.run(workspace=ws), outs[0])
    # a workspace for more tokens serves fewer
    big = mx.moe_experts_workspace(5 * T, k, E, 256, 256)
    assert torch.equal(s.run(workspace=big), outs[0])


def test_strided_activations_and_output():
    s = Layer(45, 2, 4, 384, 128, seed=4)
    want = s.run()
    wide = torch.zeros((45, 384 + 48), dtype=torch.uint8, device="cuda")
    wide[:, :384] = s.xq
    out = torch.full((45, 384 + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    s.xq = wide[:, :384]
    got = s.run(out=out[:, :384])
    assert torch.equal(got, want) and bool((out[:, 384:] == 9.0).all())
    s.check(got)


def test_nan_stays_in_its_token():
    s = Layer(70, 2, 4, 256, 128, seed=5)
    want = s.run()
    s.xq[7, 30] = 0x7F
    s.xs[moe_ref.blocked_index(70, 8, "cuda")[31, 2]] = 0xFF
    got = s.run()
    torch.cuda.synchronize()
    bad = torch.zeros(70, dtype=torch.bool, device="cuda")
    bad[7] = bad[31] = True
    assert torch.equal(got[~bad], want[~bad]) and bool(torch.isnan(got[bad]).all())


def test_weights_of_zero_and_of_either_sign():
    s = Layer(12, 3, 6, 256, 128, seed=6)
    s.w[:, 1] = 0.0
    s.w[::2, 0] *= -1
    s.check(s.run())


def test_other_stream_empty_batch_and_graph():
    s = Layer(24, 2, 8, 256, 256, seed=7)
    want = s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s.run()
    side.synchronize()
    assert torch.equal(got, want)
    e = mx.mxfp4_moe_experts(s.xq[:0], s.xs[:0], s.ids[:0], s.w[:0], s.w13, s.s13, s.w2, s.s2)
    assert e.shape == (0, 256)
    ws = mx.moe_experts_workspace(24, 2, 8, 256, 256)
    s.run(workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s.run(workspace=ws)
    s.ids.copy_(s.ids.flip(0))                     # other row counts at replay
    s.ids[4:9] = -1
    g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    assert torch.equal(replayed, s.run())
    s.check(replayed)


def test_back_to_back_calls_share_a_workspace():
    a, b = Layer(30, 2, 4, 256, 128, seed=8), Layer(30, 2, 4, 256, 128, seed=9)
    ws = mx.moe_experts_workspace(30, 2, 4, 256, 128)
    outs = [(l, l.run(workspace=ws)) for l in (a, b, a, b)]
    for l, o in outs:
        l.check(o)


def test_python_refusals():
    s = Layer(4, 2, 4, 256, 128)
    with pytest.raises(ValueError):
        mx.mxfp4_moe_experts(s.xq, s.xs, s.ids.long(), s.w, s.w13, s.s13, s.w2, s.s2)
    with pytest.raises(ValueError):
        mx.mxfp4_moe_experts(s.xq, s.xs, s.ids, s.w[:, :1], s.w13, s.s13, s.w2, s.s2)
    with pytest.raises(ValueError):
        mx.mxfp4_moe_experts(s.xq, s.xs[:16], s.ids, s.w, s.w13, s.s13, s.w2, s.s2)
    with pytest.raises(ValueError):
        mx.mxfp4_moe_experts(s.xq, s.xs, s.ids, s.w, s.w13[:, :, :64], s.s13, s.w2, s.s2)
    with pytest.raises(mx.Mxfp4Error):
        s.run(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
