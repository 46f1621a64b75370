"""The feed-forward half of a mixture-of-experts decoder layer in MXFP8 x MXFP4.

    h       = x + residual                      y = RMSNorm(h)
    logits  = y Wr^T                            ids, weights = route(logits)
    out     = sum over a token's k experts of weight * W2 (silu(G y) * (U y))

Three calls of the library (norm with its 8-bit output, routing, experts'
products) around one small dense product for the router's logits (torch's, in
bf16, so the logits are rounded to bf16). The next layer's norm adds ``out`` to
``h``.

    python -m block_scaled_fp4_mxfp4_gb300.moe_layer [--tokens 1 16 256 4096]

times a layer of random weights.
"""
import argparse

import torch

from . import mxfp4 as mx


class MoeLayer:
    """Quantizes the experts' bf16 weights once and keeps a workspace for up to
    ``max_tokens`` tokens (1.3 GB at 4096 of 8 choices, 7168 x 2048). Layers that
    run one after another on one stream may share one: pass the first one's
    ``workspace`` to the others.

    gate, up : bf16 [E, I, H]     down : bf16 [E, H, I]
    router   : bf16 [E, H]        norm : bf16 [H]
    bias     : fp32 [E] or None, added to the scores for the choice of experts
    """

    def __init__(self, gate, up, down, router, norm, k, max_tokens, bias=None, score="softmax", groups=1,
                 topk_groups=1, renormalize=True, scale=1.0, eps=1e-6, group_top=2, workspace=None):
        E, I, H = gate.shape
        self.E, self.I, self.H, self.k = E, I, H, k
        self.router, self.norm, self.bias, self.eps = router, norm, bias, eps
        self.how = dict(score=score, groups=groups, topk_groups=topk_groups, group_top=group_top, renormalize=renormalize,
                        scale=scale)
        dev = gate.device
        self.w13 = torch.empty((E, 2 * I, H // 2), dtype=torch.uint8, device=dev)
        self.s13 = torch.empty((E, mx.sf_bytes(2 * I, H, 32)), dtype=torch.uint8, device=dev)
        self.w2 = torch.empty((E, H, I // 2), dtype=torch.uint8, device=dev)
        self.s2 = torch.empty((E, mx.sf_bytes(H, I, 32)), dtype=torch.uint8, device=dev)
        for e in range(E):
            mx.mxfp4_quantize(torch.cat([gate[e], up[e]]), Aq=self.w13[e], A_sf=self.s13[e])
            mx.mxfp4_quantize(down[e], Aq=self.w2[e], A_sf=self.s2[e])
        if workspace is None:
            workspace = mx.moe_experts_workspace(max_tokens, k, E, H, I, dev)
        elif workspace.numel() < mx.moe_experts_workspace_bytes(max_tokens, k, E, H, I):
            raise ValueError(f"workspace has {workspace.numel()} bytes, {max_tokens} tokens need "
                             f"{mx.moe_experts_workspace_bytes(max_tokens, k, E, H, I)}")
        self.workspace = workspace

    def __call__(self, x, residual=None):
        """(out, h): the experts' sum and the residual stream, bf16 [T, H] (h = x without a residual)."""
        q, sf, h, y = mx.mxfp8_add_rmsnorm_quantize(x, self.norm, self.eps, residual=residual, want_y=True)
        logits = y @ self.router.T
        ids, weights = mx.moe_route(logits, self.k, bias=self.bias, **self.how)
        out = mx.mxfp4_moe_experts(q, sf, ids, weights, self.w13, self.s13, self.w2, self.s2,
                                   workspace=self.workspace)
        return out, x if h is None else h


def random_layer(E=32, H=7168, I=2048, k=8, max_tokens=4096, seed=0, **how):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = lambda *s: (torch.randn(s, device="cuda", generator=gen) * s[-1] ** -0.5).bfloat16()  # noqa: E731
    return MoeLayer(w(E, I, H), w(E, I, H), w(E, H, I), w(E, H), torch.ones(H, device="cuda").bfloat16(), k, max_tokens,
                    **how)


def main():
    ap = argparse.ArgumentParser(description="time a mixture-of-experts layer of random weights")
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 16, 256, 4096])
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--intermediate", type=int, default=2048)
    ap.add_argument("--k", type=int, default=8)
    a = ap.parse_args()
    layer = random_layer(a.experts, a.hidden, a.intermediate, a.k, max(a.tokens))
    for T in a.tokens:
        x = torch.randn((T, a.hidden), device="cuda").bfloat16()
        res = torch.randn((T, a.hidden), device="cuda").bfloat16()
        layer(x, res)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(x, res)
        for _ in range(3):
            graph.replay()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"{T:6d} tokens: {start.elapsed_time(end) * 50:9.1f} us a layer (captured, inputs warm)")
    code = mx.get_device_error()
    if code:
        raise SystemExit(f"a kernel gave up waiting (code {code})")


if __name__ == "__main__":
    main()
