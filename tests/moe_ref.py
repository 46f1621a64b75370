"""The mixture-of-experts operators from their definitions in 64 bits (plain
torch, any device), and how far fp32 arithmetic may be from them."""
import math

import torch


# ------------------------------------------------------------------ formats --

def blocked_index(R, C, device="cpu"):
    """Byte index [R, C] of scale (r, c) in the 128 x 4 blocked layout."""
    r = torch.arange(R, device=device)[:, None]
    c = torch.arange(C, device=device)[None, :]
    return ((r // 128) * (-(-C // 4)) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4


def blocked(sf, pad=0x7F):
    R, C = sf.shape
    b = torch.full((-(-R // 128) * -(-C // 4) * 512,), pad, dtype=torch.uint8, device=sf.device)
    b[blocked_index(R, C, sf.device)] = sf
    return b


def e4m3_values(codes):
    return codes.view(torch.float8_e4m3fn).float().double()


def e2m1_values(packed):
    """float64 [..., K] of packed codes [..., K / 2]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                       device=packed.device)
    v = torch.stack([packed & 15, packed >> 4], -1).long()
    return lut[v].reshape(*packed.shape[:-1], -1)


def e4m3_step(v):
    """Spacing of E4M3 at |v| (below 2^-6: that of the subnormals)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)


def mxfp8_exponent(amax):
    """Smallest e >= -127 with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(min=-127)


def mxfp8(y):
    """float64 [M, K] -> (values, exponents [M, K / 32])."""
    b = y.reshape(y.shape[0], -1, 32)
    e = mxfp8_exponent(b.abs().amax(-1))
    s = torch.exp2(e.double())[..., None]
    step = e4m3_step(b / s)
    return (torch.round(b / s / step) * step * s).reshape(y.shape), e


def random_mxfp8(gen, R, K, device, scale=1.0):
    """Codes [R, K], blocked scales and float64 values of a random MXFP8 matrix."""
    codes = torch.randint(0, 256, (R, K), generator=gen, device=device, dtype=torch.int32).to(torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)          # no NaN
    # values of ordinary size: exponents near those of normal data
    codes = torch.where(torch.rand((R, K), generator=gen, device=device) < 0.8, (codes & 0x8F) | 0x30, codes & 0xBF)
    sf = torch.randint(119, 128, (R, K // 32), generator=gen, device=device, dtype=torch.int32).to(torch.uint8)
    v = e4m3_values(codes) * torch.exp2(sf.double() - 127).repeat_interleave(32, 1)
    return codes, blocked(sf), v


def random_mxfp4(gen, N, K, device):
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device=device, dtype=torch.int32).to(torch.uint8)
    sf = torch.randint(118, 124, (N, K // 32), generator=gen, device=device, dtype=torch.int32).to(torch.uint8)
    v = e2m1_values(codes) * torch.exp2(sf.double() - 127).repeat_interleave(32, 1)
    return codes, blocked(sf), v


# -------------------------------------------------------------------- norm --

def add_rmsnorm(x, res, w, eps):
    """(h in the element type, y in float64)."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    hd = h.double()
    m = hd.square().mean(-1, keepdim=True) + eps
    r = torch.where(m == 0, torch.zeros_like(m), 1 / torch.sqrt(m))
    return h, hd * r * w.double()


# ----------------------------------------------------------------- routing --

def route(z, k, score, bias, groups, topk_groups, group_top, renormalize, scale):
    """(ids, weights float64) of one batch, row by row from the definition."""
    z = z.double().cpu()
    T, E = z.shape
    n = E // groups
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    b = None if bias is None else bias.double().cpu()
    for t in range(T):
        zt = z[t]
        if score == "softmax":
            ex = torch.where(zt == -math.inf, 0.0, torch.exp(zt - zt.max()))
            s = ex / ex.sum() if float(ex.sum()) != 0 else ex      # a row of -inf has no scores
            if bool(torch.isnan(ex.sum())):
                s = torch.where(zt == -math.inf, 0.0, torch.full_like(zt, math.nan))
        else:
            s = torch.where(zt == -math.inf, 0.0, 1 / (1 + torch.exp(-zt)))
        nan = torch.isnan(s)
        if b is None and groups == 1:
            c = torch.where(nan, s, zt)
        else:
            c = torch.where(zt == -math.inf, -math.inf, s if b is None else s + b)
        # NaN first, then the larger, then the lower index
        before = lambda v, i: (0 if math.isnan(v) else 1, -v if not math.isnan(v) else 0.0, i)  # noqa: E731
        alive = set(range(groups))
        if groups > 1:
            gs = []
            for g in range(groups):
                top = sorted((float(v) for v in c[g * n:(g + 1) * n]), key=lambda v: before(v, 0))[:min(group_top, n)]
                gs.append(sum(top))
            alive = set(sorted(range(groups), key=lambda g: before(gs[g], g))[:topk_groups])
        order = sorted((e for e in range(E) if e // n in alive and float(c[e]) != -math.inf),
                       key=lambda e: before(float(c[e]), e))[:k]
        for j, e in enumerate(order):
            ids[t, j], w[t, j] = e, s[e]
        if renormalize:
            w[t] = w[t] / (w[t].sum() + 1e-20)
    return ids, w * scale


# ----------------------------------------------------------------- experts --

def experts(x, ids, weights, w13, w2):
    """(out, bound) in float64: x [T, H], w13 [E, 2I, H], w2 [E, H, I] values; `bound` is how far a result may be that
    accumulates in fp32, rounds every product row and the result to bf16, and takes the other of two E4M3 neighbours
    only where the activation's own fp32 error reaches the midpoint between them."""
    T, H = x.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    unit = 2.0 ** -23                     # one fp32 operation, whichever way it rounds
    n1, n2 = 2 * (H // 32) + 8, 2 * (I // 32) + 8     # additions into an accumulator
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(tok):
            continue
        wt = weights[tok, slot].double()[:, None]
        xs = x[tok]
        a, aa = xs @ w13[e].T, xs.abs() @ w13[e].abs().T
        g, u = a[:, :I], a[:, I:]
        eg, eu = n1 * unit * aa[:, :I], n1 * unit * aa[:, I:]
        silu = g / (1 + torch.exp(-g))
        act = silu * u
        # |silu'| <= 1.1; the quotient and the exponential cost a few units of the result, 1.2 |g| more for the latter
        ea = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (8 + 1.2 * g.abs()) * 2 * unit * act.abs()
        q, ex = mxfp8(act)
        s = torch.exp2(ex.double()).repeat_interleave(32, 1)
        v, ev = (act / s).abs(), ea / s
        step = e4m3_step(v)
        frac = v / step - torch.floor(v / step)
        flip = (frac - 0.5).abs() * step <= ev
        # a block whose maximum is within its error of the border between two scales may take either: all of its
        # values may then be a step off
        blk = act.abs().reshape(len(tok), -1, 32)
        top, err = blk.amax(-1), ea.reshape(len(tok), -1, 32).amax(-1)
        border = torch.minimum((top - 448 * torch.exp2(ex.double())).abs(), (top - 224 * torch.exp2(ex.double())).abs())
        either = (border <= err).repeat_interleave(32, 1)
        eq = torch.where(flip | either, 2 * step * s, torch.zeros_like(s))
        y = q @ w2[e].T
        ey = eq @ w2[e].abs().T + n2 * unit * (q.abs() @ w2[e].abs().T)
        out.index_add_(0, tok, y * wt)
        bound.index_add_(0, tok, (ey + 2.0 ** -8 * (y.abs() + ey)) * wt.abs() * (1 + 2.0 ** -18))
    return out, bound + 2.0 ** -8 * (out.abs() + bound) + 1e-30
