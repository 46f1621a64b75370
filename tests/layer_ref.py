"""Low-rank adapters and the norm and rotation of heads from their definitions in 64 bits (plain torch, any device), and
how far fp32 arithmetic may be from them."""
import torch

UNIT = 2.0 ** -23          # one fp32 operation, whichever way it rounds


def lora(base, x, a, b, ids, scales, ranks):
    """(c, bound) in float64 of base [T, N], x [T, K], a [L, R, K], b [L, N, R]."""
    T, N = base.shape
    L, R, K = a.shape
    c = base.double().clone()
    bound = torch.zeros_like(c)
    n1, n2 = K // 16 + 40, R // 8 + 8          # additions into an accumulator: one a step, then over warps and splits
    for i in range(L):
        tok = torch.nonzero(ids == i).flatten()
        r = R if ranks is None else max(0, min(R, int(ranks[i])))
        if not len(tok) or not r:
            continue
        s = 1.0 if scales is None else float(scales[i])
        xi, ai, bi = x[tok].double(), a[i, :r].double(), b[i, :, :r].double()
        u = xi @ ai.T * s
        # the sum's own error, the scale, and two bf16 of 8 bits and a half step each
        eu = abs(s) * n1 * 2 * UNIT * (xi.abs() @ ai.abs().T) + (2.0 ** -17 + UNIT) * u.abs()
        d = u @ bi.T
        c[tok] += d
        bound[tok] = (eu + n2 * 2 * UNIT * u.abs()) @ bi.abs().T + 2 * UNIT * (base[tok].double().abs() + d.abs())
    return c, bound + torch.finfo(base.dtype).eps / 2 * (c.abs() + bound) + torch.finfo(base.dtype).smallest_normal * 2.0 ** -8


def head_norm_rope(x, w, table, positions, eps, interleaved):
    """(out, bound) in float64 of x [T, H, D]."""
    D = x.shape[-1]
    xd = x.double()
    if w is None:
        y = xd
    else:
        m = xd.square().mean(-1, keepdim=True) + eps
        y = xd * torch.where(m == 0, 0.0, 1 / torch.sqrt(m)) * w.double()
    z, mag = y.clone(), y.abs()
    if table is not None and table.shape[1]:
        rot = table.shape[1]
        half = rot // 2
        i = torch.arange(0, rot, 2) if interleaved else torch.arange(half)
        j = i + 1 if interleaved else i + half
        inside = (positions >= 0) & (positions < table.shape[0])
        t = table.double()[positions.long().clamp(0, table.shape[0] - 1)][:, None]
        cos, sin = t[..., :half], t[..., half:]
        z[..., i] = y[..., i] * cos - y[..., j] * sin
        z[..., j] = y[..., j] * cos + y[..., i] * sin
        mag = mag.clone()
        mag[..., i] = (y[..., i] * cos).abs() + (y[..., j] * sin).abs()
        mag[..., j] = (y[..., j] * cos).abs() + (y[..., i] * sin).abs()
        z[~inside] = float("nan")
    # the sum of squares, its root and reciprocal, four products and a sum
    e = (D + 24) * UNIT * mag
    fi = torch.finfo(x.dtype)
    return z, e + fi.eps / 2 * (z.abs() + e) + fi.smallest_normal * fi.eps
