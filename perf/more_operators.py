"""What is measured of the operators around a decoder layer's attention, for requests that bring adapters.

  lora   C = base + scale_a * (x A_a^T) B_a^T, a the adapter of each token's request: low-rank updates of many requests
         beside a projection that all of them share
  qk     queries and keys of a token: RMSNorm of each head, then the rotation by its position, in one pass
  layer  the whole feed-forward half of a mixture-of-experts layer for a few tokens: h = x + residual, its RMSNorm, the
         router's scores and choice, the experts' products in MXFP8 x MXFP4, and their weighted sum

Each case names one of them and its sizes. `run` computes it in plain torch operations, or, where `own` is true, with
this package's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # decoding one request that has an adapter, beside the package's decode projection
        dict(name="lora_decode_1", op="lora", T=1, K=7168, N=2112, R=16, L=8, mix="own", none=0.0, ragged=False,
             dtype="bf16"),
        # decoding sixteen requests, nearly all with adapters of their own
        dict(name="lora_decode_16", op="lora", T=16, K=7168, N=2112, R=32, L=64, mix="own", none=0.0, ragged=False,
             dtype="bf16"),
        # decoding and prefilling mixed: adapters of several ranks, a third of the requests without one, a projection in fp16
        dict(name="lora_ragged_333", op="lora", T=333, K=2048, N=7168, R=24, L=20, mix="runs", none=0.33, ragged=True,
             dtype="fp16"),
        # prefill of a few long prompts
        dict(name="lora_prefill_4096", op="lora", T=4096, K=7168, N=2112, R=64, L=6, mix="runs", none=0.0, ragged=False,
             dtype="bf16"),
        # decoding sixteen sequences, grouped-query heads
        dict(name="qk_decode_16", op="qk", T=16, Hq=32, Hk=8, D=128, rot=128, norm=True, interleaved=False, P=8192,
             dtype="bf16"),
        # an odd batch, only a third of each head rotated, pairs side by side, no norm
        dict(name="qk_ragged_777", op="qk", T=777, Hq=24, Hk=1, D=192, rot=64, norm=False, interleaved=True, P=40000,
             dtype="fp16"),
        # prefill of long prompts
        dict(name="qk_prefill_8192", op="qk", T=8192, Hq=64, Hk=8, D=128, rot=128, norm=True, interleaved=False, P=131072,
             dtype="bf16"),
        # decoding one sequence: the experts' weights are all the traffic
        dict(name="layer_1", op="layer", T=1, E=32, k=8, H=7168, I=2048, score="softmax", bias=False, groups=1,
             topk_groups=1, group_top=2, renormalize=True, scale=1.0, residual=True),
        # a few drafted tokens, a router with groups and a bias for balance, sizes that are no powers of two
        dict(name="layer_5", op="layer", T=5, E=40, k=6, H=2560, I=1408, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_top=2, renormalize=True, scale=2.5, residual=True),
        # decoding sixteen sequences over many small experts
        dict(name="layer_16", op="layer", T=16, E=128, k=8, H=2048, I=768, score="softmax", bias=False, groups=1,
             topk_groups=1, group_top=2, renormalize=True, scale=1.0, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "qk", "layer"])
    while op == "lora":
        c = dict(op=op, T=_log_int(rng, 1, 4096), K=8 * _log_int(rng, 32, 896), N=8 * _log_int(rng, 32, 896),
                 R=8 * _log_int(rng, 1, 16), L=_log_int(rng, 1, 64), mix=rng.choice(["own", "runs"]),
                 none=rng.choice([0.0, 0.0, 0.33]), ragged=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))
        # no more tokens' data, products or adapters than the largest listed cases
        if (c["T"] * (c["K"] + c["N"]) <= 4096 * 9280 and c["L"] * c["R"] * (c["K"] + c["N"]) <= 64 * 32 * 9280
                and c["T"] * c["L"] * c["R"] * (c["K"] + c["N"]) <= 4096 * 6 * 64 * 9280):
            return c
    while op == "qk":
        D = rng.choice([64, 96, 128, 192, 256])
        c = dict(op=op, T=_log_int(rng, 1, 8192), Hq=_log_int(rng, 1, 64), Hk=_log_int(rng, 1, 8), D=D,
                 rot=rng.choice([D, D // 2, 32]), norm=rng.random() < 0.7, interleaved=rng.random() < 0.5,
                 P=_log_int(rng, 1000, 131072), dtype=rng.choice(["bf16", "fp16"]))
        if c["T"] * (c["Hq"] + c["Hk"]) * D <= 8192 * 72 * 128:
            return c
    while True:
        groups = rng.choice([1, 1, 2, 4])
        E = groups * _log_int(rng, max(1, 8 // groups), 128 // groups)
        topk_groups = rng.randint(1, groups)
        c = dict(op=op, T=rng.randint(1, 16), E=E, k=rng.randint(1, min(8, topk_groups * (E // groups))),
                 H=128 * _log_int(rng, 4, 56), I=128 * _log_int(rng, 2, 16), score=rng.choice(["softmax", "sigmoid"]),
                 bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                 renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), residual=rng.random() < 0.8)
        # no more weights than the largest listed case
        if E * c["H"] * c["I"] <= 32 * 7168 * 2048 and c["T"] * c["k"] * c["H"] * c["I"] <= 16 * 8 * 4096 * 1024:
            return c


# ----------------------------------------------------------------- inputs --

def _pow2(n):
    """2^n in fp32, exactly, for whole n in -127 .. 127."""
    n = n.to(torch.int32)
    return torch.where(n > -127, (n + 127) << 23, 0x00400000).view(torch.float32)


def _blocked(sf):
    """Scale bytes [R, C] in the 128 x 4 blocked layout, padded with 0x7F."""
    R, C = sf.shape
    Rp, Cp = -(-R // 128) * 128, -(-C // 4) * 4
    p = torch.full((Rp, Cp), 0x7F, dtype=torch.uint8, device=sf.device)
    p[:R, :C] = sf
    return p.reshape(Rp // 128, 4, 32, Cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _unblocked(b, R, C):
    """Scale bytes [..., R, C] from the blocked layout [..., bytes]."""
    lead, n = b.shape[:-1], b.dim() - 1
    p = b.reshape(*lead, -(-R // 128), -(-C // 4), 32, 4, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return p.reshape(*lead, -(-R // 128) * 128, -(-C // 4) * 4)[..., :R, :C]


def _to_mxfp4(w):
    """fp32 [N, K] -> (packed E2M1 codes [N, K/2], scale bytes [N, K/32]); the scale is 2^(floor(log2 amax) - 2)."""
    N, K = w.shape
    b = w.reshape(N, K // 32, 32)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full((1,), -127, device=w.device, dtype=torch.int32))
    e = e.clamp(-127, 127)
    v = (b * _pow2(-e)[..., None]).reshape(N, K)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(v.abs(), edges).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _experts_weights(E, N, K, gen):
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    sf = []
    for e in range(E):
        q[e], s = _to_mxfp4(torch.randn((N, K), device="cuda", generator=gen) * K ** -0.5)
        sf.append(_blocked(s))
    return q, torch.stack(sf)


def _adapter_ids(c, gen):
    """The adapter of each token, -1 for none."""
    T, L = c["T"], c["L"]
    if c["mix"] == "own":
        # a batch of decoding requests: as few as possible share an adapter
        order = torch.randperm(L, device="cuda", generator=gen)
        ids = order[torch.arange(T, device="cuda") % L]
    else:
        # prompts of random lengths, one after another
        starts = torch.rand(T, device="cuda", generator=gen) < min(1.0, 2.0 * L / T)
        run = torch.cumsum(starts, 0)
        ids = torch.randint(0, L, (T + 1,), device="cuda", generator=gen)[run]
    if c["none"]:
        # requests, not tokens, go without an adapter
        drop = torch.rand(L, device="cuda", generator=gen) < c["none"]
        ids = torch.where(drop[ids], -1, ids)
    return ids.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    c = dict(case)
    if c["op"] == "lora":
        T, K, N, R, L = c["T"], c["K"], c["N"], c["R"], c["L"]
        # activations have a few channels far larger than the others
        amp = torch.where(torch.rand(K, device="cuda", generator=gen) < 0.01, 8.0, 1.0)
        c["x"] = (randn(T, K) * amp).bfloat16()
        c["base"] = randn(T, N).to(DTYPES[c["dtype"]])
        c["a"] = (randn(L, R, K) * K ** -0.5).bfloat16()
        c["b"] = (randn(L, N, R) * R ** -0.5).bfloat16()
        c["ids"] = _adapter_ids(c, gen)
        c["scales"] = 0.5 + 1.5 * torch.rand(L, device="cuda", generator=gen)
        c["ranks"] = None
        if c["ragged"]:
            c["ranks"] = torch.randint(1, R + 1, (L,), device="cuda", generator=gen).to(torch.int32)
    elif c["op"] == "qk":
        T, Hq, Hk, D, rot, P = c["T"], c["Hq"], c["Hk"], c["D"], c["rot"], c["P"]
        dt = DTYPES[c["dtype"]]
        # queries, keys and values of a token lie in one row, as one projection writes them
        c["qkv"] = randn(T, (Hq + 2 * Hk) * D).to(dt)
        c["wq"] = (1 + 0.2 * randn(D)).to(dt) if c["norm"] else None
        c["wk"] = (1 + 0.2 * randn(D)).to(dt) if c["norm"] else None
        # a prompt's tokens follow one another from some position on
        start = torch.randint(0, max(1, P - T + 1), (1,), device="cuda", generator=gen)
        c["pos"] = ((start + torch.arange(T, device="cuda")) % P).to(torch.int32)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * inv
        c["table"] = torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()
    else:
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        amp = torch.where(torch.rand(H, device="cuda", generator=gen) < 0.01, 20.0, 1.0)
        c["x"] = (randn(T, H) * amp).bfloat16()
        c["res"] = (randn(T, H) * 2 * amp).bfloat16() if c["residual"] else None
        c["weight"] = (1 + 0.2 * randn(H)).bfloat16()
        c["router"] = (randn(E, H) * 1.5 * H ** -0.5).bfloat16()
        c["bias_v"] = randn(E) * (0.05 if c["score"] == "sigmoid" else 0.5 / E) if c["bias"] else None
        c["w13"], c["w13_sf"] = _experts_weights(E, 2 * I, H, gen)
        c["w2"], c["w2_sf"] = _experts_weights(E, H, I, gen)
    return c


# ------------------------------------------------------------- plain forms --

def _plain_lora(s):
    T, K, N, R, L = s["T"], s["K"], s["N"], s["R"], s["L"]
    # every token by every adapter, and then only its own one's part kept
    u = (s["x"].float() @ s["a"].float().reshape(L * R, K).T).reshape(T, L, R)
    keep = (s["ids"][:, None] == torch.arange(L, device=u.device))[:, :, None]
    if s["ranks"] is not None:
        keep = keep & (torch.arange(R, device=u.device) < s["ranks"][:, None])[None]
    u = torch.where(keep, u * s["scales"][:, None], 0.0).reshape(T, L * R)
    delta = u @ s["b"].float().permute(0, 2, 1).reshape(L * R, N)
    return {"c": (s["base"].float() + delta).to(s["base"].dtype)}


def _heads(s):
    T, Hq, Hk, D = s["T"], s["Hq"], s["Hk"], s["D"]
    q = s["qkv"][:, :Hq * D].unflatten(1, (Hq, D))
    k = s["qkv"][:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    return q, k


def _plain_qk(s):
    rot, half = s["rot"], s["rot"] // 2
    t = s["table"][s["pos"].long()]
    cos, sin = t[:, None, :half], t[:, None, half:]
    out = {}
    for name, x, w in zip("qk", _heads(s), (s["wq"], s["wk"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        if s["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out[name] = torch.cat([turned, y[..., rot:]], -1).to(x.dtype)
    return out


def _mxfp8_exponents(top):
    """Exponent of the smallest power of two that leaves a largest magnitude `top` at or below 448."""
    m, x = torch.frexp(top)
    return torch.where(m > 0, x - 9 + (m > 0.875), torch.full_like(x, -127)).clamp(-127, 127)


def _as_mxfp8(y):
    """The values that fp32 [M, K] takes in MXFP8: E4M3 with one power-of-two scale for 32 of them."""
    M, K = y.shape
    b = y.reshape(M, K // 32, 32)
    e = _mxfp8_exponents(b.abs().amax(-1))[..., None]
    return ((b * _pow2(-e)).to(torch.float8_e4m3fn).float() * _pow2(e)).reshape(M, K)


def _from_mxfp4(q, sf_blocked, N, K):
    """fp32 [n, N, K] of n packed matrices."""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    val = torch.cat([mag, -mag])
    byte = torch.arange(256, device=q.device)
    w = torch.stack([val[byte & 15], val[byte >> 4]], -1)[q.long()].reshape(-1, N, K // 32, 32)
    return (w * _pow2(_unblocked(sf_blocked, N, K // 32).to(torch.int32) - 127)[..., None]).reshape(-1, N, K)


def _stable_top(v, k):
    return torch.sort(v, dim=-1, descending=True, stable=True)[1][..., :k]


def _plain_route(s, z):
    # 64 bits: two experts' scores may lie next to each other
    T, E = z.shape
    score = torch.softmax(z, -1) if s["score"] == "softmax" else torch.sigmoid(z)
    choice = score if s["bias_v"] is None else score + s["bias_v"].double()
    if s["groups"] > 1:
        G = s["groups"]
        by_group = choice.reshape(T, G, E // G)
        top = torch.sort(by_group, dim=-1, descending=True)[0][..., :s["group_top"]].sum(-1)
        keep = torch.zeros((T, G), dtype=torch.bool, device=z.device)
        keep.scatter_(1, _stable_top(top, s["topk_groups"]), True)
        choice = by_group.masked_fill(~keep[..., None], -math.inf).reshape(T, E)
    ids = _stable_top(choice, s["k"])
    w = torch.gather(score, 1, ids)
    if s["renormalize"]:
        w = w / (w.sum(-1, keepdim=True) + 1e-20)
    return ids, (w * s["scale"]).float()


def _plain_layer(s):
    T, E, k, H, I = s["T"], s["E"], s["k"], s["H"], s["I"]
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).bfloat16()
    hd = h.double()
    y = hd * torch.rsqrt(hd.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
    ids, w = _plain_route(s, y @ s["router"].double().T)
    x = _as_mxfp8(y.float())
    # every token by every expert that some token may choose, where that is less than a set of matrices a choice
    if T * k <= E:
        pick, rows, place = ids.reshape(-1), x.repeat_interleave(k, 0)[:, None, :], None
    else:
        pick, rows, place = torch.arange(E, device=x.device), x[None].expand(E, T, H), ids
    a = torch.bmm(rows, _from_mxfp4(s["w13"][pick], s["w13_sf"][pick], 2 * I, H).transpose(1, 2))
    g, u = a[..., :I], a[..., I:]
    act = g / (1 + torch.exp(-g)) * u
    act = _as_mxfp8(act.reshape(-1, I)).reshape(act.shape)
    r = torch.bmm(act, _from_mxfp4(s["w2"][pick], s["w2_sf"][pick], H, I).transpose(1, 2))
    if place is None:
        r = r.reshape(T, k, H)
    else:
        r = r[place, torch.arange(T, device=x.device)[:, None]]
    return {"out": (r * w[..., None]).sum(1).bfloat16(), "h": h, "ids": ids.to(torch.int32), "weights": w}


# ------------------------------------------------------------------- calls --

def _own(s):
    from block_scaled_fp4_mxfp4_gb300 import mxfp4 as mx

    if s["op"] == "lora":
        if "workspace" not in s:
            # kept by a user's program for all its projections
            s["workspace"] = mx.lora_workspace(s["T"], s["K"], s["R"], s["L"])
        return {"c": mx.lora_add(s["base"], s["x"], s["a"], s["b"], s["ids"], scales=s["scales"], ranks=s["ranks"],
                                 workspace=s["workspace"])}
    if s["op"] == "qk":
        q, k = mx.qk_norm_rope(*_heads(s), s["table"], s["pos"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                               interleaved=s["interleaved"])
        return {"q": q, "k": k}
    if "workspace" not in s:
        # kept by a user's program for all its layers
        s["workspace"] = mx.moe_layer_workspace(s["T"], s["k"], s["E"], s["H"], s["I"])
    out, h, ids, w = mx.mxfp4_moe_layer(
        s["x"], s["weight"], s["router"], s["w13"], s["w13_sf"], s["w2"], s["w2_sf"], s["k"], eps=EPS, residual=s["res"],
        bias=s["bias_v"], score=s["score"], groups=s["groups"], topk_groups=s["topk_groups"], group_top=s["group_top"],
        renormalize=s["renormalize"], scale=s["scale"], workspace=s["workspace"])
    return {"out": out, "h": h, "ids": ids, "weights": w}


def run(state):
    if own:
        return _own(state)
    return {"lora": _plain_lora, "qk": _plain_qk, "layer": _plain_layer}[state["op"]](state)


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "lora":
        K, N, R, L = c["K"], c["N"], c["R"], c["L"]
        have = 1 - c["none"]
        used = L * have * (1 - (1 - 1 / L) ** T) if c["mix"] == "runs" else min(T, L) * have
        rank = (R + 1) / 2 if c["ragged"] else R
        return {"bytes": int(used * rank * (K + N) * 2 + T * (have * K * 2 + N * 4 + 4)),
                "flops": int(2 * T * have * rank * (K + N))}
    if c["op"] == "qk":
        n = T * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": n * 4 + T * (c["rot"] * 4 + 4), "flops": n * (8 if c["norm"] else 3)}
    E, k, H, I = c["E"], c["k"], c["H"], c["I"]
    active = E * (1 - (1 - k / E) ** T)      # experts that some token chooses
    weights = active * 3 * H * I * (0.5 + 1 / 32)
    return {"bytes": int(weights + E * H * 2 + H * 2 + T * H * 2 * (3 + c["residual"]) + T * k * 8),
            "flops": int(6 * T * k * H * I + 2 * T * E * H)}


# ------------------------------------------------------------------- exact --

def _exact_fp4(q, sf, N, K):
    """float64 [N, K] of one packed matrix."""
    v = torch.stack([q & 15, q >> 4], -1).reshape(N, K)
    m = (v & 7).double()
    mag = torch.where(m < 5, m / 2, 2 * m - 8)
    mag = torch.where(m == 5, torch.full_like(mag, 3.0), mag)
    r = torch.arange(N, device=q.device)[:, None]
    c = torch.arange(K // 32, device=q.device)[None, :]
    at = ((r // 128) * (-(-(K // 32) // 4)) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    return torch.where(v >= 8, -mag, mag) * torch.exp2(sf[at].double() - 127).repeat_interleave(32, 1)


def _exact_mxfp8(y):
    """The MXFP8 values of float64 [M, K]."""
    b = y.reshape(y.shape[0], -1, 32)
    top = b.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    s = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(-127, 127))[..., None]
    v = b / s
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * s).reshape(y.shape)


def exact(case, seed):
    s = prepare(case, seed)
    T = s["T"]
    if s["op"] == "lora":
        c = s["base"].double()
        for a in range(s["L"]):
            tok = torch.nonzero(s["ids"] == a).flatten()
            r = s["R"] if s["ranks"] is None else int(s["ranks"][a])
            u = s["x"][tok].double() @ s["a"][a, :r].double().T
            c[tok] += float(s["scales"][a]) * (u @ s["b"][a, :, :r].double().T)
        return {"c": c}
    if s["op"] == "qk":
        rot, D = s["rot"], s["D"]
        lo = torch.arange(0, rot, 2) if s["interleaved"] else torch.arange(rot // 2)
        hi = lo + 1 if s["interleaved"] else lo + rot // 2
        angle = s["table"].double()[s["pos"].long()][:, None, :]
        out, at = {}, 0
        for name, n, w in (("q", s["Hq"], s["wq"]), ("k", s["Hk"], s["wk"])):
            y = s["qkv"][:, at:at + n * D].double().reshape(T, n, D)
            at += n * D
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * w.double()
            z = y.clone()
            z[..., lo] = y[..., lo] * angle[..., :rot // 2] - y[..., hi] * angle[..., rot // 2:]
            z[..., hi] = y[..., hi] * angle[..., :rot // 2] + y[..., lo] * angle[..., rot // 2:]
            out[name] = z
        return out
    E, k, H, I = s["E"], s["k"], s["H"], s["I"]
    h = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
    # the norm is of the sum as it is kept
    kept = h.bfloat16().double()
    y = kept / torch.sqrt((kept * kept).sum(-1, keepdim=True) / H + EPS) * s["weight"].double()
    z = torch.einsum("th,eh->te", y, s["router"].double())
    if s["score"] == "softmax":
        p = torch.exp(z - z.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    c = p.clone() if s["bias_v"] is None else p + s["bias_v"].double()
    if s["groups"] > 1:
        n = E // s["groups"]
        c = c.reshape(T, s["groups"], n)
        best = c.topk(min(s["group_top"], n), dim=-1)[0].sum(-1)
        order = torch.argsort(-best, dim=-1, stable=True)
        c[torch.arange(T, device=z.device)[:, None], order[:, s["topk_groups"]:]] = -math.inf
        c = c.reshape(T, E)
    ids = torch.argsort(-c, dim=-1, stable=True)[:, :k]
    w = p[torch.arange(T, device=z.device)[:, None], ids]
    if s["renormalize"]:
        w = w / (w.sum(-1, keepdim=True) + 1e-20)
    w = w * s["scale"]
    x = _exact_mxfp8(y)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(tok):
            continue
        a = x[tok] @ _exact_fp4(s["w13"][e], s["w13_sf"][e], 2 * I, H).T
        g, u = a[:, :I], a[:, I:]
        act = _exact_mxfp8(g * torch.sigmoid(g) * u)
        out.index_add_(0, tok, (act @ _exact_fp4(s["w2"][e], s["w2_sf"][e], H, I).T) * w[tok, slot][:, None])
    return {"out": out, "h": h, "ids": ids.to(torch.int32), "weights": w}
