"""Low-rank adapters beside a projection against their definition in 64 bits: sizes that end inside tiles, adapters of
every rank, tokens without one, in place and beside, strided rows, streams and graphs."""
import pytest
import torch

import layer_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")


def case(T, K, N, R, L, dtype=torch.bfloat16, ragged=False, seed=0, none=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed + T)
    rn = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x, base = rn(T, K).bfloat16(), rn(T, N).to(dtype)
    a, b = (rn(L, R, K) * K ** -0.5).bfloat16(), rn(L, N, R).bfloat16()
    ids = torch.randint(0, L, (T,), device="cuda", generator=gen)
    ids = torch.where(torch.rand(T, device="cuda", generator=gen) < none, -1, ids).to(torch.int32)
    scales = rn(L)
    ranks = torch.randint(0, R + 1, (L,), device="cuda", generator=gen).to(torch.int32) if ragged else None
    return base, x, a, b, ids, scales, ranks


def check(c, ref):
    want, bound = ref
    worst = float(((c.double() - want).abs() / bound).max())
    assert worst <= 1.0, worst
    assert mx.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,R,L", [
    (1, 8, 8, 8, 1), (1, 7168, 2112, 16, 4), (3, 72, 40, 24, 2), (8, 520, 264, 8, 64), (9, 256, 96, 40, 1),
    (16, 1024, 512, 32, 3), (33, 64, 128, 64, 2), (64, 136, 200, 48, 5), (65, 136, 200, 48, 5), (130, 2048, 72, 16, 1),
    (200, 264, 1000, 72, 7), (333, 512, 328, 128, 300), (700, 96, 64, 256, 3), (2500, 64, 40, 8, 4096),
])
def test_against_the_definition(T, K, N, R, L, dtype):
    if dtype is torch.float16 and L * R * (K + N) > 1 << 26:
        pytest.skip("covered in bf16")
    args = case(T, K, N, R, L, dtype, ragged=T % 2 == 1)
    base, x, a, b, ids, scales, ranks = args
    c = mx.lora_add(base, x, a, b, ids, scales, ranks)
    assert c.dtype is dtype and c.data_ptr() != base.data_ptr()
    check(c, layer_ref.lora(*args))
    # a token without an adapter keeps its row bit for bit
    assert torch.equal(c[ids < 0], base[ids < 0])
    # in place, and again: the same bits
    inplace = base.clone()
    assert mx.lora_add(inplace, x, a, b, ids, scales, ranks, C=inplace) is inplace
    assert torch.equal(inplace[ids >= 0], c[ids >= 0]) and torch.equal(inplace[ids < 0], base[ids < 0])


@pytest.mark.parametrize("T", [5, 150])
def test_what_lies_beyond_a_rank_is_not_used(T):
    args = case(T, 128, 96, 32, 4, ragged=True, none=0.0)
    base, x, a, b, ids, scales, ranks = args
    ranks.copy_(torch.tensor([0, 1, 17, 32]))
    want = mx.lora_add(base, x, a, b, ids, scales, ranks)
    check(want, layer_ref.lora(*args))
    for i, r in enumerate(ranks.tolist()):
        a[i, r:] = float("nan")
        b[i, :, r:] = float("inf")
    assert torch.equal(mx.lora_add(base, x, a, b, ids, scales, ranks), want)
    # ranks out of their range are taken as the nearest end of it
    ranks.copy_(torch.tensor([-5, 1, 17, 99]))
    assert torch.equal(mx.lora_add(base, x, a, b, ids, scales, ranks), want)


@pytest.mark.parametrize("T", [40, 300])
def test_no_token_has_an_adapter(T):
    base, x, a, b, ids, scales, ranks = case(T, 64, 64, 8, 2)
    ids.copy_(torch.where(torch.arange(T, device="cuda") % 2 == 0, -1, 2))
    c = mx.lora_add(base, x, a, b, ids)
    assert torch.equal(c, base)
    before = base.clone()
    mx.lora_add(base, x, a, b, ids, C=base)
    assert torch.equal(base, before)


@pytest.mark.parametrize("T", [20, 200])
def test_a_token_does_not_depend_on_its_neighbours(T):
    """NaN and infinity in one token's row, or in another adapter, stay there."""
    args = case(T, 256, 128, 16, 3, none=0.0)
    base, x, a, b, ids, scales, _ = args
    want = mx.lora_add(base, x, a, b, ids, scales)
    x2, a2 = x.clone(), a.clone()
    x2[7] = float("nan")
    x2[11, 5] = float("inf")
    a2[2] = float("inf")
    got = mx.lora_add(base, x2, a2, b, ids, scales)
    clean = ids != 2
    clean[[7, 11]] = False
    assert bool(clean.any()) and torch.equal(got[clean], want[clean])
    assert bool(torch.isnan(got[7]).all())
    order = torch.randperm(T, device="cuda")
    assert torch.equal(mx.lora_add(base[order].contiguous(), x[order].contiguous(), a, b, ids[order].contiguous(), scales),
                       want[order])


def test_strided_rows_are_read_and_written_in_place_only():
    base, x, a, b, ids, scales, _ = case(90, 128, 64, 16, 3)
    wide_x = torch.full((90, 200), float("nan"), device="cuda").bfloat16()
    wide_x[:, 8:136] = x
    wide = torch.full((90, 96), 7.0, device="cuda").bfloat16()
    wide[:, 16:80] = base
    out = torch.full((91, 104), 3.0, device="cuda").bfloat16()
    mx.lora_add(wide[:, 16:80], wide_x[:, 8:136], a, b, ids, scales, C=out[:90, 24:88])
    assert torch.equal(out[:90, 24:88], mx.lora_add(base, x, a, b, ids, scales))
    out[:90, 24:88] = 3.0
    assert bool((out == 3.0).all())


@pytest.mark.parametrize("T", [16, 500])
def test_streams_and_graphs(T):
    """On a side stream, captured and replayed on new inputs, and two captured calls with workspaces of their own."""
    base, x, a, b, ids, scales, _ = case(T, 512, 256, 32, 5)
    ws = [mx.lora_workspace(T, 512, 32, 5).fill_(0xFF) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = mx.lora_add(base, x, a, b, ids, scales, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, mx.lora_add(base, x, a, b, ids, scales, workspace=ws[0]))
    graphs, outs = [], []
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.lora_add(base, x, a, b, ids, scales, workspace=w))
        graphs.append(g)
    x.mul_(2)
    ids.copy_(ids.flip(0))
    for g in graphs:
        g.replay()
    fresh = mx.lora_add(base, x, a, b, ids, scales)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], fresh) and torch.equal(outs[1], fresh) and not torch.equal(fresh, first)


def test_offsets_beyond_32_bits():
    """Adapters whose elements lie more than 2^31 apart."""
    L, R, K, N = 20, 256, 1 << 19, 64
    a = torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda")
    b = torch.randn((L, N, R), device="cuda").bfloat16()
    a[L - 1, :, K - 600:] = torch.randn((R, 600), device="cuda").bfloat16()
    x = torch.randn((2, K), device="cuda").bfloat16()
    base = torch.zeros((2, N), device="cuda").bfloat16()
    ids = torch.tensor([L - 1, 0], dtype=torch.int32, device="cuda")
    c = mx.lora_add(base, x, a, b, ids)
    u = x[0, K - 600:].double() @ a[L - 1, :, K - 600:].double().T
    want = u @ b[L - 1].double().T
    assert float((c[0].double() - want).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    assert not c[1].any()


def test_zero_tokens():
    base, x, a, b, ids, scales, _ = case(4, 64, 64, 8, 2)
    assert mx.lora_add(base[:0], x[:0], a, b, ids[:0]).shape == (0, 64)


def test_refusals_of_the_binding():
    base, x, a, b, ids, scales, _ = case(4, 64, 64, 8, 2)
    with pytest.raises(ValueError):
        mx.lora_add(base.float(), x, a, b, ids)
    with pytest.raises(ValueError):
        mx.lora_add(base, x.half(), a, b, ids)
    with pytest.raises(ValueError):
        mx.lora_add(base, x, a, b.transpose(1, 2), ids)
    with pytest.raises(ValueError):
        mx.lora_add(base, x, a, b, ids.long())
    with pytest.raises(ValueError):
        mx.lora_add(base, x, a, b, ids[:3])
    with pytest.raises(ValueError):
        mx.lora_add(base, x, a, b, ids, scales[:1])
    with pytest.raises(ValueError):
        mx.lora_add(base, x, a, b, ids, C=base.cpu())
    with pytest.raises(mx.Mxfp4Error):
        mx.lora_add(base, x, a, b, ids, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mx.Mxfp4Error):
        mx.lora_add(base, x[:, :60], a[:, :, :60].contiguous(), b, ids)


@pytest.mark.parametrize("T", [16, 130])
@pytest.mark.parametrize("K", [8, 56, 72, 16392])
def test_lengths_of_the_sum_that_leave_splits_short_or_empty(T, K):
    args = case(T, K, 48, 24, 2, none=0.0)
    base, x, a, b, ids, scales, ranks = args
    check(mx.lora_add(base, x, a, b, ids, scales, ranks), layer_ref.lora(*args))


@pytest.mark.parametrize("T", [64, 65, 127, 128, 129, 193, 257])
@pytest.mark.parametrize("R", [8, 120, 128, 136, 256])
def test_one_adapter_for_all_tokens(T, R):
    args = case(T, 200, 72, R, 1, none=0.0)
    base, x, a, b, ids, scales, ranks = args
    check(mx.lora_add(base, x, a, b, ids, scales, ranks), layer_ref.lora(*args))


def test_waits_that_run_out_end_the_call_and_are_reported():
    """Large enough that some wait is longer than the limit: a few hundred tokens in L2 often pass within one nanosecond."""
    base, x, a, b, ids, scales, _ = case(4096, 7168, 64, 64, 2, none=0.0)
    want = mx.lora_add(base, x, a, b, ids, scales)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0
    mx.set_wait_limit_ns(1)
    try:
        mx.lora_add(base, x, a, b, ids, scales)
        torch.cuda.synchronize()
    finally:
        mx.set_wait_limit_ns(0)
    assert 80 < mx.get_device_error() < 96
    again = mx.lora_add(base, x, a, b, ids, scales)
    torch.cuda.synchronize()
    assert mx.get_device_error() == 0 and torch.equal(again, want)


def test_two_graphs_that_share_a_workspace():
    cases = [case(40, 256, 128, 32, 5), case(500, 512, 64, 16, 9)]
    size = max(mx.lora_workspace_bytes(40, 256, 32, 5), mx.lora_workspace_bytes(500, 512, 16, 9))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    want = [mx.lora_add(*c) for c in cases]
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = mx.lora_add(*c, workspace=ws)
        graphs.append((g, o))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graphs[i][0].replay()
        assert torch.equal(graphs[i][1], want[i])
    assert mx.get_device_error() == 0


@pytest.mark.parametrize("T", [16, 300, 3000])
def test_two_streams_at_once(T):
    cases = [case(T, 1024, 512, 32, 5, seed=i) for i in range(2)]
    want = [mx.lora_add(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(mx.lora_add(*cases[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])
    assert mx.get_device_error() == 0


@pytest.mark.parametrize("T", [8192, 8193, 20011])
def test_long_batches_of_runs_and_of_mixed_ids(T):
    """Prompts whose tokens share an adapter, tokens without one, mixed tokens, and a run that ends inside a warp's ids."""
    base, x, a, b, ids, scales, ranks = case(T, 64, 40, 16, 5, ragged=True)
    ids[:3000], ids[5000:6000], ids[-2050:-7] = 2, -1, 4
    args = base, x, a, b, ids, scales, ranks
    c = mx.lora_add(*args)
    check(c, layer_ref.lora(*args))
    assert torch.equal(c[ids < 0], base[ids < 0])
    assert torch.equal(mx.lora_add(base, x, a, b, ids, scales, ranks, C=base), c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,R,L", [
    (300, 8, 8, 8, 1), (257, 136, 72, 40, 1), (700, 520, 200, 24, 2), (1100, 1096, 1000, 56, 3), (1500, 2056, 64, 64, 3),
    (2600, 4096, 328, 48, 5), (5000, 264, 136, 16, 6), (9000, 72, 264, 64, 40),
])
def test_batches_of_well_filled_tiles(T, K, N, R, L, dtype):
    """Ends of K, N and ranks inside a tile's steps, ragged ranks with NaN behind them, rows that are views, in place."""
    base, x, a, b, ids, scales, ranks = case(T, K, N, R, L, dtype, ragged=True)
    for l in range(L):
        a[l, int(ranks[l]):], b[l, :, int(ranks[l]):] = float("nan"), float("nan")
    want = layer_ref.lora(base, x, torch.nan_to_num(a), torch.nan_to_num(b), ids, scales, ranks)
    wide = torch.full((T, N + 24), 7.0, device="cuda").to(dtype)
    c, xs = wide[:, 8:8 + N], torch.cat([x, x[:, :8]], 1)[:, :K]
    assert mx.lora_add(base, xs, a, b, ids, scales, ranks, C=c) is c
    check(c, want)
    assert bool((wide[:, :8] == 7.0).all()) and bool((wide[:, 8 + N:] == 7.0).all())
    assert torch.equal(c[ids < 0], base[ids < 0])
    c.copy_(base)
    first = mx.lora_add(base, x, a, b, ids, scales, ranks)
    assert torch.equal(mx.lora_add(c, x, a, b, ids, scales, ranks, C=c), first)
    assert bool((wide[:, :8] == 7.0).all()) and bool((wide[:, 8 + N:] == 7.0).all())
    assert mx.get_device_error() == 0
