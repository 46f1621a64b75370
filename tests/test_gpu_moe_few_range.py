"""The mixture-of-experts layer of few tokens over its whole range: rows of any finite size, beside one another, and an eps
of any size."""
import pytest
import torch

import moe_ref

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("block_scaled_fp4_mxfp4_gb300.mxfp4")
from test_gpu_moe_few import call, check, make  # noqa: E402


@pytest.mark.parametrize("T,E,k,H,I", [(1, 6, 3, 1024, 128), (5, 6, 3, 4224, 128), (16, 40, 4, 256, 256), (3, 511, 8, 384, 128)])
@pytest.mark.parametrize("power", [51, 58, 64, 100, 120, -60, -64, -100, -118])
def test_rows_whose_squares_leave_fp32(T, E, k, H, I, power):
    s = make(T, E, H, I)
    s["x"], s["res"] = s["x"] * 2.0 ** power, s["res"] * 2.0 ** power
    check(s, call(s, k, eps=0.0), k, eps=0.0)
    if power > 0:
        check(s, call(s, k), k)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_of_all_sizes_beside_one_another(score):
    """Each is what it is alone, the ordinary ones among them; one value far above the others of its row; zeros."""
    s = make(9, 24, 512, 256)
    ordinary = call(s, 3, score=score)
    for t, power in ((1, 60), (2, 110), (4, -70), (5, -120)):
        s["x"][t], s["res"][t] = s["x"][t] * 2.0 ** power, s["res"][t] * 2.0 ** power
    s["x"][6], s["res"][6] = 0, 0
    s["x"][7, 100], s["res"][7, 100] = 2.0 ** 126, 2.0 ** 126
    for eps in (0.0, 1e-6):
        how = dict(eps=eps, score=score)
        got = call(s, 3, **how)
        check(s, got, 3, **how)
        for t in range(9):
            alone = call(dict(s, x=s["x"][t:t + 1], res=s["res"][t:t + 1]), 3, **how)
            assert all(torch.equal(a, b[t:t + 1]) for a, b in zip(alone, got))
    for t in (0, 3, 8):
        assert all(torch.equal(a[t], b[t]) for a, b in zip(ordinary, got))


@pytest.mark.parametrize("power", [0, 60, -40])
def test_an_eps_next_to_the_largest_number(power):
    """K eps leaves fp32, or is far above the row's squares."""
    s = make(4, 8, 1024, 128)
    s["x"], s["res"] = s["x"] * 2.0 ** power, s["res"] * 2.0 ** power
    for eps in (2.0 ** 127, 1e30, 1e8):
        check(s, call(s, 2, eps=eps), 2, eps=eps)


def test_a_row_that_is_not_finite_beside_a_row_of_any_size():
    s = make(4, 12, 256, 128)
    s["x"][0], s["res"][0] = s["x"][0] * 2.0 ** 100, s["res"][0] * 2.0 ** 100
    want = call(s, 3)
    s["x"][1, 17], s["x"][2, 3] = float("nan"), float("-inf")
    got = call(s, 3)
    assert all(torch.equal(a[[0, 3]], b[[0, 3]]) for a, b in zip(got, want))
    assert not bool(torch.isfinite(got[0][1:3]).any())
    assert int(got[2].min()) >= 0 and int(got[2].max()) < 12
