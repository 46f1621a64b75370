"""Outputs of qk_norm_rope whose strides make heads of different tokens share elements are refused, all others taken: the
check against a list of all elements' places. Without a GPU."""
import random

import pytest
import torch

from block_scaled_fp4_mxfp4_gb300 import build as libbuild

libbuild.build()
from block_scaled_fp4_mxfp4_gb300 import mxfp4 as mx  # noqa: E402

L = mx.lib()
INVALID, NO_DEVICE = 1, 7

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run")


def qk(T, H, D, st, sh, keys=False):
    """Status of a call whose queries (or keys) go to places st and sh apart."""
    q, k = ((0, 0, 0), (H, st, sh)) if keys else ((H, st, sh), (0, 0, 0))
    return L.qk_norm_rope(1 << 20, 8, 8, 1 << 20, 8, 8, None, None, None, None, 0, 0, 1e-6, T, q[0], k[0], D, 0, 0, 0,
                          1 << 30, q[1], q[2], 1 << 30, k[1], k[2], None)


def shared(T, H, D, st, sh):
    places = [t * st + h * sh for t in range(T) for h in range(H)]
    places.sort()
    return any(b - a < D for a, b in zip(places, places[1:]))


@pytest.mark.parametrize("T,H,D,st,sh,want", [
    (2, 2, 64, 64, 64, INVALID), (2, 2, 64, -64, 64, INVALID), (2, 2, 64, 128, 64, NO_DEVICE), (2, 2, 64, 64, 128, NO_DEVICE),
    (2, 2, 64, 64, -128, NO_DEVICE), (9, 4, 64, 192, 64, INVALID), (9, 4, 64, 256, 64, NO_DEVICE), (9, 4, 64, 64, 576, NO_DEVICE),
    (9, 4, 64, 64, 568, INVALID), (3, 2, 8, 16, 24, NO_DEVICE), (4, 2, 8, 16, 24, NO_DEVICE), (4, 3, 8, 16, 24, INVALID),
    (1, 3, 64, 0, 64, NO_DEVICE), (3, 1, 64, 64, 0, NO_DEVICE), (2, 1 << 20, 64, 64, 128, NO_DEVICE), (2, 1 << 20, 64, 64, 64, INVALID),
    (40000, 40000, 64, 64, 64 * 40000, NO_DEVICE), (40000, 40000, 64, 128 * 20001, 128, INVALID),
    (4, 4, 64, 1 << 61, 64, NO_DEVICE), (4, 4, 64, -(1 << 62), 1 << 61, INVALID),
])
def test_places_that_heads_share(T, H, D, st, sh, want):
    for keys in (False, True):
        assert qk(T, H, D, st, sh, keys) == want


def test_against_all_places():
    rng = random.Random(7)
    seen = set()
    for _ in range(4000):
        T, H, D = rng.randint(1, 7), rng.randint(1, 7), 8 * rng.randint(1, 4)
        st, sh = (8 * rng.randint(-16, 16) for _ in range(2))
        want = INVALID if shared(T, H, D, st, sh) else NO_DEVICE
        assert qk(T, H, D, st, sh) == want, (T, H, D, st, sh)
        seen.add((want, abs(st) >= H * abs(sh), abs(sh) >= T * abs(st)))
    assert len(seen) > 4
