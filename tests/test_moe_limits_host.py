"""The sizes that the experts' products take: the workspace query and the call agree, without a GPU."""
import pytest
import torch

from block_scaled_fp4_mxfp4_gb300 import build as libbuild

libbuild.build()
from block_scaled_fp4_mxfp4_gb300 import mxfp4 as mx  # noqa: E402

SHAPE, NO_DEVICE = 2, 7

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="calls with stand-in addresses")


def call(T, k, E, H, I, ldx):
    return mx.lib().mxfp4_moe_experts(256, ldx, 256, 256, 256, 256, 256, 256, 256, 256, H, T, k, E, H, I, 256, 1 << 62,
                                      None)


@pytest.mark.parametrize("T,k,E,H,I", [
    (1, 1, 1, 128, 128), (1 << 20, 8, 8, 4096, 16384), ((1 << 30) - 1, 1, 1, 128, 128), (1 << 30, 1, 1, 128, 128),
    (1 << 25, 32, 1, 128, 128), (100, 2, 4, 1 << 20, 128), (100, 2, 4, (1 << 20) + 128, 128), (100, 2, 4, 128, 1 << 20),
    (100, 2, 4, 128, (1 << 20) + 128), (100, 2, 512, 128, 1 << 20), (100, 2, 511, 128, 1 << 20),
    (1 << 25, 8, 1, 128, 16384), (1 << 25, 8, 1, 32768, 128), (1 << 25, 8, 1, 128, 8192), (1 << 25, 8, 1, 16384, 128),
])
@pytest.mark.parametrize("wide", [False, True])
def test_query_and_call_agree(T, k, E, H, I, wide):
    """Rows of activations may lie any distance apart."""
    status = call(T, k, E, H, I, 1 << 40 if wide else H)
    assert status in (SHAPE, NO_DEVICE)
    assert (status == SHAPE) == (mx.moe_experts_workspace_bytes(T, k, E, H, I) == 0)
