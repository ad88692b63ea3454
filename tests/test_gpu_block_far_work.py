"""Long runs of empty sequences between tiles: a block that looks for its next tile keeps nobody waiting beyond a wait's
limit of about a second."""
import pytest
import torch

import block_reference as ref
from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import BF16, cu_of, pack, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


@pytest.mark.parametrize("n,D,H,front", [(200_000, 64, 4, False), (200_000, 128, 4, True), (6_000_000, 128, 32, False)])
def test_empty_sequences_between_tiles(n, D, H, front):
    """6 million empty sequences are 192 million blocks without a tile for 32 heads, which the dq kernel takes more than a
    second to pass over."""
    q, k, v, dout = pack([1024], 0, H, 1, D, BF16)
    cu = torch.zeros(n + 2, dtype=torch.int32, device="cuda")
    cu[1 if front else -1:] = 1024
    op = layers.PackedAttention(H, 1, D)
    out, lse = op.forward(q, k, v, cu)
    op.check_status()
    got = (out, lse, *op.backward(dout, q, k, v, out, lse, cu))
    op.check_status()
    exact = ref.attention(q, k, v, [1024], True, op.scale, dout)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), got):
        within(x, *exact[name], name)
