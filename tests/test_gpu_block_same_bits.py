"""Narrow heads' backward pass with several tiles a block: the same bits on every call, whichever warp is late."""

import pytest
import torch

import block_reference as ref
from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import BF16, FP16, cu_of, pack, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("lens,H,K,causal", [([900, 517, 0, 640, 1300, 1], 64, 32, True), ([700] * 5, 16, 16, False),
                                             ([3000, 2000], 2, 1, True)])
def test_backward_again_and_again(lens, H, K, causal, dtype):
    q, k, v, dout = pack(lens, 77, H, K, 64, dtype)
    cu = cu_of(lens)
    op = layers.PackedAttention(H, K, 64, causal=causal)
    out, lse = op.forward(q, k, v, cu)
    first = op.backward(dout, q, k, v, out, lse, cu)
    exact = ref.attention(q, k, v, lens, causal, op.scale, dout)
    for name, x in zip(("dq", "dk", "dv"), first):
        within(x, *exact[name], name)
    for _ in range(20):
        for x, y in zip(first, op.backward(dout, q, k, v, out, lse, cu)):
            assert torch.equal(x, y)
    op.check_status()
