"""Attention in every way its kernels are launched: blocks that go on from tile to tile, in turn and in the order of their
work, narrow and wide heads, and clusters that share a tile, against the 64-bit definition; and the same bits again."""
import math

import pytest
import torch

import block_reference as ref
from block_regimes import CASES, ways
from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import cu_of, pack, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


@pytest.mark.parametrize("lens,tail,H,K,D,dtype,causal,want", CASES)
def test_attention_in_every_way(lens, tail, H, K, D, dtype, causal, want):
    assert ways(lens, tail, H, K, D, dtype, causal, torch.cuda.get_device_properties(0).multi_processor_count) == want
    q, k, v, dout = pack(lens, tail, H, K, D, dtype)
    cu, held = cu_of(lens), sum(lens)
    op = layers.PackedAttention(H, K, D, causal=causal)

    def both():
        out, lse = op.forward(q, k, v, cu)
        return (out, lse, *op.backward(dout, q, k, v, out, lse, cu))

    got = both()
    op.check_status()
    exact = ref.attention(q, k, v, lens, causal, op.scale, dout)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), got):
        within(x, *exact[name], name)
    assert (got[1][:, held:] == -math.inf).all() and not any(got[i][held:].any() for i in (0, 2, 3, 4))
    for _ in range(3):
        for x, y in zip(got, both()):
            assert torch.equal(x, y)
    op.check_status()
