"""Attention kernels whose waits run out: the status says so, the call returns, and the next call is right.

The limit of a wait is set to one cycle, so that whatever a block's roles still have to wait for runs out: nothing is
missing, and every role gives up and returns.  (Waits that are over at once pass, so single blocks may still finish.)"""
import pytest
import torch

from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import BF16, FP16, cu_of, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


@pytest.fixture
def short():
    """Calls with the short limit; the default comes back whatever happens."""
    def run(call):
        dq.dq_attention_wait_limit(1)
        try:
            return call()
        finally:
            dq.dq_attention_wait_limit(0)
    yield run
    dq.dq_attention_wait_limit(0)


CASES = [
    # lens, heads, kv heads, dim, dtype, causal
    ([2048], 4, 2, 64, BF16, False),                     # a block a tile
    ([2048, 1500], 8, 2, 128, BF16, True),
    ([900, 517, 640, 1300], 16, 8, 128, FP16, True),     # several tiles a block
    ([900, 517, 640, 1300], 16, 8, 64, BF16, False),
    ([4100], 1, 1, 128, BF16, True),                     # blocks share a tile
    ([4100], 1, 1, 64, FP16, False),
]


@pytest.mark.parametrize("lens,H,K,D,dtype,causal", CASES)
def test_waits_that_run_out(lens, H, K, D, dtype, causal, short):
    q, k, v, dout = pack(lens, 130, H, K, D, dtype)
    cu = cu_of(lens)
    op = layers.PackedAttention(H, K, D, causal=causal)

    def forward():
        return op.forward(q, k, v, cu)

    def backward():
        return op.backward(dout, q, k, v, *good[:2], cu)

    good = forward()
    good = (*good, *backward())
    op.check_status()
    for _ in range(3):
        for call, want in ((forward, good[:2]), (backward, good[2:])):
            short(call)
            torch.cuda.synchronize()
            with pytest.raises(RuntimeError, match="status 2"):
                op.check_status()
            op.check_status()                            # read once, then clear
            for a, b in zip(call(), want):
                assert torch.equal(a, b)
            op.check_status()


def test_the_limit_is_checked():
    for bad in (-1, 8_000_000_001):
        with pytest.raises(dq.DQError) as e:
            dq.dq_attention_wait_limit(bad)
        assert e.value.status == dq.DQ_ERR_INVALID_ARG
