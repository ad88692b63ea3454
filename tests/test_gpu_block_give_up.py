"""Attention kernels whose waits run out: the status says so, the call returns, and the next call is right.

Under the self-test no wait waits, so that every role of a block gives up where it would have waited, with copies, products
and requests for work in flight.  (Waits that are over at once pass, so single blocks may still finish.)"""
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
    """Calls under the self-test, which ends with them whatever happens."""
    def run(call):
        dq.dq_attention_give_up_selftest(True)
        try:
            return call()
        finally:
            dq.dq_attention_give_up_selftest(False)
    yield run
    dq.dq_attention_give_up_selftest(False)


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


def test_the_status_of_a_call_on_another_stream(short):
    """check_status(stream=...) waits for that stream's calls; the current stream's need not have to."""
    q, k, v, _ = pack([4100], 0, 8, 8, 128, BF16)
    cu = cu_of([4100])
    op = layers.PackedAttention(8, 8, 128)
    op.forward(q, k, v, cu)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                op.forward(q, k, v, cu)                  # some milliseconds before the call that gives up
        short(lambda: op.forward(q, k, v, cu, stream=stream))
        with pytest.raises(RuntimeError, match="status 2"):
            op.check_status(stream=stream)
        op.check_status(stream=stream)
