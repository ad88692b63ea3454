"""A row that sees one key has that key's weight of 1 whatever its score: out is the key's value, and its gradient does not
reach the score, so dq of the row is 0 and it adds nothing to dk."""
import pytest
import torch

from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import BF16, FP16, cu_of, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,K,D", [(6, 2, 64), (1, 1, 8), (4, 1, 96), (8, 8, 128)])
@pytest.mark.parametrize("n", [1, 40])
def test_sequences_of_one_token(n, H, K, D, causal, dtype):
    lens = [1, 0] * n
    q, k, v, dout = pack(lens, 3, H, K, D, dtype, scale=3.0)
    cu = cu_of(lens)
    op = layers.PackedAttention(H, K, D, causal=causal)
    out, lse = op.forward(q, k, v, cu)
    assert torch.equal(out[:n], v[:n].repeat_interleave(H // K, 1))
    dq_, dk, dv = op.backward(dout, q, k, v, out, lse, cu)
    op.check_status()
    assert not dq_.any() and not dk.any()
    want = dout[:n].double().view(n, K, H // K, D).sum(2)
    u = torch.finfo(dtype).eps / 2            # P and the result are rounded
    assert ((dv[:n].double() - want).abs() <= 2 * u * dout[:n].double().abs().view(n, K, H // K, D).sum(2) + 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
def test_first_causal_row(D, dtype):
    lens = [300, 5, 129, 2300]
    q, k, v, dout = pack(lens, 0, 2, 1, D, dtype, scale=3.0)
    cu = cu_of(lens)
    op = layers.PackedAttention(2, 1, D)
    out, lse = op.forward(q, k, v, cu)
    first = cu[:-1].long()
    assert torch.equal(out[first], v[first].repeat_interleave(2, 1))
    dout[:] = torch.where(torch.isin(torch.arange(sum(lens), device=cu.device), first)[:, None, None], dout, 0)
    dq_, dk, _ = op.backward(dout, q, k, v, out, lse, cu)
    op.check_status()
    assert not dq_.any() and not dk.any()     # no other row has a gradient
