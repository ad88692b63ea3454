"""Rows whose every visible key scores -inf, on the GPU: no weights, so an output of 0, an lse of -inf and no part in any
gradient; the other rows are as they are without them."""
import math

import pytest
import torch

from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import BF16, DEV, cu_of, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("n,gone", [(90, 40), (300, 140), (700, 300), (2300, 1100)])
@pytest.mark.parametrize("H,K", [(2, 1), (1, 1)])
def test_rows_that_see_only_minus_infinity(n, gone, H, K, D):
    """The first ``gone`` keys' scores overflow to -inf in fp32 (1e20 times -1e20), the others do not see that element;
    under the causal mask the first ``gone`` queries see no other keys.  For the rest the hidden keys have weights of 0.

    Tolerances: P and the stored output are each rounded to 8 bits (2^-8 together), and |out| <= max |v|; dv adds the
    rounding of P and of the result over the sum of |P dout|; dq and dk are checked to be finite and, where only hidden
    rows or keys enter, 0."""
    q, k, v, dout = (x.contiguous() for x in pack([n], 0, H, K, D, BF16))
    q[:, :, 0] = 1e20
    k[:, :, 0] = 0
    k[:gone, :, 0] = -1e20
    op = layers.PackedAttention(H, K, D)
    cu = cu_of([n])
    out, lse = op.forward(q, k, v, cu)
    assert not out[:gone].any() and (lse[:, :gone] == -math.inf).all()
    s = torch.einsum("thd,sd->hts", q[gone:].double(), k[gone:, 0].double()) * op.scale
    s = s.masked_fill(torch.ones(n - gone, n - gone, dtype=torch.bool, device=DEV).triu(1), -math.inf)
    p = s.softmax(-1)
    exact = torch.einsum("hts,sd->thd", p, v[gone:, 0].double())
    assert ((out[gone:].double() - exact).abs() <= 2 * 2.0 ** -8 * v.abs().max().double()).all()
    assert ((lse[:, gone:].double() - s.logsumexp(-1)).abs() <= 1e-4).all()

    dq_, dk, dv = op.backward(dout, q, k, v, out, lse, cu)
    op.check_status()
    assert all(x.isfinite().all() for x in (dq_, dk, dv))
    assert not dq_[:gone].any() and not dk[:gone].any() and not dv[:gone].any()
    exact = torch.einsum("hts,thd->sd", p, dout[gone:].double())
    size = torch.einsum("hts,thd->sd", p, dout[gone:].double().abs())
    assert ((dv[gone:, 0].double() - exact).abs() <= 2 * 2.0 ** -8 * size + 1e-6).all()


@pytest.mark.parametrize("D", [64, 128])
def test_a_sequence_without_any_weight(D):
    """Both ways, every score -inf: zeros; its neighbours are untouched."""
    lens = [60, 200, 130]
    q, k, v, dout = (x.contiguous() for x in pack(lens, 0, 2, 1, D, BF16))
    cu = cu_of(lens)
    op = layers.PackedAttention(2, 1, D, causal=False)

    def run():
        out, lse = op.forward(q, k, v, cu)
        return (out, lse.t(), *op.backward(dout, q, k, v, out, lse, cu))

    clean = run()
    q[60:260, :, 0], k[60:260, :, 0] = 1e20, -1e20
    got = run()
    op.check_status()
    for a, b in zip(clean, got):
        assert torch.equal(a[:60], b[:60]) and torch.equal(a[260:], b[260:])
    assert (got[1][60:260] == -math.inf).all()
    for i in (0, 2, 3, 4):
        assert not got[i][60:260].any()
