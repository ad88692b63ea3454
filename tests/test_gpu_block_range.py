"""Attention gradients over fp16's whole range, and rows that see no finite score, on the GPU.

Bounds: those of block_reference, whose ``low`` term grants every weight and every dS an absolute rounding step.  With
fp16 that step is here taken from what the kernels hold: weights times 2^12 (rounded by at most 2^-25 / 2^12 = 2^-37), and
P (dP - delta) times 2^12 and a power of two F that brings |dP - delta| <= B = 2 |dout_i| max |v_j| (Cauchy; delta is a
mean of dP) to between 1/2 and 1, so that it is rounded by at most 2^-37 2 B = 2^-35 |dout_i| max |v_j|."""
import math

import pytest
import torch

import block_reference as ref
from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import BF16, DEV, FP16, cu_of, pack, within

pytestmark = pytest.mark.gpu
NAMES = ("out", "lse", "dq", "dk", "dv")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


def exact16(q, k, v, lens, causal, scale, dout):
    """ref.attention with the step described above; results' own storage keeps fp16's."""
    held = 2.0 ** -35 * max(1.0, dout.double().norm(dim=-1).max().item() * v.double().norm(dim=-1).max().item())
    step = ref.STEP[FP16]
    ref.STEP[FP16] = min(step, held)
    try:
        r = ref.attention(q, k, v, lens, causal, scale, dout)
    finally:
        ref.STEP[FP16] = step
    return {n: (x, b + step if n != "lse" else b) for n, (x, b) in r.items()}


def run(op, q, k, v, dout, cu):
    out, lse = op.forward(q, k, v, cu)
    got = (out, lse, *op.backward(dout, q, k, v, out, lse, cu))
    op.check_status()
    return got


SHAPES = [
    # lens, heads, kv heads, dim, causal
    ([100, 0, 1, 128], 2, 1, 64, True),          # one tile of keys
    ([1024], 2, 2, 64, True),
    ([700, 324], 2, 1, 128, False),
    ([513, 257], 3, 1, 80, True),
    ([2300], 1, 1, 128, True),                   # blocks share a tile's loop
    ([2300, 90], 1, 1, 40, False),
]


@pytest.mark.parametrize("lens,H,K,D,causal", SHAPES)
def test_small_gradients_fp16(lens, H, K, D, causal):
    """dout of 1e-5: P (dP - delta) lies below fp16's range while dq and dk do not (q and k are small and the scale is
    large, which multiplies both by 2^10)."""
    q, k, v, dout = pack(lens, 7, H, K, D, FP16)
    q, k, dout = (q * 2.0 ** -10).contiguous(), (k * 2.0 ** -10).contiguous(), (dout.float() * 1e-4).to(FP16)
    scale = 2.0 ** 20 / math.sqrt(D)
    op = layers.PackedAttention(H, K, D, causal=causal, scale=scale)
    got = run(op, q, k, v, dout, cu_of(lens))
    exact = exact16(q, k, v, lens, causal, scale, dout)
    for name, x in zip(NAMES, got):
        within(x, *exact[name], name)


@pytest.mark.parametrize("lens,H,K,D,causal", SHAPES)
def test_large_gradients_fp16(lens, H, K, D, causal):
    """dout of standard deviation 12,000: dP - delta passes 65,504, the gradients do not."""
    if H > K:
        H = K                                    # a shared head's dv would pass it
    q, k, v, dout = pack(lens, 7, H, K, D, FP16, seed=3)
    dout = (dout.float() * 1.2e5).clamp(-36000, 36000).to(FP16)
    op = layers.PackedAttention(H, K, D, causal=causal)
    got = run(op, q, k, v, dout, cu_of(lens))
    exact = exact16(q, k, v, lens, causal, op.scale, dout)
    for name, x in zip(NAMES, got):
        assert exact[name][0][exact[name][0] > -math.inf].abs().max() < 65504
        within(x, *exact[name], name)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_different_magnitude_fp16(D):
    """dq of a row has the accuracy of that row's own gradient, whatever the others' are."""
    lens = [600, 300]
    q, k, v, dout = pack(lens, 0, 2, 1, D, FP16)
    q, k = (q * 2.0 ** -10).contiguous(), (k * 2.0 ** -10).contiguous()
    scale = 2.0 ** 20 / math.sqrt(D)
    small = torch.arange(900, device=DEV) % 3 != 0
    dout = torch.where(small[:, None, None], dout.float() * 1e-4, dout.float() * 1e-1).to(FP16)
    op = layers.PackedAttention(2, 1, D, scale=scale)
    got = run(op, q, k, v, dout, cu_of(lens))
    for rows in (small, ~small):
        exact = exact16(q, k, v, lens, True, scale, torch.where(rows[:, None, None], dout, 0))
        within(got[2][rows], exact["dq"][0][rows], exact["dq"][1][rows], "dq")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bad", [math.nan, math.inf, 60000.0])
@pytest.mark.parametrize("D", [64, 128])
def test_sequences_are_apart_fp16(causal, bad, D):
    """What one sequence or the padding holds changes no bit of the others: not their factors either."""
    lens, tail = [170, 150, 390], 60
    q, k, v, dout = (x.contiguous() for x in pack(lens, tail, 4, 2, D, FP16))
    cu = cu_of(lens)
    op = layers.PackedAttention(4, 2, D, causal=causal)
    clean = run(op, q, k, v, dout, cu)
    for x in (q, k, v, dout):
        x[170:320] = bad
        x[710:] = bad
    dirty = run(op, q, k, v, dout, cu)
    for a, b, name in zip(clean, dirty, NAMES):
        if name == "lse":
            a, b = a.t(), b.t()
        assert torch.equal(a[:170], b[:170]) and torch.equal(a[320:], b[320:]), name


def test_no_gradient_fp16():
    """dout of zeros, in some rows or in all: gradients of zero, nothing divided by it."""
    lens = [300, 20]
    q, k, v, dout = pack(lens, 0, 2, 1, 64, FP16)
    op = layers.PackedAttention(2, 1, 64)
    dout[::2] = 0
    got = run(op, q, k, v, dout, cu_of(lens))
    assert not got[2][::2].any()
    exact = exact16(q, k, v, lens, True, op.scale, dout)
    for name, x in zip(NAMES, got):
        within(x, *exact[name], name)
    for x in run(op, q, k, v, torch.zeros_like(dout), cu_of(lens))[2:]:
        assert not x.any()
    for x in run(op, q, k, torch.zeros_like(v), dout, cu_of(lens))[2:4]:
        assert not x.any()
