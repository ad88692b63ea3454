"""Numbers that the kernels' parameters cannot hold are refused by the operators as a ValueError, where they are given."""
import math

import pytest
import torch

from quantized_hop_gradient_gb300 import build, layers


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def test_attention_scale():
    for bad in (0.0, -1.0, 1e39, 1e-50, math.inf, math.nan):
        with pytest.raises(ValueError):
            layers.PackedAttention(2, 1, 64, scale=bad, device="cpu")
    assert layers.PackedAttention(2, 1, 64, device="cpu").scale == 0.125


def test_dropout_rate_is_the_kernels():
    """A rate that rounds to 1 - 2^-17 in fp32 is refused here as the kernel's entry refuses it."""
    for bad in (-1e-3, 1.0, 1 - 2.0 ** -17, 1 - 2.0 ** -17 - 1e-12, math.nan):
        with pytest.raises(ValueError):
            layers.Dropout(bad)
    assert layers.Dropout(0.1).p == torch.tensor(0.1).item()
    layers.Dropout(1 - 2.0 ** -16)


def test_dropout_round(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)       # a host tensor passes the device check
    monkeypatch.setattr(layers.dq, "dq_dropout_add", lambda *a: None)
    x = torch.ones(8)
    op = layers.Dropout(0.5)
    for bad in (-1, 1 << 64):
        for call in (op.forward, op.backward):
            with pytest.raises(ValueError):
                call(x, round=bad)
    op.forward(x, round=(1 << 64) - 1)


@pytest.mark.gpu
def test_norm_numbers():
    t = layers.rope_table(8, 64)
    for bad in (dict(eps=0.0), dict(eps=1e-60), dict(eps=math.nan), dict(weight_offset=math.inf), dict(weight_offset=1e39)):
        with pytest.raises(ValueError):
            layers.QKNormRope(64, t, **bad)
