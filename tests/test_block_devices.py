"""The attention block's calls take tensors of the current device only: every argument, and what the operator holds
itself, on another device is refused before anything is launched.  Stand-ins for tensors; no GPU."""
import pytest
import torch

from quantized_hop_gradient_gb300 import build, layers

BF16 = torch.bfloat16


class OnDevice:
    """What the checks read of a tensor, on a device that this machine need not have."""

    def __init__(self, t, index):
        self.t, self.index = t, index
        self.shape, self.dtype, self.is_cuda = t.shape, t.dtype, index >= 0
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def launches(monkeypatch):
    build.build()
    count = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name in ("dq_attention_forward", "dq_attention_backward", "dq_qk_norm_rope", "dq_qk_norm_rope_backward",
                 "dq_dropout_add", "dq_get_device_status"):
        monkeypatch.setattr(layers.dq, name, lambda *a, _n=name: count.append(_n))
    monkeypatch.setattr(layers.torch, "empty", lambda *s, dtype=None, device=None, _e=torch.empty:
                        OnDevice(_e(*s, dtype=dtype), device.index))
    return count


def heads(n):
    return torch.zeros(6, n, 16, dtype=BF16)


def attention(backward):
    op = layers.PackedAttention(4, 2, 16, device="cpu")
    t = {"q": heads(4), "k": heads(2), "v": heads(2), "cu_seqlens": torch.tensor([0, 6], dtype=torch.int32),
         "out": heads(4), "lse": torch.zeros(4, 6)}
    if backward:
        t |= {"dout": heads(4), "dq_": heads(4), "dk": heads(2), "dv": heads(2)}
    return op, op.backward if backward else op.forward, t, "status"


def norms(backward):
    op = object.__new__(layers.QKNormRope)
    op.head_dim, op.eps, op.weight_offset, op.interleaved = 16, 1e-6, 0.0, False
    op.table = torch.zeros(8, 16)
    t = {"q": heads(4), "k": heads(2), "wq": torch.ones(16), "wk": torch.ones(16),
         "positions": torch.arange(6, dtype=torch.int32)}
    if backward:
        t |= {"dq_out": heads(4), "dk_out": heads(2), "dq_": heads(4), "dk": heads(2)}
    else:
        t |= {"q_out": heads(4), "k_out": heads(2)}
    return op, op.backward if backward else op.forward, t, "table"


def dropout(backward):
    op = layers.Dropout(0.1)
    t = {"dy": heads(4)} if backward else {"x": heads(4), "residual": heads(4)}
    return op, op.backward if backward else op.forward, t | {"out": heads(4)}, None


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("make", [attention, norms, dropout])
def test_tensors_of_another_device_are_refused(make, backward, launches):
    op, call, tensors, own = make(backward)
    held = getattr(op, own) if own else None
    names = list(tensors) + ([own] if own else [])

    def run(where):
        if own:
            setattr(op, own, OnDevice(held, where.get(own, where["*"])))
        call(**{n: OnDevice(t, where.get(n, where["*"])) for n, t in tensors.items()})

    run({"*": 0})
    assert len(launches) == 1
    for name in names:                       # one of them elsewhere: another GPU, or the host
        for index in (1, -1):
            with pytest.raises(ValueError):
                run({"*": 0, name: index})
    for index in (1, -1):                    # all of them together
        with pytest.raises(ValueError):
            run({"*": index})
    assert len(launches) == 1


def test_status_of_another_device_is_refused(launches):
    op = attention(False)[0]
    op.status = OnDevice(op.status, 1)
    with pytest.raises(ValueError):
        op.check_status()
