"""One worker's attention block: the operators that produce the gradients the
exchange carries.

``QKNormRope`` normalises queries and keys per head and rotates them by their
positions, ``PackedAttention`` attends within the sequences of a pack, and
``Dropout`` draws its mask from the counter-based generator and adds the
residual.  Each has ``forward`` and ``backward``; what the backward pass needs
is passed back in by the caller, who also owns every tensor.  Heads are
``[tokens, heads, head_dim]`` tensors whose last dimension is dense, slices of a
joint projection among them.

Work goes to torch's current stream, or to ``stream``, under which outputs and
scratch are then allocated too; a tensor that another stream made or will free
has to be ordered by the caller, as with any torch operator.  Every tensor of a
call, an operator's own included, is on the current device.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import dq


def _on_stream(call):
    """Adds the keyword ``stream``: a stream or its handle, under which the call allocates and launches."""
    @functools.wraps(call)
    def run(self, *args, stream=None, **kw):
        if stream is None:
            return call(self, *args, **kw)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
            return call(self, *args, **kw)
    return run


def _fp32(x: float) -> float:
    """x as the kernels' parameters hold it; what they could not hold is refused where it is given."""
    return ctypes.c_float(x).value


def _heads(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, gpu: int) -> bytes:
    """The view of a checked [tokens, heads, head_dim] tensor; gpu: the current device, on which the call will run."""
    s = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != gpu or (s[2] != 1 and shape[2] > 1 and t.numel()):
        raise ValueError(f"{name}: expected {list(shape)} of {dtype} on GPU {gpu} (the current one) with a dense last "
                         f"dimension, got {list(t.shape)} of {t.dtype} on {t.device}, strides {s}")
    return dq.heads_bytes(t.data_ptr(), s[0], s[1])


def _vector(name: str, t: torch.Tensor, n: int, dtypes: tuple, gpu: int) -> torch.Tensor:
    if t.dim() != 1 or t.shape[0] != n or t.dtype not in dtypes or t.get_device() != gpu or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: expected {n} dense values of {' or '.join(map(str, dtypes))} on GPU {gpu} (the current "
                         f"one), got {list(t.shape)} of {t.dtype} on {t.device}")
    return t


def _own(name: str, t: torch.Tensor, gpu: int):
    """An operator's own tensor has to be where the call will run."""
    if t.get_device() != gpu:
        raise ValueError(f"the operator's {name} is on {t.device}, the current device is GPU {gpu}")


def rope_table(n_positions: int, rot_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines, then sines, of p * theta^(-2i / rot_dim) for position p and pair i < rot_dim / 2, computed in 64
    bits and rounded once to fp32: [n_positions, rot_dim].  Lay it out once and keep it."""
    if rot_dim % 2:
        raise ValueError("rot_dim is even")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * theta ** (-i / max(rot_dim, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class PackedAttention:
    """Softmax attention within each sequence of a pack, with grouped heads: query head h reads key head
    h // (n_heads // n_kv_heads).  bf16 or fp16, head_dim a multiple of 8 up to 128.

    ``cu_seqlens``: int32 on the GPU, ascending from 0: sequence s holds the tokens from ``cu_seqlens[s]`` to
    ``cu_seqlens[s + 1]``, any length from 0.  Tokens behind the last one are padding: output and gradients 0,
    lse -inf.  The lengths are read on the GPU only."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, *, causal: bool = True, scale: float = None,
                 device="cuda"):
        if n_kv_heads < 1 or n_heads < 1 or n_heads % n_kv_heads:
            raise ValueError("n_heads is a multiple of n_kv_heads")
        if head_dim % 8 or not 8 <= head_dim <= 128:
            raise ValueError("head_dim is a multiple of 8 from 8 to 128")
        self.n_heads, self.n_kv_heads, self.head_dim, self.causal = n_heads, n_kv_heads, head_dim, bool(causal)
        self.scale = _fp32(1.0 / math.sqrt(head_dim) if scale is None else scale)
        if not 0.0 < self.scale <= 3.4e38:
            raise ValueError("scale is positive and finite in fp32")
        dq.lib()
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def _shape(self, q, cu_seqlens, gpu) -> bytes:
        if q.dtype is not torch.bfloat16 and q.dtype is not torch.float16:
            raise ValueError(f"attention takes bf16 or fp16, got {q.dtype}")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens holds one value more than there are sequences")
        n = cu_seqlens.shape[0]
        _vector("cu_seqlens", cu_seqlens, n, (torch.int32,), gpu)
        _own("status word", self.status, gpu)
        return dq.attention_bytes(dq.DTYPES[q.dtype], self.n_heads, self.n_kv_heads, self.head_dim, self.causal,
                                  self.scale, q.shape[0], n - 1, cu_seqlens.data_ptr())

    def _lse(self, lse, T, gpu):
        if lse.shape != (self.n_heads, T) or lse.dtype is not torch.float32 or not lse.is_contiguous() \
                or lse.get_device() != gpu:
            raise ValueError(f"lse: expected dense fp32 [{self.n_heads}, {T}] on GPU {gpu} (the current one)")

    @_on_stream
    def forward(self, q, k, v, cu_seqlens, out=None, lse=None):
        """(out, lse): the attention output, [tokens, n_heads, head_dim], and the log-sum-exp of each row's
        scores, fp32 [n_heads, tokens]."""
        T, dtype, gpu = q.shape[0], q.dtype, torch.cuda.current_device()
        of_q, of_k = (T, self.n_heads, self.head_dim), (T, self.n_kv_heads, self.head_dim)
        views = _heads("q", q, of_q, dtype, gpu), _heads("k", k, of_k, dtype, gpu), _heads("v", v, of_k, dtype, gpu)
        a = self._shape(q, cu_seqlens, gpu)
        if out is None:
            out = torch.empty(of_q, dtype=dtype, device=q.device)
        if lse is None:
            lse = torch.empty((self.n_heads, T), dtype=torch.float32, device=q.device)
        else:
            self._lse(lse, T, gpu)
        to = _heads("out", out, of_q, dtype, gpu)
        if T:
            dq.dq_attention_forward(a, *views, to, lse, self.status)
        return out, lse

    @_on_stream
    def backward(self, dout, q, k, v, out, lse, cu_seqlens, dq_=None, dk=None, dv=None):
        """(dq, dk, dv) from the gradient of ``out``, the inputs and the results of ``forward``."""
        T, dtype, device, gpu = q.shape[0], q.dtype, q.device, torch.cuda.current_device()
        of_q, of_k = (T, self.n_heads, self.head_dim), (T, self.n_kv_heads, self.head_dim)
        views = [_heads("dout", dout, of_q, dtype, gpu), _heads("q", q, of_q, dtype, gpu),
                 _heads("k", k, of_k, dtype, gpu), _heads("v", v, of_k, dtype, gpu),
                 _heads("out", out, of_q, dtype, gpu)]
        self._lse(lse, T, gpu)
        a = self._shape(q, cu_seqlens, gpu)
        dq_ = torch.empty(of_q, dtype=dtype, device=device) if dq_ is None else dq_
        dk = torch.empty(of_k, dtype=dtype, device=device) if dk is None else dk
        dv = torch.empty(of_k, dtype=dtype, device=device) if dv is None else dv
        grads = (_heads("dq", dq_, of_q, dtype, gpu), _heads("dk", dk, of_k, dtype, gpu),
                 _heads("dv", dv, of_k, dtype, gpu))
        if T:
            n = dq.dq_attention_backward_workspace_bytes(a)
            ws = torch.empty(n, dtype=torch.uint8, device=device)
            dq.dq_attention_backward(a, *views, lse, *grads, ws, n, self.status)
        return dq_, dk, dv

    @_on_stream
    def check_status(self):
        """Raises if a call on the current stream, or on ``stream``, reported a device error since the last check, and
        synchronises that stream.  Calls on other streams count once they are done."""
        _own("status word", self.status, torch.cuda.current_device())
        s = dq.dq_get_device_status(self.status)
        if s != dq.DQ_DEVICE_OK:
            self.status.zero_()
            raise RuntimeError(f"attention: device status {s} (a wait ran out)")


class QKNormRope:
    """RMS norm of each query and key head with its weight, then the rotation of the first ``table.shape[1]``
    elements by the token's position, in one pass.

    ``table``: fp32 [n_positions, rot_dim], as ``rope_table`` lays it out.  ``interleaved`` pairs elements 2i and
    2i + 1 instead of i and i + rot_dim / 2.  ``weight_offset`` is added to the weights (1 where they are kept as
    their distance from one).  Weights are fp32 or of the activations' type; their gradients are fp32."""

    def __init__(self, head_dim: int, table: torch.Tensor, *, eps: float = 1e-6, weight_offset: float = 0.0,
                 interleaved: bool = False):
        if head_dim % 8 or not 8 <= head_dim <= 256:
            raise ValueError("head_dim is a multiple of 8 from 8 to 256")
        if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous() or not table.is_cuda:
            raise ValueError("table: expected dense fp32 [positions, rot_dim] on the GPU")
        if table.shape[1] % (8 if interleaved else 16) or table.shape[1] > head_dim:
            raise ValueError("rot_dim is at most head_dim and a multiple of 16 (interleaved: of 8)")
        self.head_dim, self.table, self.eps = head_dim, table, _fp32(eps)
        self.weight_offset, self.interleaved = _fp32(weight_offset), bool(interleaved)
        if not self.eps > 0 or not math.isfinite(self.weight_offset):
            raise ValueError("eps is positive and weight_offset finite in fp32")
        dq.lib()

    def _shape(self, q, k, wq, wk, positions):
        """(parameters, view of q, view of k, current device)."""
        dtype, D, gpu = q.dtype, self.head_dim, torch.cuda.current_device()
        if dtype not in dq.DTYPES:
            raise ValueError(f"expected bf16, fp16 or fp32, got {dtype}")
        if q.dim() != 3 or k.dim() != 3:
            raise ValueError("q and k are [tokens, heads, head_dim]")
        (T, H, _), K = q.shape, k.shape[1]
        of_q, of_k = _heads("q", q, (T, H, D), dtype, gpu), _heads("k", k, (T, K, D), dtype, gpu)
        _vector("wq", wq, D, (torch.float32, dtype), gpu)
        _vector("wk", wk, D, (wq.dtype,), gpu)
        _vector("positions", positions, T, (torch.int32,), gpu)
        _own("table", self.table, gpu)
        rows, rot = self.table.shape
        return dq.norm_rope_bytes(dq.DTYPES[dtype], dq.DTYPES[wq.dtype], H, K, D, rot, self.interleaved, self.eps,
                                  self.weight_offset, T, rows), of_q, of_k, gpu

    @_on_stream
    def forward(self, q, k, wq, wk, positions, q_out=None, k_out=None):
        """(q_out, k_out); ``positions``: int32, one for each token.  Outputs may be the inputs themselves."""
        p, of_q, of_k, gpu = self._shape(q, k, wq, wk, positions)
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
        k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device) if k_out is None else k_out
        to_q, to_k = _heads("q_out", q_out, q.shape, q.dtype, gpu), _heads("k_out", k_out, k.shape, q.dtype, gpu)
        if q.shape[0]:
            dq.dq_qk_norm_rope(p, of_q, of_k, wq, wk, positions, self.table, to_q, to_k)
        return q_out, k_out

    @_on_stream
    def backward(self, dq_out, dk_out, q, k, wq, wk, positions, dq_=None, dk=None):
        """(dq, dk, dwq, dwk) from the gradients of ``forward``'s results and its inputs."""
        p, of_q, of_k, gpu = self._shape(q, k, wq, wk, positions)
        dtype, device = q.dtype, q.device
        dq_ = torch.empty(q.shape, dtype=dtype, device=device) if dq_ is None else dq_
        dk = torch.empty(k.shape, dtype=dtype, device=device) if dk is None else dk
        views = (_heads("dq_out", dq_out, q.shape, dtype, gpu), _heads("dk_out", dk_out, k.shape, dtype, gpu))
        grads = _heads("dq", dq_, q.shape, dtype, gpu), _heads("dk", dk, k.shape, dtype, gpu)
        dwq = torch.empty(self.head_dim, dtype=torch.float32, device=device)
        dwk = torch.empty(self.head_dim, dtype=torch.float32, device=device)
        n = dq.dq_qk_norm_rope_backward_workspace_bytes(p)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        dq.dq_qk_norm_rope_backward(p, *views, of_q, of_k, wq, wk, positions, self.table, *grads, dwq, dwk, ws, n)
        return dq_, dk, dwq, dwk


class Dropout:
    """Dropout at rate ``p`` (realised in steps of 2^-16) with the residual sum.  The mask depends on ``seed``,
    ``site`` (a number of the caller's for the place in the model and the worker), ``round`` (the training step)
    and the element's index, and on nothing else; the backward pass draws it again.  All of these are numbers on the host:
    a captured graph draws the mask of the round that it was captured with."""

    def __init__(self, p: float, *, seed: int = 0, site: int = 0):
        self.p = _fp32(p)
        if not 0.0 <= self.p < 1.0 - 2.0 ** -17:
            raise ValueError("p is at least 0 and below 1 - 2^-17 in fp32")
        if not (0 <= site < 1 << 32 and 0 <= seed < 1 << 64):
            raise ValueError("site has 32 bits, seed 64")
        self.seed, self.site = seed, site
        dq.lib()

    def _run(self, x, residual, out, round):
        shape, dtype, gpu = x.shape, x.dtype, torch.cuda.current_device()
        if dtype not in dq.DTYPES:
            raise ValueError(f"expected bf16, fp16 or fp32, got {dtype}")
        if not 0 <= round < 1 << 64:
            raise ValueError("round has 64 bits")
        out = torch.empty(shape, dtype=dtype, device=x.device) if out is None else out
        for name, t in (("x", x), ("residual", residual), ("out", out)):
            if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()
                                  or t.get_device() != gpu):
                raise ValueError(f"{name}: expected dense {dtype} {list(shape)} on GPU {gpu} (the current one)")
        dq.dq_dropout_add(dq.dropout_bytes(dq.DTYPES[dtype], self.p, self.site, self.seed, round), x, residual, out,
                          x.numel())
        return out

    @_on_stream
    def forward(self, x, residual=None, *, round: int = 0, out=None):
        """residual + the kept elements of x, scaled; ``out`` may be x or residual."""
        return self._run(x, residual, out, round)

    @_on_stream
    def backward(self, dy, *, round: int = 0, out=None):
        """The gradient of x.  (The gradient of the residual is dy itself.)"""
        return self._run(dy, None, out, round)
