"""The attention block's calls in a captured graph: replayed on new inputs, and on new lengths in the same tensors, the
results are those of direct calls, bit for bit."""
import pytest
import torch

from quantized_hop_gradient_gb300 import build, dq, layers
from test_gpu_block import BF16, DEV, FP16, cu_of, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


def replayed(call, inputs, others):
    """call(*inputs) captured, then replayed with each set of values in the inputs' place, against direct calls."""
    call(*inputs)                                   # kernels' attributes are set on a first call
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(*inputs)
    for values in others:
        want = call(*values)
        for x, y in zip(inputs, values):
            x.copy_(y)
        for _ in range(2):
            for x in got:
                x.fill_(7.0)
            graph.replay()
            for x, y in zip(got, want):
                assert torch.equal(x, y)


@pytest.mark.parametrize("lens,others,H,K,D,dtype", [
    ([100, 0, 80], [[1, 177, 2]], 4, 2, 64, BF16),
    ([900, 517, 640, 1300], [[1300, 1, 2056, 0], [839] * 4], 16, 8, 128, FP16),
    ([2300], [[2200]], 1, 1, 128, BF16),
])
def test_attention(lens, others, H, K, D, dtype):
    op = layers.PackedAttention(H, K, D)
    tail = 30

    def case(lens_, seed):
        *t, dout = pack(lens_, sum(lens) + tail - sum(lens_), H, K, D, dtype, seed=seed)
        return *t, cu_of(lens_), dout

    def both(q, k, v, cu, dout):
        out, lse = op.forward(q, k, v, cu)
        return (out, lse, *op.backward(dout, q, k, v, out, lse, cu))

    replayed(both, case(lens, 0), [case(x, 1 + i) for i, x in enumerate([lens] + others)])
    op.check_status()


def test_qk_norm_rope():
    T, H, K, D = 700, 4, 2, 64
    op = layers.QKNormRope(D, layers.rope_table(1000, D))

    def case(seed):
        q, k, _, dyq = pack([T], 0, H, K, D, BF16, seed=seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        return (q, k, torch.randn(D, generator=g, device=DEV), torch.randn(D, generator=g, device=DEV),
                torch.randint(0, 1000, (T,), generator=g, device=DEV, dtype=torch.int32), dyq, k.clone())

    def both(q, k, wq, wk, pos, dyq, dyk):
        return (*op.forward(q, k, wq, wk, pos), *op.backward(dyq, dyk, q, k, wq, wk, pos))

    replayed(both, case(0), [case(1), case(2)])


def test_dropout():
    op = layers.Dropout(0.3, seed=4, site=1)
    case = lambda seed: tuple(pack([50], 0, 2, 1, 64, BF16, seed=seed)[i].contiguous() for i in (0, 3))   # noqa: E731
    replayed(lambda x, dy: (op.forward(x, x, round=5), op.backward(dy, round=5)), case(0), [case(1), case(2)])
