"""How the attention kernels are launched, without a GPU: the cases that the GPU tests run reach every way of each kernel,
so that a change of the rules cannot leave one untested."""
import ctypes as C

import pytest

from block_regimes import CASES, ways
from quantized_hop_gradient_gb300 import build, dq


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    dq.lib()


@pytest.mark.parametrize("sms", [148, 152])
def test_cases_reach_their_ways(sms):
    for *case, want in CASES:
        assert ways(*case, sms) == want, case
    for kernel, all_ways in enumerate(({"few", "ordered", "many", 2, 8}, {"few", "many", 2, 4}, {"few", "ordered", "many", 4, 8})):
        for wide in (False, True):   # heads of up to 64, and more: two forms of each kernel
            reached = {c[-1][kernel] for c in CASES if (c[4] > 64) == wide}
            assert reached >= all_ways, (kernel, wide)


def test_plan_refuses_bad_arguments():
    a = dq.attention_bytes(dq.DQ_BF16, 4, 2, 64, 1, 0.125, 100, 2, 4096)
    plan = (dq.dq_attention_launch * 3)()
    L = dq.lib()
    for sms, out in ((0, plan), (-1, plan), (152, None)):
        with pytest.raises(dq.DQError) as e:
            dq._call("dq_attention_plan", a, sms, out)
        assert e.value.status == dq.DQ_ERR_INVALID_ARG
    bad = dq.dq_attention(dtype=7, n_heads=4, n_kv_heads=2, head_dim=64, causal=1, scale=0.125, n_tokens=1, n_seqs=1, cu_seqlens=4096)
    assert L.dq_attention_plan(C.byref(bad), 152, plan) == dq.DQ_ERR_INVALID_ARG
