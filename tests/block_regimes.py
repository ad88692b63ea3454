"""Calls whose attention kernels are launched in each of the ways there are on a GPU of about 150 SMs, with the ways."""
import torch

from quantized_hop_gradient_gb300 import dq

BF16, FP16 = torch.bfloat16, torch.float16
MIXED = [900, 517, 0, 640, 1300, 1]

# lens, tail, heads, kv heads, dim, dtype, causal; for the forward, the dq and the dk, dv kernel: "few" (at most a block a
# SM), "ordered" (several, in the order of their work), "many" (several, in turn), or the split of a tile's loop
CASES = [
    (MIXED, 77, 16, 8, 64, BF16, True, ("ordered", "many", "ordered")),
    (MIXED, 77, 16, 8, 96, FP16, False, ("ordered", "many", "ordered")),
    (MIXED, 0, 16, 8, 128, BF16, True, ("ordered", "many", "ordered")),
    (MIXED, 77, 16, 8, 128, FP16, False, ("ordered", "many", "ordered")),
    (MIXED, 77, 64, 32, 64, FP16, True, ("many", "many", "many")),
    (MIXED, 77, 64, 32, 96, BF16, True, ("many", "many", "many")),
    (MIXED, 77, 64, 32, 128, BF16, False, ("many", "many", "many")),
    (MIXED, 77, 64, 32, 128, FP16, True, ("many", "many", "many")),
    ([1024, 700] * 3, 0, 15, 15, 128, BF16, True, ("ordered", "many", "many")),   # two tiles of one head
    ([1024, 700] * 3, 0, 15, 15, 64, BF16, False, ("ordered", "many", "many")),
    ([4200], 5, 1, 1, 64, BF16, True, (8, 4, 4)),
    ([4200], 0, 1, 1, 128, FP16, False, (8, 4, 4)),
    ([4200], 0, 1, 1, 96, BF16, True, (8, 4, 4)),
    ([2000], 9, 4, 1, 64, FP16, True, (4, 2, 8)),
    ([2000], 0, 4, 1, 128, BF16, False, (4, 2, 8)),
    ([2000], 0, 4, 1, 72, BF16, True, (4, 2, 8)),
    ([1800], 3, 2, 1, 64, FP16, False, (2, 2, 4)),
    ([1800], 0, 2, 1, 128, BF16, True, (2, 2, 4)),
    ([300, 200], 0, 2, 1, 64, BF16, False, ("few", "few", "few")),
    ([300, 200], 0, 2, 1, 128, BF16, True, ("few", "few", "few")),
]


def ways(lens, tail, H, K, D, dtype, causal, n_sms):
    a = dq.attention_bytes(dq.DTYPES[dtype], H, K, D, causal, 0.125, sum(lens) + tail, len(lens), 4096)
    way = []
    for x in dq.dq_attention_plan(a, n_sms):
        if x.split > 1:
            way.append(x.split)
        elif x.blocks <= n_sms:
            way.append("few")
        else:
            way.append("ordered" if x.by_work else "many")
    return tuple(way)
