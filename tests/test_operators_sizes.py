"""Sizes past 32 bits: the library takes C ints, which ctypes cuts to their low 32
bits without a word, so the binding refuses what does not fit (meta tensors: nothing
is allocated, and the refusal comes before the device is looked at)."""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe

BIG = 2 ** 32 + 64  # 64 in its low 32 bits


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


CALLS = {
    "norm rows": lambda: moe.moe_norm(t(BIG, 1)),
    "norm row length": lambda: moe.moe_norm(t(1, BIG)),
    "residual rows": lambda: moe.moe_norm_residual(t(BIG, 2), t(BIG, 2)),
    "residual row length": lambda: moe.moe_norm_residual(t(2, BIG), t(2, BIG)),
    "route tokens": lambda: moe.moe_route_grouped(t(BIG, 64), t(8, 64), None, 2),
    "route groups": lambda: moe.moe_route_grouped(t(4, 64), t(8, 64), None, 2, groups=2 ** 32 + 1),
    "route topk_groups": lambda: moe.moe_route_grouped(t(4, 64), t(8, 64), None, 2, topk_groups=1 - 2 ** 32),
    "route group_top": lambda: moe.moe_route_grouped(t(4, 64), t(8, 64), None, 2, group_top=2 ** 32 + 1),
    "route k": lambda: moe.moe_route_grouped(t(4, 64), t(8, 64), None, 2 ** 32 + 2),
    "linear rows": lambda: moe.moe_linear(t(BIG, 64), t(64, 64)),
    "linear columns": lambda: moe.moe_linear(t(4, 64), t(BIG, 64)),
    "linear depth": lambda: moe.moe_linear(t(4, BIG), t(64, BIG)),
    "grouped columns": lambda: moe.moe_linear_grouped(t(4, 64), t(3, dtype=torch.int32), t(2, BIG, 64)),
    "grouped k": lambda: moe.moe_linear_grouped(
        t(4, 64), t(3, dtype=torch.int32), t(2, 64, 64), perm=t(8, dtype=torch.int32), k=2 ** 32 + 2, rows=8),
    "route workspace": lambda: moe.moe_route_grouped_workspace_bytes(BIG, 4096, 128, 8, 1),
    "linear workspace": lambda: moe.moe_linear_workspace_bytes(BIG, 64, 4096, "none", 0),
    "grouped workspace": lambda: moe.moe_linear_grouped_workspace_bytes(8, BIG, 64, 4096, "none", 0),
}


@pytest.mark.parametrize("name", CALLS)
def test_sizes_past_32_bits_are_refused(name):
    with pytest.raises(ValueError, match="32 bits"):
        CALLS[name]()
