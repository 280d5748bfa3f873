"""Refusals of moe_block_forward's options: on the host, nothing is launched."""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


H, WG, UP, DOWN, S = t(2, 128), t(4, 128), t(4, 2, 128, 128), t(4, 128, 128), t(4, 1, 1, dtype=torch.float32)
SHARED = dict(ws_up=t(2, 128, 128), ws_down=t(128, 128))


@pytest.mark.parametrize("text,kw", [
    ("need w_up_scale and w_down_scale", dict(w_up_scale=S)),
    ("need w_up_scale and w_down_scale", dict(w_down_scale=S)),
    ("need ws_up_scale and ws_down_scale", dict(ws_up_scale=S, **SHARED)),
    ("without a shared expert", dict(ws_up_scale=S, ws_down_scale=S)),
    ("few takes no 8-bit experts", dict(few=True, w_up_scale=S, w_down_scale=S)),
    ("few takes no 8-bit experts", dict(few=True, ws_up_scale=S, ws_down_scale=S, **SHARED)),
    ("few takes no capacity", dict(few=True, capacity=3)),
    ("must be GPU tensors", dict(few=True)),
    ("must be GPU tensors", dict(w_up_scale=S, w_down_scale=S)),
])
def test_refusals(text, kw):
    with pytest.raises(ValueError, match=text):
        moe.moe_block_forward(H, WG, UP, DOWN, 2, **kw)


def test_8bit_is_bf16():
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        moe.moe_block_forward(H.float(), WG.float(), UP, DOWN, 2, w_up_scale=S, w_down_scale=S)
