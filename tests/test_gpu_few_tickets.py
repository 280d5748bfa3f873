"""GPU: moe_layer_few where a ticket holds several tasks, and K slices of the down tasks:
small experts, up to 64 tokens, spread over all experts or all on the same ones (fewer tasks
than the sizes allow: the last tickets end inside their batch or past the last task).
Bounds as tests/test_gpu_few.py."""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe
from tests.test_gpu_few import BF16, FP32, layer64, make, near

pytestmark = pytest.mark.gpu

CASES = [  # T, H, E, k, F, Fs, act, dtype
    (64, 256, 64, 8, 512, 0, "swiglu", BF16), (32, 128, 200, 8, 1024, 64, "geglu", BF16),
    (16, 512, 32, 4, 256, 256, "swiglu", BF16), (40, 512, 128, 8, 256, 256, "swiglu", FP32),
    (64, 1024, 64, 8, 512, 64, "gelu", BF16), (9, 64, 256, 8, 448, 0, "silu", FP32),
    (64, 2048, 64, 6, 192, 128, "swiglu", BF16), (8, 1024, 60, 8, 576, 0, "none", BF16),
    (4, 1024, 64, 6, 512, 512, "swiglu", BF16),
]


@pytest.mark.parametrize("same", [False, True], ids=["spread", "same"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_H%d_E%d_k%d_F%d_Fs%d_%s_%s" % (*c[:7], str(c[7])[6:]))
def test_tickets(case, same):
    T, H, E, k, F, Fs, act, dtype = case
    print(f"\n[gpu] few tickets {case} same={same}", flush=True)
    route = dict(score="softmax", groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0)
    x, wg, b, p, _ = make(T, H, E, k, F, Fs, act, dtype, True, "choice", T + F, **route)
    if same:  # rows of one direction choose the same experts
        x = (x[:1].float() * (1 + torch.arange(T, device="cuda")[:, None] / 64)).to(dtype)
        b = torch.zeros_like(b)
        b[:k] = 10.0
    out, idx, w = moe.moe_layer_few(x, wg, b, k=k, act=act, bias_mode="choice", **route, **p)
    if same:
        assert (idx.sort(1).values == torch.arange(k, device="cuda", dtype=torch.int32)).all()
    near(out, *layer64(x, p, idx, w, act, dtype), dtype, act)
    for _ in range(5):
        again = moe.moe_layer_few(x, wg, b, k=k, act=act, bias_mode="choice", **route, **p)
        assert torch.equal(again[0], out) and torch.equal(again[1], idx) and torch.equal(again[2], w)
