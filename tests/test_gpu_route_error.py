"""GPU: how far the softmax weights of moe_route_grouped are from float64 where a score
is one sum over all of H (an H with few factors of two, which no K slices divide).

u = 2^-24. An addition rounds by u / sqrt(6) of its result in the mean (u / sqrt(3) of the
power of two below it). In one chain over a score s of K products, partial sums are
s j / K plus noise of sqrt(j / K), so the sum is off by u sqrt((s^2 / 3 + 1 / 2) K / 6):
with |s| = 2.8 (the largest of a few hundred) u sqrt(0.52 K), 33 u for K = 2112 and 46 u
for 4096. Over n sums side by side, each with partial sums n times smaller in s and
sqrt(n) in noise, it is u sqrt((s^2 / (3 n^2) + 1 / (2 n)) K / 6): 14 u for n = 4 and
K = 4096, 8 u for n = 8. bf16 products come 32 to an addition of the matrix core, which
rounds less than half as often: 2 sums of 4096 stay below 17 u / sqrt(2) = 12 u. A softmax
weight is off by its score's error and a weighted mean of the others', plus a few u for
exp and the division: the norm of the error over a call is held to 16 u of the weights'
norm, which one chain of fp32 passes for every H here."""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("H", [2112, 2880, 4032, 4096])
def test_softmax_weights(H, renorm, dtype):
    for T, E in ((16, 256), (64, 256), (300, 200), (1024, 128), (1000, 60), (1500, 256), (2500, 256), (6000, 128)):
        if dtype == torch.float32 and T > 2048:
            continue
        print(f"\n[gpu] route error T={T} H={H} E={E} renorm={renorm} {dtype}", flush=True)
        g = torch.Generator(device="cuda").manual_seed(T + H + E)
        x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
        wg = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).to(dtype)
        idx, w = moe.moe_route_grouped(x, wg, None, 4, score="softmax", renorm=renorm)
        want = torch.softmax(x.double() @ wg.double().t(), 1).gather(1, idx.long())
        if renorm:
            want = want / want.sum(1, keepdim=True)
        rel = float((w.double() - want).norm() / want.norm())
        assert rel <= 16 * U, f"T={T} E={E}: {rel / U:.1f} u"
