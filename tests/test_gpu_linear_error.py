"""GPU: how far fp32 products are from float64 where one workgroup sums all of K.

u = 2^-24. An addition rounds by u / sqrt(6) of its result in the mean. Sums of K products
of random sign have partial sums of s j / K plus noise of sqrt(j / K): over one chain the
error is u sqrt((1 / 3 + 1 / 2) K / 6) of the result's mean size, 24 u for K = 4096. Over
4 sums side by side it is u sqrt((1 / (3 * 16) + 1 / 8) K / 6): 10 u. The epilogue adds a
few u; a gated product of two such sums has sqrt(2) times that: 15 u. Held to 12 u and
18 u of the result's norm at K = 4096, as sqrt(K) below."""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def randn(g, *shape, std=1.0):
    return torch.empty(shape, device="cuda").normal_(0, std, generator=g)


@pytest.mark.parametrize("K", [1024, 2048, 3392, 4096])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("M,N", [(512, 4096), (1000, 2112), (137, 1664), (200, 64)])
def test_dense(M, N, K, act):
    print(f"\n[gpu] linear error {M} {N} {K} {act} {moe.moe_linear_path(M, N, K, act, 0)}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + K)
    two = (2,) if act == "swiglu" else ()
    x, w = randn(g, M, K), randn(g, *two, N, K, std=K ** -0.5)
    got = moe.moe_linear(x, w, act=act)
    a = x.double() @ w.reshape(-1, K).double().t()
    want = a if act == "none" else a[:, :N] * torch.sigmoid(a[:, :N]) * a[:, N:]
    rel = float((got.double() - want).norm() / want.norm())
    bound = (12 if act == "none" else 18) * (K / 4096) ** 0.5 + 2
    assert rel <= bound * U, f"{rel / U:.1f} u, bound {bound:.1f}"


def test_grouped():
    E, T, k, N, K = 8, 512, 2, 1088, 4032
    print("\n[gpu] linear error grouped", flush=True)
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = randn(g, T, K), randn(g, E, N, K, std=K ** -0.5)
    perm = torch.randperm(T * k, generator=g, device="cuda").int()
    off = torch.arange(0, T * k + 1, T * k // E, dtype=torch.int32, device="cuda")
    got = moe.moe_linear_grouped(x, off, w, perm=perm, k=k)
    want = torch.cat([x[perm[int(off[e]):int(off[e + 1])].long() // k].double() @ w[e].double().t()
                      for e in range(E)])
    rel = float((got.double() - want).norm() / want.norm())
    assert rel <= 14 * U, f"{rel / U:.1f} u"
