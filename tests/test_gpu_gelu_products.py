"""GPU: the bf16 GeLU of moe_linear's epilogue on known arguments: every bf16 value, and
sums of two, is the correctly rounded a Phi(a) except within a band around the rounding
borders. The band: the fp32 value is off by at most 5e-6 relative for |a| <= 6 (the
fitted polynomial 1.0e-6, its fp32 evaluation with p down to -30: 2^-24 * 30 * ln 2 * 2 =
2.5e-6, exp2 and the last product 2^-23) and by 6e-9 beyond, where Phi(-6) = 1e-9 stands
for the tail."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_amd as moe

pytestmark = pytest.mark.gpu
REL, TAIL = 5e-6, 6e-9


def bf16_all():
    """Every finite bf16 value."""
    b = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    return b[torch.isfinite(b)]


def rows_of(a, b=None):
    """x [n,64] and w [64,64] with a (+ b) in column 0 of the product."""
    x = torch.zeros((a.numel(), 64), dtype=torch.bfloat16)
    x[:, 0] = a
    if b is not None:
        x[:, 1] = b
    w = torch.zeros((64, 64), dtype=torch.bfloat16)
    w[:, :2] = 1.0
    return x.cuda(), w.cuda()


def check(got, a, tag):
    """got bf16 [n,64] against gelu(a), a float64 [n] on the GPU."""
    want = a * torch.special.ndtr(a)
    band = torch.where(a.abs() <= 6, REL * want.abs(), TAIL) + 1e-38
    lo, hi = (want - band).bfloat16(), (want + band).bfloat16()
    ok = (got >= lo[:, None]) & (got <= hi[:, None])
    bad = (~ok[:, 0]).nonzero().flatten()
    assert ok.all(), f"{tag}: {bad.numel()} of {a.numel()}, first {float(a[bad[0]])}: {float(got[bad[0], 0])}"


@pytest.mark.parametrize("act", ["gelu", "geglu"])
def test_every_value(act):
    print(f"\n[gpu] gelu {act}", flush=True)
    a = bf16_all()
    for b in (None, 2.0 ** -9 * a, torch.full_like(a, 0.3)):
        keep = torch.ones_like(a, dtype=torch.bool) if b is None else (a.abs() < 64) & (a.abs() > 2.0 ** -60)
        ab, bb = a[keep], None if b is None else b[keep]
        x, w = rows_of(ab, bb)
        exact = ab.double() if b is None else ab.double() + bb.double()
        exact = exact.float().double().cuda()  # the product's one addition
        if act == "geglu":
            w = torch.stack([w, torch.zeros_like(w)])
            got = moe.moe_linear(x, w, torch.tensor([[0.0], [1.0]]).expand(2, 64).bfloat16().contiguous().cuda(),
                                 act=act)  # times an up half of 1
        else:
            got = moe.moe_linear(x, w, act=act)
        for part in range(0, 64, 21):
            check(got[:, part:part + 1].expand(-1, 1), exact, f"{act} column {part}")


def test_paths_agree():
    """The same values through every bf16 path."""
    g = torch.Generator().manual_seed(0)
    v = (6 * torch.randn(17, generator=g)).bfloat16()
    for M, N, K in ((17, 64, 64), (901, 960, 64), (257, 2112, 2048), (1101, 4160, 320), (2601, 4160, 128)):
        print(f"\n[gpu] gelu path {moe.moe_linear_path(M, N, K, 'gelu', 1)}", flush=True)
        x = torch.zeros((M, K), dtype=torch.bfloat16)
        x[:, 0] = v[torch.arange(M) % 17]
        w = torch.zeros((N, K), dtype=torch.bfloat16)
        w[:, 0] = 1.0
        got = moe.moe_linear(x.cuda(), w.cuda(), act="gelu")
        check(got[:, :64], x[:, 0].double().cuda(), (M, N, K))
        assert (got == got[:, :1]).all()
