"""GPU: moe_route_grouped on every path that its sizes choose: one launch of 16, 32 and
64 tokens a workgroup, two launches for few and for many tokens, with every number of
K slices (asserted by the workspace, which holds the slices' scores).

The definition in float64 (torch, all tokens at once). Ids are compared exactly, on
scores that are exact (one-hot tokens, whole-number gates) or that are drawn again
until the decisions are clear; weights to 2e-5: scores of up to 4096 products are off
by at most about 4e-6, sigmoid and softmax pass on at most twice that, relative, the
renormalisation doubles it, and a few ulp."""
import math

import pytest
import torch

import sparse_mixture_experts_05_amd as moe

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
RTOL_W, CLEAR = 2e-5, 4e-5


def definition(s, bias, k, score, groups, topk_groups, group_top, renorm, scale):
    """(ids, weights, each token's least distance of two different values that a decision
    is between) from scores s [T,E] in float64."""
    T, E = s.shape
    p = torch.sigmoid(s) if score == "sigmoid" else torch.softmax(s, 1)
    v = p if bias is None else p + bias.double()
    off = torch.isnan(v) | torch.isneginf(v)
    v = v.masked_fill(off, -math.inf)
    key = s if bias is None else v

    def least(a):  # sorted rows
        d = a[:, :-1] - a[:, 1:]
        d = d.masked_fill(~torch.isfinite(d) | (d == 0), math.inf)
        return d.min(1).values if d.shape[1] else torch.full((T,), math.inf, device=s.device)

    gap = torch.full((T,), math.inf, dtype=torch.float64, device=s.device)
    allowed = torch.ones((T, E), dtype=torch.bool, device=s.device)
    if topk_groups < groups:
        per = E // groups
        b = v.view(T, groups, per).sort(dim=2, descending=True).values[:, :, :group_top]
        gs = torch.where(torch.isneginf(b[:, :, 0]), b[:, :, 0], b.masked_fill(torch.isneginf(b), 0).sum(2))
        o = gs.sort(dim=1, descending=True, stable=True)
        gap = least(o.values)
        chosen = torch.zeros((T, groups), dtype=torch.bool, device=s.device)
        chosen.scatter_(1, o.indices[:, :topk_groups], True)
        allowed = chosen.repeat_interleave(per, 1)
    # experts that are off rank behind the ones that are on, lower ids first
    rank = key.masked_fill(off, -1e300).masked_fill(~allowed, -math.inf)
    o = rank.sort(dim=1, descending=True, stable=True)
    top = o.values[:, : k + 1]
    gap = torch.minimum(gap, least(top.masked_fill(top < -1e299, -math.inf)))
    ids = o.indices[:, :k]
    w = p.gather(1, ids).masked_fill(off.gather(1, ids), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return ids, w * scale, gap


def check(x, wg, bias, k, want, **kw):
    ids, w, _ = want
    got_i, got_w = moe.moe_route_grouped(x, wg, bias, k, **kw)
    bad = (got_i != ids).any(1).nonzero().flatten()
    assert bad.numel() == 0, f"{bad.numel()} tokens differ, first {bad[0]}: {got_i[bad[0]]} for {ids[bad[0]]}"
    torch.testing.assert_close(got_w.double(), w, rtol=RTOL_W, atol=1e-30)


def slices(T, H, E, k, dtype):
    """K slices of the two-launch paths, from the workspace; 0: one launch."""
    need = moe.moe_route_grouped_workspace_bytes(T, H, E, k, int(dtype == BF16))
    n = need // (T * E * 4)
    assert need == 0 or need == -(-n * T * E * 4 // 256) * 256
    return n


ONE = [  # (E, k, groups, topk_groups, group_top) of one launch from 16384 tokens on
    (16, 4, 4, 2, 2), (32, 2, 1, 1, 1), (60, 4, 6, 3, 1), (64, 8, 64, 8, 2), (128, 8, 8, 4, 2),
    (128, 1, 32, 5, 1), (255, 8, 5, 2, 2), (256, 8, 8, 4, 2), (256, 3, 32, 9, 2), (252, 8, 63, 3, 1),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("cfg", ONE, ids=str)
def test_exact_scores(cfg, score):
    """Ties between experts and groups and experts that are off, 64 tokens a workgroup
    (whole and ragged last ones), 32 for 64 experts or less, and two launches."""
    E, k, groups, tg, gt = cfg
    for T, H in ((16384, 64), (16385, 128), (16447, 64), (8200, 64), (20000, 192)):
        print(f"\n[gpu] route exact {cfg} {score} T={T} H={H}", flush=True)
        one = T >= 16384 or E <= 64
        assert (slices(T, H, E, k, BF16) == 0) == one
        g = torch.Generator(device="cuda").manual_seed(E * 31 + T)
        hot = torch.randint(H, (T,), generator=g, device="cuda")
        x = torch.zeros((T, H), device="cuda").scatter_(1, hot[:, None], 1.0)
        wg = torch.randint(5, (E, H), generator=g, device="cuda").float()
        # one step a group where its scores are sums: equal sums then tie in every bit
        n = groups if gt == 2 and groups > 1 else E
        bias = 8.0 * torch.randint(3, (n,), generator=g, device="cuda").float().repeat_interleave(E // n)
        bias[torch.randint(E, (3,), generator=g, device="cuda")] = -math.inf
        bias[torch.randint(E, (1,), generator=g, device="cuda")] = math.nan
        bias[: E // groups if groups > 1 else 2] = -math.inf
        s = wg.double().t()[hot]
        for b in (bias, None):
            kw = dict(score=score, groups=groups, topk_groups=tg, group_top=gt, renorm=bool(T % 2), scale=2.5)
            want = definition(s, b, k, **kw)
            assert want[2].min() > 1e-5
            check(x.bfloat16(), wg.bfloat16(), b, k, want, **kw)


def clear_rows(T, H, E, k, dtype, bias, seed, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    wg = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).to(dtype)
    for _ in range(200):
        s = x.double() @ wg.double().t()
        want = definition(s, bias, k, **kw)
        bad = (want[2] < CLEAR).nonzero().flatten()
        if bad.numel() == 0:
            return x, wg, want
        x[bad] = torch.randn((bad.numel(), H), generator=g, device="cuda").to(dtype)
    raise RuntimeError("no rows with clear decisions")


def random_rows(T, H, E, dtype, expect):
    """Sigmoid with a choice bias, groups and renormalisation; softmax without any."""
    k, groups = min(8, E // 8), next(n for n in (4, 3, 5) if E % n == 0)
    assert slices(T, H, E, k, dtype) == expect, (T, H, E)
    g = torch.Generator(device="cuda").manual_seed(E)
    bias = 0.05 * torch.randn(E, generator=g, device="cuda")
    for n, (b, kw) in enumerate((
            (bias, dict(score="sigmoid", groups=groups, topk_groups=2, group_top=2, renorm=True, scale=2.5)),
            (None, dict(score="softmax", groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.5)))):
        print(f"\n[gpu] route random T={T} H={H} E={E} {kw['score']} {dtype} slices={expect}", flush=True)
        x, wg, want = clear_rows(T, H, E, k, dtype, b, T + H + n, **kw)
        check(x, wg, b, k, want, **kw)


FEW = [  # (T, H, E, K slices): bf16, two launches below 2048 tokens
    (1, 4096, 128, 16), (2, 4096, 256, 16), (4, 2560, 256, 8), (5, 4096, 128, 16), (16, 4096, 128, 16),
    (16, 2112, 128, 1), (17, 2176, 128, 2), (48, 2304, 256, 4), (48, 4096, 60, 16), (100, 2560, 60, 8),
    (300, 4096, 256, 2), (300, 2112, 64, 1), (1023, 4096, 128, 2), (1024, 4096, 128, 2), (1025, 4096, 255, 1),
    (2047, 4096, 60, 2), (640, 4096, 60, 4), (65, 2176, 64, 2), (200, 2304, 128, 4),
]


@pytest.mark.parametrize("T,H,E,n", FEW)
def test_few_tokens(T, H, E, n):
    random_rows(T, H, E, BF16, n)


MANY = [  # (T, H, E, K slices): bf16, two launches of large tiles
    (2048, 1024, 256, 16), (2049, 512, 256, 8), (2100, 256, 256, 4), (2048, 1024, 128, 8), (2111, 320, 128, 1),
    (4099, 256, 128, 2), (9000, 128, 200, 2), (16383, 64, 256, 1), (16383, 128, 65, 1), (3000, 4096, 129, 8),
]


@pytest.mark.parametrize("T,H,E,n", MANY)
def test_many_tokens(T, H, E, n):
    random_rows(T, H, E, BF16, n)


F32 = [  # (T, H, E, K slices): fp32, two launches
    (1, 4096, 128, 16), (3, 2048, 256, 16), (16, 1024, 60, 8), (48, 512, 128, 4), (100, 256, 256, 2),
    (17, 320, 60, 1), (511, 4096, 128, 8), (512, 4096, 256, 16), (513, 1024, 64, 8), (700, 512, 255, 4),
    (1023, 256, 128, 2), (1025, 2112, 200, 1), (3000, 2048, 256, 4),
]


@pytest.mark.parametrize("T,H,E,n", F32)
def test_fp32(T, H, E, n):
    random_rows(T, H, E, FP32, n)
