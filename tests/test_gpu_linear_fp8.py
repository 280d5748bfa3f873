"""GPU: moe_linear_fp8 and moe_linear_grouped_fp8 against the formula in float64.

Tolerance, element by element (u = 2^-24). The matrix core adds the products of 8
neighbours of K at a time: it lines them up with the one of the largest exponents and
cuts the others at 2^-13 of that power of two, toward zero (measured: beside one product
of 2^16, 2^3 counts and 2^2 does not, of either sign, wherever the two stand in the 8,
and all count in another 8). The power of two is at most the largest product, so 8
products are off by at most 7 * 2^-13 max|x| max|w| over the 8; on ordinary data the cuts
cancel (1.5e-5 of the result, its bf16 rounding is 2e-3). The 16 sums of a block are
added in fp32 in an order of its own: 256 u of sum|x w| is more than any takes. A block's
sum is scaled (two roundings of the scale and the FMA's), and K / 128 of them added: a is
off by at most
    d = sum of the cuts + (256 + K / 128 + 3) u sum|s x w| + 2 u |a|.
From there on as tests/test_gpu_linear.py."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_amd as moe
from tests.test_gpu_linear import ACTS, HALF, U, act64, near, randn, segments

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
GUARD = 64


def rows8(M, K, seed, std=1.0):
    """(x, x_scale): e4m3 rows with scales of any mantissa that differ from block to block."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty((M, K), device="cuda").normal_(0, 60, generator=g).clamp_(-448, 448).to(FP8)
    s = torch.empty((K // 128, M), device="cuda").uniform_(0.3, 3.0, generator=g) * (std / 60)
    return x, s


def weight8(lead, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.empty((*lead, N, K), device="cuda").normal_(0, 60, generator=g).clamp_(-448, 448).to(FP8)
    s = torch.empty((*lead, -(-N // 128), K // 128), device="cuda").uniform_(0.3, 3.0, generator=g)
    return w, s * (K ** -0.5 / 60)


def wide(w, s):
    """[N, K] in 64 bits."""
    return w.double() * s.double().repeat_interleave(128, 0)[:len(w)].repeat_interleave(128, 1)


def top8(v):
    """The largest |v| of each 8 neighbours (a block's elements share their scale)."""
    return v.abs().view(len(v), -1, 8).amax(2)


def product64(x, xs, w, ws, bias, act, res):
    """(y, its error bound before rounding) of one segment; w [N,K] or [2,N,K]."""
    K = x.shape[1]
    xf = x.double() * xs.double().t().repeat_interleave(128, 1)
    halves = []
    for h in range(2 if w.dim() == 3 else 1):
        wf = wide(w[h], ws[h]) if w.dim() == 3 else wide(w, ws)
        a = xf @ wf.t()
        d = (256 + K // 128 + 3) * U * (xf.abs() @ wf.abs().t())
        d = d + 7 * 2.0 ** -13 * (top8(xf) @ top8(wf).t())
        if bias is not None:
            a = a + (bias[h] if w.dim() == 3 else bias).double()
        halves.append((a, d + 2 * U * a.abs()))
    e = 1e-4 if act in ("gelu", "geglu") else 8 * U
    (a, d) = halves[0]
    y = act64(a, act)
    err = 1.13 * d + e * y.abs()
    if w.dim() == 3:
        b, db = halves[1]
        err = err * (b.abs() + db) + y.abs() * db
        y = y * b
    if res is not None:
        y = y + res.double()
        err = err + 2 * U * (y.abs() + res.double().abs())
    return y, err


def make(M, N, K, act, bias, res, seed, E=None):
    two = (2,) if act in ("geglu", "swiglu") else ()
    lead = () if E is None else (E,)
    w, ws = weight8((*lead, *two), N, K, seed + 1)
    return dict(w=w, w_scale=ws, bias=randn((*lead, *two, N), BF16, seed + 2, 0.5) if bias else None,
                residual=randn((M, N), BF16, seed + 3) if res else None)


DENSE = [  # (M, N, K)
    (1, 64, 128), (1, 512, 4096), (2, 128, 384), (15, 320, 1024), (16, 64, 8192), (17, 192, 128),
    (33, 1024, 512), (63, 64, 128), (65, 448, 384), (200, 640, 768), (255, 320, 1408),
    (257, 576, 256), (513, 1024, 2048), (1025, 512, 8192), (1100, 2112, 256), (2100, 1344, 256),
    (4095, 4096, 1024),
]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K):
    for i, act in enumerate(ACTS):
        bias, res = i % 2 == 0, i in (0, 1, 4)
        print(f"\n[gpu] linear_fp8 {M} {N} {K} {act} bias={bias} res={res} "
              f"{moe.moe_linear_fp8_path(M, N, K, act)}", flush=True)
        x, xs = rows8(M, K, 7)
        p = make(M, N, K, act, bias, res, 100 * i)
        whole = torch.full((M + 2 * GUARD, N), 3.0, dtype=BF16, device="cuda")
        y = whole[GUARD:GUARD + M]
        got = moe.moe_linear_fp8(x, xs, act=act, y=y, **p)
        assert got is y
        near(y, *product64(x, xs, p["w"], p["w_scale"], p["bias"], act, p["residual"]), BF16, act)
        assert (whole[:GUARD] == 3.0).all() and (whole[-GUARD:] == 3.0).all()
        if res:  # accumulated in place
            acc = p["residual"].clone()
            moe.moe_linear_fp8(x, xs, p["w"], p["w_scale"], p["bias"], act, residual=acc, y=acc)
            assert torch.equal(acc, y)


GROUPED = [  # (E, T, k, N, K, segments, rows past the last segment)
    (1, 3, 1, 64, 128, "even", 0), (8, 4, 2, 128, 256, "ragged", 0), (128, 16, 8, 256, 512, "ragged", 0),
    (128, 1, 8, 64, 4096, "ragged", 0), (16, 40, 4, 320, 384, "one", 0), (5, 37, 3, 192, 384, "even", 9),
    (256, 100, 8, 64, 128, "ragged", 33), (8, 700, 2, 448, 640, "ragged", 0), (7, 300, 2, 256, 8192, "one", 5),
    (16, 1024, 4, 512, 256, "ragged", 100), (64, 2048, 6, 320, 512, "ragged", 0),
    (4, 513, 1, 1344, 256, "even", 0), (3, 20, 2, 64, 128, "none", 40), (8, 4096, 2, 256, 4096, "even", 0),
    (2, 8, 8, 128, 128, "ragged", 0), (8, 4096, 2, 2112, 256, "ragged", 11),
]


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "E%d_T%d_k%d_%dx%d_%s_%d" % c)
def test_grouped(case):
    E, T, k, N, K, kind, past = case
    rng = np.random.default_rng(E * 1000 + T)
    rows = T * k
    counts = segments(kind, E, rows - past, rng)
    off = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    perm_h = rng.permutation(rows)
    for i, act in enumerate(ACTS):
        gather, bias, res = i % 2 == 0, i in (1, 2, 4), i in (0, 3, 4)
        print(f"\n[gpu] grouped_fp8 {case} {act} gather={gather} bias={bias} res={res} "
              f"{moe.moe_linear_fp8_path(rows, N, K, act, E)}", flush=True)
        x, xs = rows8(T if gather else rows, K, 7)
        p = make(rows, N, K, act, bias, res, 100 * i, E)
        perm = torch.tensor(perm_h, dtype=torch.int32, device="cuda") if gather else None
        y = torch.full((rows, N), 3.0, dtype=BF16, device="cuda")
        got = moe.moe_linear_grouped_fp8(x, xs, offsets, act=act, perm=perm, k=k, rows=rows, y=y, **p)
        assert got is y
        assert (y[off[-1]:] == 3.0).all(), "rows past the last segment were written"
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if lo == hi:
                continue
            at = torch.tensor(perm_h[lo:hi] // k, device="cuda") if gather else slice(lo, hi)
            near(y[lo:hi], *product64(x[at], xs[:, at], p["w"][e], p["w_scale"][e],
                                      p["bias"][e] if bias else None, act,
                                      p["residual"][lo:hi] if res else None), BF16, f"{act} expert {e}")
        if res:
            acc = p["residual"].clone()
            moe.moe_linear_grouped_fp8(x, xs, offsets, p["w"], p["w_scale"], p["bias"], act, residual=acc,
                                       perm=perm, k=k, rows=rows, y=acc)
            assert torch.equal(acc[:off[-1]], y[:off[-1]])
            assert torch.equal(acc[off[-1]:], p["residual"][off[-1]:])


def test_every_code():
    """All 256 codes against each other, one product a row and column: the value of every
    finite code, and NaN where one of the two is."""
    print("\n[gpu] linear_fp8 codes", flush=True)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    x = torch.zeros((256, 128), dtype=torch.uint8, device="cuda")
    w = torch.zeros((256, 128), dtype=torch.uint8, device="cuda")
    for at in (0, 17, 63, 64, 127):
        x.zero_(), w.zero_()
        x[:, at], w[:, at] = codes, codes
        one = torch.ones((1, 256), device="cuda")
        y = moe.moe_linear_fp8(x.view(FP8), one, w.view(FP8), torch.ones((2, 1), device="cuda"))
        v = codes.view(FP8).double()
        want = v[:, None] * v[None, :]
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(y), nan)
        assert torch.equal(y.double()[~nan], want[~nan].to(BF16).double())


def test_bad_offsets_and_perm_stay_inside():
    """Offsets and permutations out of range are clamped: no access leaves the buffers."""
    print("\n[gpu] grouped_fp8 bad offsets", flush=True)
    for T in (32, 600, 9000):
        E, k, N, K = 4, 2, 128, 128
        x, xs = rows8(T, K, 1)
        w, ws = weight8((E,), N, K, 2)
        perm = torch.full((T * k,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        perm[::2] = -5
        off = torch.tensor([-7, 10, 5, 2 ** 31 - 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        moe.moe_linear_grouped_fp8(x, xs, off, w, ws, perm=perm, k=k)
        torch.cuda.synchronize()


def test_overlapping_offsets_stay_in_the_workspace():
    """Offsets that go back and forth name more tiles than rows can have; no K slice's
    partial tile may land past the workspace."""
    print("\n[gpu] grouped_fp8 overlapping offsets", flush=True)
    E, rows, N, K = 4, 600, 192, 8192
    assert moe.moe_linear_fp8_path(rows, N, K, "none", E)[1] > 1
    x, xs = rows8(rows, K, 1)
    w, ws = weight8((E,), N, K, 2)
    off = torch.tensor([0, rows] * (E // 2) + [rows], dtype=torch.int32, device="cuda")
    need = moe.moe_linear_grouped_fp8_workspace_bytes(E, rows, N, K, "none")
    assert need > 0
    buf = torch.full((need + (8 << 20),), 77, dtype=torch.uint8, device="cuda")
    y = torch.full((rows + 64, N), 3.0, dtype=BF16, device="cuda")
    moe.moe_linear_grouped_fp8(x, xs, off, w, ws, y=y[:rows], ws=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 77).all() and (y[rows:] == 3.0).all()


def test_nan_rows_stay_alone():
    """A NaN code, or a scale that is NaN or infinite, reaches only its own row's outputs."""
    print("\n[gpu] linear_fp8 nan rows", flush=True)
    for M in (5, 40, 700):
        x, xs = rows8(M, 256, 1)
        w, ws = weight8((2,), 128, 256, 2)
        want = moe.moe_linear_fp8(x, xs, w, ws, act="swiglu")
        x.view(torch.uint8)[2, 200] = 0x7f
        xs[1, 4] = float("nan")
        xs[0, 3] = float("inf")
        got = moe.moe_linear_fp8(x, xs, w, ws, act="swiglu")
        keep = [i for i in range(M) if i not in (2, 3, 4)]
        assert torch.equal(got[keep], want[keep])
        assert torch.isnan(got[2]).all() and torch.isnan(got[4]).all()


def test_streams_and_two_graphs():
    """Captured graphs with workspaces of their own, replayed in turn with eager calls
    between; a call on another stream; repeated calls, same bits."""
    print("\n[gpu] linear_fp8 graphs", flush=True)
    cases = []
    for M, N, K in ((1, 512, 4096), (64, 256, 2048), (1200, 512, 2048), (4000, 4096, 256)):
        x, xs = rows8(M, K, 1)
        w, ws = weight8((2,), N, K, 2)
        moe.moe_linear_fp8(x, xs, w, ws, act="swiglu")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = moe.moe_linear_fp8(x, xs, w, ws, act="swiglu")
        cases.append((x, xs, w, ws, g, y))
    side = torch.cuda.Stream()
    for rep in range(4):
        for i, (x, xs, w, ws, g, y) in enumerate(cases):
            nx, ns = rows8(*x.shape, 50 + 3 * rep + i)
            x.copy_(nx), xs.copy_(ns)
            g.replay()
        for x, xs, w, ws, g, y in cases:
            want = moe.moe_linear_fp8(x, xs, w, ws, act="swiglu")
            side.wait_stream(torch.cuda.current_stream())
            other = moe.moe_linear_fp8(x, xs, w, ws, act="swiglu", stream=side)
            side.synchronize()
            assert torch.equal(want, y) and torch.equal(want, other), rep


def test_quantized_block_of_experts():
    """The operators in a row, as a gated block of experts runs them: quantise the tokens
    and the weights, up through the permutation, quantise, down; against the dequantised
    operands in 64 bits. Each step's input is the kernel's own, so each is held to its own
    bound."""
    print("\n[gpu] experts in 8 bits", flush=True)
    E, T, k, H, F = 16, 96, 4, 512, 320 * 2
    x = randn((T, H), BF16, 1)
    up, us = moe.moe_quantize_weight(randn((E, 2, F, H), BF16, 2, H ** -0.5))
    down, ds = moe.moe_quantize_weight(randn((E, H, F), BF16, 3, F ** -0.5))
    idx, wgt = moe.moe_route_grouped(x, randn((E, H), BF16, 4, H ** -0.5), None, k)
    d = moe.moe_dispatch(idx, x, E, gather=False)
    q, s = moe.moe_quantize(x)
    a = moe.moe_linear_grouped_fp8(q, s, d["offsets"], up, us, act="swiglu", perm=d["perm"], k=k)
    aq, as_ = moe.moe_quantize(a)
    ys = moe.moe_linear_grouped_fp8(aq, as_, d["offsets"], down, ds)
    out = moe.moe_combine(ys, d["inv"], wgt)
    off, perm = d["offsets"].tolist(), d["perm"].long()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        at = perm[lo:hi] // k
        near(a[lo:hi], *product64(q[at], s[:, at], up[e], us[e], None, "swiglu", None), BF16, "up")
        near(ys[lo:hi], *product64(aq[lo:hi], as_[:, lo:hi], down[e], ds[e], None, "none", None), BF16, "down")
    want = (wgt.double()[:, :, None] * ys.double()[d["inv"].long()].view(T, k, H)).sum(1)
    assert ((out.double() - want).abs() <= HALF[BF16] * 1.02 * want.abs() + 1e-5).all()
