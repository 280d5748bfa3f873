"""GPU: every kernel of moe_linear and moe_linear_grouped, by the path that the sizes
take. The other product tests choose sizes; these choose the path and assert it, so
that another estimate of the paths' times cannot leave a kernel without a test.
Reference and tolerance: tests/test_gpu_linear.py."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_amd as moe
from tests.test_gpu_linear import BOTH, ID, make, near, product64, randn

pytestmark = pytest.mark.gpu
PLAIN, GATED = ("none", "gelu", "silu"), ("geglu", "swiglu")
BF16, FP32 = torch.bfloat16, torch.float32
GUARD = 64  # rows around an output that nothing may write


def path_of(M, N, K, act, dtype, E=None):
    return moe.moe_linear_path(M, N, K, act, int(dtype == BF16), E)


def guarded(M, N, dtype):
    """(whole buffer of threes, its M rows in the middle)."""
    whole = torch.full((M + 2 * GUARD, N), 3.0, dtype=dtype, device="cuda")
    return whole, whole[GUARD:GUARD + M]


def guards_kept(whole):
    return bool((whole[:GUARD] == 3.0).all() and (whole[-GUARD:] == 3.0).all())


DENSE = [  # (path, slices, M, N, K, acts, type)
    ("rows", 1, 17, 64, 64, PLAIN, BF16), ("rows", 1, 19, 192, 320, GATED, BF16),
    ("tiles", 1, 901, 960, 64, PLAIN, BF16), ("tiles", 2, 257, 2112, 2048, PLAIN, BF16),
    ("tiles", 4, 201, 1088, 2048, PLAIN, BF16), ("tiles", 8, 2600, 64, 2112, PLAIN, BF16),
    ("tiles", 16, 1300, 64, 4096, PLAIN, BF16),
    ("tiles", 1, 1303, 448, 64, GATED, BF16), ("tiles", 2, 201, 1344, 2048, GATED, BF16),
    ("tiles", 4, 65, 1344, 2112, GATED, BF16), ("tiles", 8, 1701, 64, 2048, GATED, BF16),
    ("256x128", 1, 1101, 4160, 320, PLAIN, BF16), ("256x128", 1, 1701, 2112, 192, GATED, BF16),
    ("256x256", 1, 2601, 4160, 128, PLAIN, BF16), ("256x256", 1, 1301, 4160, 128, GATED, BF16),
    ("256x128", 4, 2101, 320, 8192, PLAIN, BF16), ("256x128", 2, 1025, 2112, 8192, PLAIN, BF16),
    ("256x128", 7, 515, 704, 14336, PLAIN, BF16), ("256x128", 4, 701, 448, 8192, GATED, BF16),
    ("256x256", 3, 257, 8256, 8192, PLAIN, BF16), ("256x256", 3, 257, 4160, 8192, GATED, BF16),
    ("tiles", 1, 17, 64, 64, PLAIN, FP32), ("tiles", 2, 33, 192, 512, GATED, FP32),
    ("tiles", 4, 17, 64, 1024, PLAIN, FP32), ("tiles", 8, 65, 64, 2112, GATED, FP32),
    ("tiles", 16, 17, 64, 4096, PLAIN, FP32), ("tiles", 1, 1301, 2112, 128, PLAIN, FP32),
]


@pytest.mark.parametrize("case", DENSE, ids=lambda c: "%s_%d_%dx%dx%d_%s_%s" % (*c[:5], c[5][-1], ID(c[6])))
def test_dense(case):
    path, slices, M, N, K, acts, dtype = case
    for i, act in enumerate(acts):
        assert path_of(M, N, K, act, dtype) == (path, slices)
        bias, res = i != 1, i != 0
        print(f"\n[gpu] path {case[:5]} {act} bias={bias} res={res} {dtype}", flush=True)
        x = randn((M, K), dtype, 7)
        p = make(M, N, K, act, bias, res, dtype, 100 * i)
        whole, y = guarded(M, N, dtype)
        moe.moe_linear(x, act=act, y=y, **p)
        near(y, *product64(x, p["w"], p["bias"], act, p["residual"], dtype), dtype, act)
        assert guards_kept(whole)
        if res:
            acc = p["residual"].clone()
            moe.moe_linear(x, p["w"], p["bias"], act, residual=acc, y=acc)
            assert torch.equal(acc, y)


GROUPED = [  # (path, slices, E, rows, N, K, acts, type)
    ("rows", 1, 8, 37, 64, 64, PLAIN, BF16), ("rows", 1, 8, 37, 64, 192, GATED, BF16),
    ("tiles", 1, 8, 2100, 448, 64, PLAIN, BF16), ("tiles", 2, 3, 65, 4160, 2048, PLAIN, BF16),
    ("tiles", 4, 3, 701, 320, 2048, PLAIN, BF16), ("tiles", 8, 3, 2601, 64, 2048, PLAIN, BF16),
    ("tiles", 16, 3, 1300, 64, 4096, PLAIN, BF16),
    ("tiles", 1, 3, 3100, 192, 64, GATED, BF16), ("tiles", 2, 8, 18, 960, 2048, GATED, BF16),
    ("tiles", 4, 3, 600, 192, 2112, GATED, BF16), ("tiles", 8, 8, 900, 64, 4096, GATED, BF16),
    ("256x128", 1, 3, 901, 4160, 704, PLAIN, BF16), ("256x128", 1, 8, 2601, 2112, 512, PLAIN, BF16),
    ("256x128", 1, 3, 3101, 1088, 320, GATED, BF16), ("256x128", 1, 8, 2601, 960, 512, GATED, BF16),
    ("256x256", 1, 8, 1701, 4160, 320, PLAIN, BF16), ("256x256", 1, 8, 2601, 2112, 192, GATED, BF16),
    ("256x128", 0, 3, 2101, 320, 8192, PLAIN, BF16), ("256x128", 0, 3, 1701, 192, 8192, GATED, BF16),
    ("256x256", 0, 3, 515, 2112, 12352, PLAIN, BF16), ("256x256", 0, 3, 515, 1088, 12352, GATED, BF16),
    ("tiles", 1, 8, 17, 64, 64, GATED, FP32), ("tiles", 2, 8, 65, 64, 512, PLAIN, FP32),
    ("tiles", 4, 3, 17, 64, 1024, GATED, FP32), ("tiles", 8, 3, 33, 64, 2048, PLAIN, FP32),
    ("tiles", 16, 3, 17, 64, 4096, GATED, FP32), ("tiles", 1, 8, 1301, 1088, 128, PLAIN, FP32),
]


def ragged(E, rows, past, seed):
    """Offsets of E segments in rows - past rows: an empty one, a long one, odd ones."""
    rng = np.random.default_rng(seed)
    p = rng.random(E) ** 2 + 0.05
    p[E // 2] = 0
    p[E - 1] += 1
    return np.concatenate([[0], np.cumsum(rng.multinomial(rows - past, p / p.sum()))])


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "%s_%d_E%d_%dx%dx%d_%s_%s" % (*c[:6], c[6][-1], ID(c[7])))
def test_grouped(case):
    path, slices, E, rows, N, K, acts, dtype = case
    k = 3
    T, past = -(-rows // k), 5
    off = ragged(E, rows, past, rows + N)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    perm_h = np.random.default_rng(rows).permutation(T * k)
    last = int(off[-1])
    for i, act in enumerate(acts):
        assert path_of(rows, N, K, act, dtype, E) == (path, slices)
        gather, bias, res = i != 1, i != 1, i != 0
        print(f"\n[gpu] path {case[:6]} {act} gather={gather} bias={bias} res={res} {dtype}", flush=True)
        x = randn((T if gather else rows, K), dtype, 7)
        p = make(rows, N, K, act, bias, res, dtype, 100 * i, E)
        perm = torch.tensor(perm_h, dtype=torch.int32, device="cuda") if gather else None
        whole, y = guarded(rows, N, dtype)
        moe.moe_linear_grouped(x, offsets, act=act, perm=perm, k=k, rows=rows, y=y, **p)
        assert guards_kept(whole) and (y[last:] == 3.0).all()
        want = torch.zeros((last, N), dtype=torch.float64, device="cuda")
        err = torch.zeros_like(want)
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if lo == hi:
                continue
            xs = x[torch.tensor(perm_h[lo:hi] // k, device="cuda")] if gather else x[lo:hi]
            want[lo:hi], err[lo:hi] = product64(xs, p["w"][e], p["bias"][e] if bias else None, act,
                                                p["residual"][lo:hi] if res else None, dtype)
        near(y[:last], want, err, dtype, act)
        if res:
            acc = p["residual"].clone()
            moe.moe_linear_grouped(x, offsets, p["w"], p["bias"], act, residual=acc, perm=perm, k=k,
                                   rows=rows, y=acc)
            assert torch.equal(acc[:last], y[:last]) and torch.equal(acc[last:], p["residual"][last:])


CLAMPED = [  # (path, slices, E, T, k, N, K, act, type)
    ("rows", 1, 4, 32, 2, 128, 128, "none", BF16), ("tiles", 8, 4, 1301, 2, 64, 2048, "none", BF16),
    ("tiles", 1, 4, 2000, 2, 192, 64, "swiglu", BF16), ("256x128", 1, 4, 451, 2, 4160, 704, "none", BF16),
    ("256x256", 1, 4, 1300, 2, 4160, 192, "none", BF16), ("256x256", 1, 4, 1300, 2, 2112, 192, "swiglu", BF16),
    ("256x128", 0, 4, 1050, 2, 320, 8192, "none", BF16), ("256x256", 0, 4, 258, 2, 2112, 8192, "swiglu", BF16),
    ("tiles", 8, 4, 17, 2, 64, 2048, "none", FP32), ("tiles", 1, 4, 600, 2, 1088, 128, "swiglu", FP32),
]


@pytest.mark.parametrize("case", CLAMPED, ids=lambda c: "%s_%d_%s_%s" % (c[0], c[1], c[7], ID(c[8])))
def test_offsets_and_perm_out_of_range(case):
    """Offsets and perm entries out of range count as clamped ones: the rows that one
    segment then holds have its product, and nothing else is written."""
    path, slices, E, T, k, N, K, act, dtype = case
    print(f"\n[gpu] clamped {case}", flush=True)
    rows = T * k
    assert path_of(rows, N, K, act, dtype, E) == (path, slices)
    two = (2,) if act in GATED else ()
    x, w = randn((T, K), dtype, 1), randn((E, *two, N, K), dtype, 2, K ** -0.5)
    perm = torch.arange(rows, dtype=torch.int32, device="cuda")
    perm[::3], perm[1::3] = 2 ** 31 - 1, -5
    big = 2 ** 31 - 1
    whole, y = guarded(rows, N, dtype)
    # segments [0, 10), none, [5, rows), none: rows 5 to 9 are in two
    off = torch.tensor([-7, 10, 5, big, big], dtype=torch.int32, device="cuda")
    moe.moe_linear_grouped(x, off, w, act=act, perm=perm, k=k, y=y)
    assert guards_kept(whole)
    src = x[perm.clamp(0, rows - 1).long() // k]
    for lo, hi, e in ((0, 5, 0), (10, rows, 2)):
        near(y[lo:hi], *product64(src[lo:hi], w[e], None, act, None, dtype), dtype, f"rows {lo} to {hi}")
    # nothing in any segment: nothing written
    whole.fill_(3.0)
    for o in ([0] * 5, [-1, -9, -big, -2, -3], [big] * 5, [rows, 3, 2, 1, 0]):
        moe.moe_linear_grouped(x, torch.tensor(o, dtype=torch.int32, device="cuda"), w, act=act, perm=perm,
                               k=k, y=y)
        torch.cuda.synchronize()
        assert (whole == 3.0).all(), o


OVERLAPPING = [  # (path, slices, rows, N, K, act, type), 16 experts
    ("tiles", 16, 1300, 64, 4096, "none", BF16), ("tiles", 2, 200, 960, 2048, "none", BF16),
    ("tiles", 8, 900, 64, 4096, "swiglu", BF16), ("256x128", 1, 5000, 1088, 512, "none", BF16),
    ("256x128", 1, 5000, 448, 704, "swiglu", BF16), ("256x256", 1, 5000, 4160, 64, "swiglu", BF16),
    ("256x128", 0, 4000, 192, 9216, "none", BF16), ("256x128", 0, 4000, 64, 12352, "swiglu", BF16),
    ("256x256", 0, 4000, 448, 9216, "none", BF16), ("256x256", 0, 515, 1344, 8192, "swiglu", BF16),
]


@pytest.mark.parametrize("case", OVERLAPPING, ids=lambda c: "%s_%d_%s_%s" % (*c[:2], *map(ID, c[5:])))
def test_overlapping_offsets(case):
    """Offsets that go back and forth name more tiles than a launch has room for: no
    partial tile or table entry lands past the workspace, no row outside the buffer."""
    path, slices, rows, N, K, act, dtype = case
    print(f"\n[gpu] overlapping {case}", flush=True)
    E = 16
    assert path_of(rows, N, K, act, dtype, E) == (path, slices)
    two = (2,) if act in GATED else ()
    x, w = randn((rows, K), dtype, 1), randn((E, *two, N, K), dtype, 2, K ** -0.5)
    off = torch.tensor([0, rows] * (E // 2) + [rows], dtype=torch.int32, device="cuda")
    need = moe.moe_linear_grouped_workspace_bytes(E, rows, N, K, act, int(dtype == BF16))
    assert need > 0
    buf = torch.full((need + (8 << 20),), 77, dtype=torch.uint8, device="cuda")
    whole, y = guarded(rows, N, dtype)
    moe.moe_linear_grouped(x, off, w, act=act, y=y, ws=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 77).all() and guards_kept(whole)


@pytest.mark.parametrize("case", [c for c in DENSE if c[5] is GATED or c[0] == "256x128"],
                         ids=lambda c: "%s_%d_%s_%s" % (*c[:2], c[5][-1], ID(c[6])))
def test_nan_rows_stay_alone(case):
    """A NaN or infinite row reaches only its own outputs."""
    path, slices, M, N, K, acts, dtype = case
    act = acts[-1]
    assert path_of(M, N, K, act, dtype) == (path, slices)
    print(f"\n[gpu] nan rows {case[:5]} {act} {dtype}", flush=True)
    x = randn((M, K), dtype, 1)
    p = make(M, N, K, act, True, False, dtype, 2)
    want = moe.moe_linear(x, act=act, **p)
    bad = sorted({0, 4, M // 2, M - 1})
    for i, r in enumerate(bad):
        x[r, (7 * i) % K] = float("nan") if i % 2 == 0 else float("inf")
    got = moe.moe_linear(x, act=act, **p)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[bad[0]]).all() and torch.isnan(got[bad[-2]]).all()


def test_unused_workspace_is_not_touched():
    """A call that needs no workspace takes any tensor as one, an operand of its own too."""
    print("\n[gpu] unused workspace", flush=True)
    x, w = randn((5, 256), BF16, 1), randn((128, 256), BF16, 2)
    assert moe.moe_linear_workspace_bytes(5, 128, 256, "none", 1) == 0
    keep = x.clone()
    got = moe.moe_linear(x, w, ws=x)
    assert torch.equal(got, moe.moe_linear(x, w)) and torch.equal(x, keep)
