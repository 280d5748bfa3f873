"""GPU: the 8-bit products on every kernel and number of K slices that their planner picks,
with operands past 4 GiB, on streams other than their own, and on kernels of one path whose
results have to be the same. Tolerances as tests/test_gpu_linear_fp8.py."""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_amd as moe
from tests.test_gpu_linear import near, segments
from tests.test_gpu_linear_fp8 import BF16, FP8, make, product64, rows8, weight8
from tests.test_linear_fp8_path import SHAPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "%d_%d_%d_%s_%s_%s_%d" % c)
def test_paths(case):
    M, N, K, act, E, path, slices = case
    print(f"\n[gpu] linear_fp8 path {case}", flush=True)
    x, xs = rows8(M, K, 3)
    p = make(M, N, K, act, True, M % 2 == 1, 5, E)
    y = torch.full((M + 64, N), 3.0, dtype=BF16, device="cuda")
    if E is None:
        moe.moe_linear_fp8(x, xs, act=act, y=y[:M], **p)
        near(y[:M], *product64(x, xs, p["w"], p["w_scale"], p["bias"], act, p["residual"]), BF16, act)
        again = moe.moe_linear_fp8(x, xs, act=act, **p)
    else:
        off = np.concatenate([[0], np.cumsum(segments("ragged", E, M, np.random.default_rng(M)))])
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        moe.moe_linear_grouped_fp8(x, xs, offsets, act=act, y=y[:M], **p)
        for e in range(E):
            s = slice(int(off[e]), int(off[e + 1]))
            if s.start < s.stop:
                near(y[s], *product64(x[s], xs[:, s], p["w"][e], p["w_scale"][e], p["bias"][e], act,
                                      None if p["residual"] is None else p["residual"][s]), BF16, f"expert {e}")
        again = moe.moe_linear_grouped_fp8(x, xs, offsets, act=act, **p)
    assert (y[M:] == 3.0).all() and torch.equal(again, y[:M])


def test_rows_past_4_gib():
    """Token rows past 4 GiB: a gather from there keeps 64-bit addresses."""
    T, K, N, E, rows = (1 << 20) + 640, 4096, 2048, 2, 300
    print(f"\n[gpu] grouped_fp8 gathers from {T} rows", flush=True)
    assert moe.moe_linear_fp8_path(rows, N, K, "none", E)[0] != "rows"
    x = torch.zeros((T, K), dtype=torch.uint8, device="cuda").view(FP8)
    xs = torch.ones((K // 128, T), device="cuda")
    rng = np.random.default_rng(0)
    at = np.concatenate([[0, T - 1, (1 << 20) - 1, 1 << 20], rng.choice(T - 600, rows - 4, replace=False) + 5])
    perm = torch.tensor(rng.permutation(at), dtype=torch.int32, device="cuda")
    some, scale = rows8(rows, K, 1)
    x.view(torch.uint8)[perm.long()] = some.view(torch.uint8)
    xs[:, perm.long()] = scale
    w, ws = weight8((E,), N, K, 2)
    offsets = torch.tensor([0, 100, rows], dtype=torch.int32, device="cuda")
    y = moe.moe_linear_grouped_fp8(x, xs, offsets, w, ws, perm=perm, k=1, rows=rows)
    for e, s in enumerate((slice(0, 100), slice(100, rows))):
        near(y[s], *product64(some[s], scale[:, s], w[e], ws[e], None, "none", None), BF16, f"expert {e}")


def test_weights_past_4_gib():
    """One matrix of weights past 4 GiB, and experts that start past it."""
    M, K = 40, 4096
    N = (1 << 20) + 64
    print(f"\n[gpu] linear_fp8 weights of {N} x {K}", flush=True)
    x, xs = rows8(M, K, 1)
    w = torch.zeros((N, K), dtype=torch.uint8, device="cuda").view(FP8)
    ws = torch.ones((-(-N // 128), K // 128), device="cuda")
    part, scale = weight8((), 192, K, 2)
    for at in (0, (1 << 19), N - 192):  # the last two blocks of scales hold its last 192 rows
        at = at // 128 * 128
        n = min(192, N - at)
        w.view(torch.uint8)[at:at + n] = part.view(torch.uint8)[:n]
        ws[at // 128:at // 128 + -(-n // 128)] = scale[:-(-n // 128)]
    y = moe.moe_linear_fp8(x, xs, w, ws)
    for at in (0, (1 << 19), N - 192):
        at = at // 128 * 128
        n = min(192, N - at)
        near(y[:, at:at + n], *product64(x, xs, part[:n], scale[:-(-n // 128)], None, "none", None), BF16, str(at))
    assert (y[:, 192:1 << 19] == 0).all()
    del w, ws, y
    E, N, rows = 40, 2048, 400
    w, ws = weight8((E, 2), N // 2 * 7, K, 3)  # 40 x 2 x 7168 x 4096
    assert w.numel() > 1 << 31
    offsets = torch.arange(E + 1, dtype=torch.int32, device="cuda") * (rows // E)
    x, xs = rows8(rows, K, 4)
    y = moe.moe_linear_grouped_fp8(x, xs, offsets, w, ws, act="swiglu")
    for e in (0, E // 2, E - 1):
        s = slice(e * 10, e * 10 + 10)
        near(y[s], *product64(x[s], xs[:, s], w[e], ws[e], None, "swiglu", None), BF16, f"expert {e}")


def test_rows_do_not_depend_on_their_place():
    """A row's output is the same wherever in the buffer it lies and whatever lies beside it,
    for one size of call: row pairs go round the waves of a tile."""
    print("\n[gpu] linear_fp8 places", flush=True)
    for M, N, K in ((300, 704, 256), (2048, 4160, 1024), (8200, 4160, 1024)):
        x, xs = rows8(M, K, 1)
        w, ws = weight8((), N, K, 2)
        y = moe.moe_linear_fp8(x, xs, w, ws)
        order = torch.randperm(M, generator=torch.Generator().manual_seed(0)).cuda()
        mixed = moe.moe_linear_fp8(x.view(torch.uint8)[order].view(FP8), xs[:, order].contiguous(), w, ws)
        assert torch.equal(mixed, y[order])
