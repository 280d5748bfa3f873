"""GPU: moe_linear_grouped_fp8 with offsets and permutations out of range, values and
guards. Segment e is [clamp(offsets[e], 0, rows), clamp(offsets[e + 1], its start, rows)),
buffer row p reads token clamp(perm[p], 0, T k - 1) / k: so the call has a defined
result in every row that one segment has, and in a row of two that of either. Bounds as
tests/test_gpu_linear_fp8.py."""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe
from tests.test_gpu_linear import HALF, near
from tests.test_gpu_linear_fp8 import BF16, GUARD, product64, rows8, weight8

pytestmark = pytest.mark.gpu
BIG = 2 ** 31 - 1


@pytest.mark.parametrize("T,N,K,act,paths", [
    (32, 128, 128, "none", ("rows", 1)), (300, 1024, 1024, "none", ("64x64", 1)),
    (300, 192, 8192, "none", ("64x64", 0)), (9000, 128, 128, "swiglu", ("128x128", 1)),
    (9000, 1024, 512, "gelu", ("256x256", 1)),
], ids=lambda v: str(v) if not isinstance(v, tuple) else "%s_%d" % v)
def test_clamped(T, N, K, act, paths):
    E, k = 4, 2
    rows, name, slices = T * k, *moe.moe_linear_fp8_path(T * k, N, K, act, E)
    print(f"\n[gpu] grouped_fp8 clamped {T} {N} {K} {act} {name} {slices}", flush=True)
    assert name == paths[0] and (slices == paths[1] or (paths[1] == 0 and slices > 1))
    two = (2,) if act == "swiglu" else ()
    x, xs = rows8(T, K, 1)
    w, ws = weight8((E, *two), N, K, 2)
    perm = torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).contiguous()
    perm[::3], perm[1::7] = BIG, -5
    off = torch.tensor([-7, 10, 5, BIG, BIG], dtype=torch.int32, device="cuda")
    need = moe.moe_linear_grouped_fp8_workspace_bytes(E, rows, N, K, act)
    buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    whole = torch.full((rows + 2 * GUARD, N), 3.0, dtype=BF16, device="cuda")
    y = whole[GUARD:GUARD + rows]
    moe.moe_linear_grouped_fp8(x, xs, off, w, ws, act=act, perm=perm, k=k, y=y, ws=buf[:need] if need else None)
    assert (whole[:GUARD] == 3.0).all() and (whole[-GUARD:] == 3.0).all() and (buf[need:] == 77).all()
    at = perm.long().clamp(0, rows - 1) // k
    e0 = product64(x[at[:10]], xs[:, at[:10]], w[0], ws[0], None, act, None)       # [0, 10)
    e2 = product64(x[at[5:]], xs[:, at[5:]], w[2], ws[2], None, act, None)         # [5, rows)
    near(y[:5], e0[0][:5], e0[1][:5], BF16, "first segment")
    near(y[10:], e2[0][5:], e2[1][5:], BF16, "third segment")
    both = y[5:10].double()
    off_by = [(both - v).abs() - (d + HALF[BF16] * v.abs() * (1 + 2.0 ** -6))
              for v, d in ((e0[0][5:], e0[1][5:]), (e2[0][:5], e2[1][:5]))]
    assert (torch.minimum(*off_by) <= 0).all(), "rows of two segments"


def test_segments_that_end_before_the_buffer():
    """Offsets past the rows at the front leave every row as it was: the first segment
    starts behind the last row."""
    print("\n[gpu] grouped_fp8 nothing left", flush=True)
    E, rows, N, K = 3, 70, 128, 256
    x, xs = rows8(rows, K, 1)
    w, ws = weight8((E,), N, K, 2)
    for off in ([BIG, 0, 5, 3], [rows] * 4, [0, -1, -2, -3], [-9, -9, -9, -9]):
        y = torch.full((rows, N), 3.0, dtype=BF16, device="cuda")
        moe.moe_linear_grouped_fp8(x, xs, torch.tensor(off, dtype=torch.int32, device="cuda"), w, ws, y=y)
        lo, hi = (0, 5) if off[0] == BIG else (0, 0)  # its second segment is [0, 5)
        assert (y[hi:] == 3.0).all() and (y[lo:hi] != 3.0).any(1).all()
