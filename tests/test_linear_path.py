"""The host query of a product's path: refusals, and that it agrees with the workspace
that the product asks for."""
import ctypes

import pytest

import sparse_mixture_experts_05_amd as moe


def query(E=1, rows=32, N=64, K=64, act=0, grouped=0, dt=1, slices=None):
    return moe.lib().moe_linear_path(E, rows, N, K, act, grouped, dt, slices)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), -1), (dict(E=2), -1), (dict(rows=0), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(act=5), -1),
    (dict(act=-1), -1), (dict(grouped=2), -1), (dict(grouped=-1), -1), (dict(dt=2), -1),
    (dict(N=96), -2), (dict(K=32), -2), (dict(E=257, grouped=1), -2), (dict(rows=1 << 22, N=1 << 14), -2),
])
def test_refusals(kw, status):
    assert query(**kw) == status


def test_without_slices():
    n = ctypes.c_int(-1)
    assert query() == query(slices=ctypes.byref(n)) >= 0
    assert n.value == 1


def test_binding():
    assert moe.moe_linear_path(4095, 4096, 4096, "none", 1) == ("256x256", 1)
    assert moe.moe_linear_path(1024, 4096, 4096, "none", 1) == ("256x128", 1)
    assert moe.moe_linear_path(1, 4096, 4096, "none", 1) == ("rows", 1)
    assert moe.moe_linear_path(16, 64, 64, "none", 0)[0] == "tiles"
    with pytest.raises(moe.MoEError):
        moe.moe_linear_path(16, 60, 64, "none", 1)
    with pytest.raises(ValueError, match="act must be one of"):
        moe.moe_linear_path(16, 64, 64, "tanh", 1)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("E", [None, 8])
def test_workspace_agrees(E, act, dt):
    """No workspace for one slice of the rows or tiles path, one for more; the large
    tiles need one for a grouped launch's table and for K slices."""
    for M in (1, 17, 64, 257, 700, 1300, 2600):
        for N in (64, 192, 1088, 4160):
            for K in (64, 704, 2048, 4096):
                path, slices = moe.moe_linear_path(M, N, K, act, dt, E)
                need = (moe.moe_linear_workspace_bytes(M, N, K, act, dt) if E is None else
                        moe.moe_linear_grouped_workspace_bytes(E, M, N, K, act, dt))
                many = slices > 1 or (path.startswith("256") and E is not None)
                assert (need > 0) == many, (M, N, K, path, slices, need)


# (M, N, K, act): a few 256-row tiles whose K slices leave most of the chip idle. The
# other paths were two to four times as fast, with a workspace of at most a few MiB.
FEW_TILES = [
    (1, 64, 8192, "none"), (16, 64, 8192, "none"), (64, 64, 8192, "none"), (256, 64, 8192, "none"),
    (1024, 64, 8192, "none"), (16, 512, 8192, "none"), (128, 512, 8192, "none"), (256, 512, 8192, "none"),
    (64, 1024, 8192, "none"), (256, 1024, 8192, "none"), (64, 512, 14336, "none"), (512, 512, 14336, "none"),
    (128, 1024, 14336, "none"), (256, 64, 28672, "none"), (64, 1024, 28672, "none"), (64, 512, 8192, "swiglu"),
    (256, 512, 8192, "swiglu"),
]


@pytest.mark.parametrize("M,N,K,act", FEW_TILES)
def test_long_k_with_few_tiles(M, N, K, act):
    path, _ = moe.moe_linear_path(M, N, K, act, 1)
    assert path in ("rows", "tiles")
    assert moe.moe_linear_workspace_bytes(M, N, K, act, 1) <= 16 << 20


@pytest.mark.parametrize("M,N,K,path", [
    (256, 4096, 8192, "256x128"), (512, 4096, 8192, "256x128"), (1024, 1024, 8192, "256x128"),
    (2048, 4096, 8192, "256x128"), (256, 4096, 28672, "256x128"), (1024, 512, 28672, "256x128"),
])
def test_long_k_with_enough_tiles(M, N, K, path):
    """Where the large tiles are the fastest, the smaller of the two (their K slices fill
    the chip with half the rows)."""
    assert moe.moe_linear_path(M, N, K, "none", 1)[0] == path


def test_refused_sizes_are_refused_whatever_they_would_cost():
    """Row and column counts whose tiles no int holds, at a K that the large tiles slice."""
    for rows, N, K in ((2 ** 31 - 1, (1 << 18) - 64, 8192), (2 ** 31 - 1, 1 << 17, 8192), (2 ** 31 - 1, 64, 8192)):
        for grouped in (0, 1):
            got = query(E=256 if grouped else 1, rows=rows, N=N, K=K, grouped=grouped)
            assert got == -2
