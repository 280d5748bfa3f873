"""The 8-bit products' choice of a path: sizes for every kernel and number of K slices,
dense and over segments. They keep the GPU tests of the paths (test_gpu_linear_fp8_paths.py)
on what they name; a query launches nothing."""
import pytest

import sparse_mixture_experts_05_amd as moe

SHAPES = [  # (M, N, K, act, E or None, path, K slices)
    (16, 192, 512, "none", None, "rows", 1), (64, 320, 512, "swiglu", 16, "rows", 1),
    (300, 704, 256, "silu", None, "64x64", 1), (900, 704, 512, "gelu", 8, "64x64", 1),
    (384, 2048, 8192, "none", None, "64x64", 2), (2067, 256, 8960, "none", 2, "64x64", 2),
    (239, 768, 12928, "swiglu", None, "64x64", 4), (4531, 64, 4864, "none", 2, "64x64", 4),
    (256, 1024, 14336, "none", None, "64x64", 8), (600, 192, 8192, "none", 4, "64x64", 8),
    (32, 192, 8192, "swiglu", None, "64x64", 16), (5, 192, 12032, "swiglu", 8, "64x64", 16),
    (1500, 1600, 384, "geglu", None, "128x128", 1), (2500, 2048, 1024, "none", 6, "128x128", 1),
    (12521, 64, 9344, "swiglu", None, "128x128", 2), (113, 512, 11008, "none", 32, "128x128", 2),
    (9, 4800, 14208, "swiglu", None, "128x128", 4), (2130, 384, 9600, "none", 2, "128x128", 4),
    (35, 4096, 17536, "none", None, "128x128", 8), (503, 896, 18688, "none", 2, "128x128", 8),
    (633, 8512, 768, "swiglu", None, "256x256", 1), (6000, 1024, 512, "swiglu", 8, "256x256", 1),
    (8200, 4160, 1024, "gelu", None, "256x256", 1), (3001, 1088, 256, "geglu", 16, "256x256", 1),
]


@pytest.mark.parametrize("M,N,K,act,E,path,slices", SHAPES)
def test_path(M, N, K, act, E, path, slices):
    assert moe.moe_linear_fp8_path(M, N, K, act, E) == (path, slices)
    ask = moe.moe_linear_fp8_workspace_bytes if E is None else moe.moe_linear_grouped_fp8_workspace_bytes
    need = ask(*(() if E is None else (E,)), M, N, K, act)
    assert (need > 0) == (slices > 1)


def test_all_are_there():
    want = {("rows", 1), ("256x256", 1)} | {("64x64", 2 ** i) for i in range(5)} | {("128x128", 2 ** i) for i in range(4)}
    for grouped in (False, True):
        assert {(p, n) for _, _, _, _, E, p, n in SHAPES if (E is not None) == grouped} == want
