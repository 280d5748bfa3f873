"""Refusals of the quantisation and of the 8-bit products: host validation only,
nothing is launched."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_05_amd as moe

P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(16)]  # far apart, never dereferenced
ODD16, ODD4 = ctypes.c_void_p(0x10000008), ctypes.c_void_p(0x10000002)


def at(p, n):
    return ctypes.c_void_p(p.value + n)


def quantize(x=P[0], rows=5, K=256, dt=1, q=P[1], s=P[2]):
    return moe.lib().moe_quantize(x, rows, K, dt, q, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(x=ODD16), -1), (dict(q=ODD16), -1),
    (dict(s=ODD4), -1), (dict(rows=0), -1), (dict(rows=-1), -1), (dict(K=0), -1), (dict(dt=2), -1),
    (dict(K=64), -2), (dict(K=192), -2), (dict(rows=2 ** 31 - 1, K=2 ** 20, q=at(P[0], 1 << 55), s=at(P[0], 1 << 60)), -2),
    (dict(q=P[0]), -1), (dict(q=at(P[0], 5 * 256 * 2 - 16)), -1), (dict(s=at(P[0], 16)), -1),
    (dict(s=at(P[1], 5 * 256 - 4)), -1), (dict(s=at(P[1], -36)), -1),
])
def test_quantize_refusals(kw, status):
    assert quantize(**kw) == status


def weight(w=P[0], count=3, N=192, K=256, dt=1, q=P[1], s=P[2]):
    return moe.lib().moe_quantize_weight(w, count, N, K, dt, q, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(w=ODD16), -1), (dict(count=0), -1),
    (dict(N=0), -1), (dict(K=-128), -1), (dict(dt=-1), -1), (dict(N=100), -2), (dict(K=64), -2),
    (dict(q=P[0]), -1), (dict(s=at(P[1], 3 * 192 * 256 - 4)), -1), (dict(s=at(P[1], -44)), -1),
    (dict(count=1 << 24, N=128, K=128, q=at(P[0], 1 << 45), s=at(P[0], 1 << 50)), -2),
])
def test_quantize_weight_refusals(kw, status):
    assert weight(**kw) == status


M, N, K, E = 32, 192, 256, 8
X, XS, W, WS, B, RES, Y, SCRATCH, PERM, OFF = P[:10]


def linear(x=X, xs=XS, w=W, ws=WS, b=B, act=4, res=RES, M=M, N=N, K=K, y=Y, scratch=SCRATCH, n=1 << 40):
    return moe.lib().moe_linear_fp8(x, xs, w, ws, b, act, res, M, N, K, y, scratch, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(xs=None), -1), (dict(w=None), -1), (dict(ws=None), -1), (dict(y=None), -1),
    (dict(act=5), -1), (dict(act=-1), -1), (dict(M=0), -1), (dict(N=0), -1), (dict(K=0), -1),
    (dict(x=ODD16), -1), (dict(w=ODD16), -1), (dict(b=ODD16), -1), (dict(res=ODD16), -1),
    (dict(y=ODD16), -1), (dict(scratch=ODD16), -1), (dict(xs=ODD4), -1), (dict(ws=ODD4), -1),
    (dict(N=96), -2), (dict(K=64), -2), (dict(M=2 ** 31 - 1, N=1 << 24), -2),
    (dict(y=at(X, M * K - 16)), -1), (dict(y=at(X, 16 - M * N * 2)), -1),
    (dict(y=at(XS, M * K // 128 * 4 - 16)), -1), (dict(y=at(W, 2 * N * K - 16)), -1),
    (dict(y=at(WS, 2 * 2 * 2 * 4 - 16)), -1), (dict(y=at(B, 2 * N * 2 - 16)), -1), (dict(y=at(RES, 16)), -1),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def test_linear_workspace():
    need = moe.lib().moe_linear_fp8_workspace_bytes(M, N, 8192, 4)
    assert need > 0
    assert linear(K=8192, scratch=None) == -3 and linear(K=8192, n=need - 1) == -3
    for p in (X, XS, W, WS, B, RES, Y):
        assert linear(K=8192, scratch=p) == -1
        assert linear(K=8192, scratch=at(p, 16 - need)) == -1
    assert moe.lib().moe_linear_fp8_workspace_bytes(M, N, 8192 + 64, 4) == 0


def grouped(x=X, xs=XS, perm=PERM, k=2, T=16, off=OFF, E=E, rows=32, w=W, ws=WS, b=B, act=4, res=RES, N=N,
            K=K, y=Y, scratch=SCRATCH, n=1 << 40):
    return moe.lib().moe_linear_grouped_fp8(x, xs, perm, k, T, off, E, rows, w, ws, b, act, res, N, K, y,
                                            scratch, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(off=None), -1), (dict(x=None), -1), (dict(xs=None), -1), (dict(ws=None), -1), (dict(E=0), -1),
    (dict(rows=0), -1), (dict(T=0), -1), (dict(k=0), -1), (dict(k=9), -2), (dict(rows=33), -2),
    (dict(E=257), -2), (dict(N=32), -2), (dict(K=192), -2), (dict(act=7), -1), (dict(y=PERM), -1),
    (dict(y=at(OFF, 16)), -1), (dict(y=at(XS, 16 * 2 * 4 - 16)), -1),
    (dict(y=at(WS, E * 2 * 2 * 2 * 4 - 16)), -1), (dict(y=at(W, E * 2 * N * K - 16)), -1),
])
def test_grouped_refusals(kw, status):
    assert grouped(**kw) == status


def test_paths():
    """Sizes that are refused have no path; the query needs no GPU."""
    L = moe.lib()
    assert L.moe_linear_fp8_path(1, 8, 64, 64, 0, 0, None) == -2
    assert L.moe_linear_fp8_path(2, 8, 64, 128, 0, 0, None) == -1
    assert L.moe_linear_fp8_path(1, 8, 64, 128, 0, 2, None) == -1
    assert L.moe_linear_fp8_path(1, 8, 64, 128, 0, 0, None) >= 0
    with pytest.raises(moe.MoEError):
        moe.moe_linear_fp8_path(8, 64, 100, "none")


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def f8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


def f32(*shape):
    return t(*shape, dtype=torch.float32)


I5 = t(5, dtype=torch.int32)
BAD = [
    ("x must have 2 dimensions", lambda: moe.moe_quantize(t(128))),
    ("unsupported dtype", lambda: moe.moe_quantize(t(2, 128, dtype=torch.float16))),
    ("q must be torch.float8_e4m3fn", lambda: moe.moe_quantize(t(2, 128), q=t(2, 128, dtype=torch.uint8))),
    ("scale has shape", lambda: moe.moe_quantize(t(2, 256), scale=f32(2, 1))),
    ("must be contiguous", lambda: moe.moe_quantize(t(128, 128).t())),
    ("must be GPU tensors", lambda: moe.moe_quantize(t(2, 128))),
    ("two dimensions or more", lambda: moe.moe_quantize_weight(t(128))),
    ("scale has shape", lambda: moe.moe_quantize_weight(t(3, 192, 128), scale=f32(3, 1, 1))),
    ("must be GPU tensors", lambda: moe.moe_quantize_weight(t(3, 192, 128))),
    ("x must be torch.float8_e4m3fn", lambda: moe.moe_linear_fp8(t(2, 128), f32(1, 2), f8(64, 128), f32(1, 1))),
    ("w must be torch.float8_e4m3fn", lambda: moe.moe_linear_fp8(f8(2, 128), f32(1, 2), t(64, 128), f32(1, 1))),
    ("x_scale has shape", lambda: moe.moe_linear_fp8(f8(2, 128), f32(2, 1), f8(64, 128), f32(1, 1))),
    ("x_scale is required", lambda: moe.moe_linear_fp8(f8(2, 128), None, f8(64, 128), f32(1, 1))),
    ("w_scale is required", lambda: moe.moe_linear_fp8(f8(2, 128), f32(1, 2), f8(64, 128), None)),
    ("w_scale has shape", lambda: moe.moe_linear_fp8(f8(2, 128), f32(1, 2), f8(192, 128), f32(1, 1))),
    ("w must have 3 dimensions", lambda: moe.moe_linear_fp8(
        f8(2, 128), f32(1, 2), f8(64, 128), f32(1, 1), act="swiglu")),
    ("bias must be torch.bfloat16", lambda: moe.moe_linear_fp8(
        f8(2, 128), f32(1, 2), f8(64, 128), f32(1, 1), f32(64))),
    ("residual has shape", lambda: moe.moe_linear_fp8(
        f8(2, 128), f32(1, 2), f8(64, 128), f32(1, 1), residual=t(1, 64))),
    ("act must be one of", lambda: moe.moe_linear_fp8(f8(2, 128), f32(1, 2), f8(64, 128), f32(1, 1), act="x")),
    ("must be GPU tensors", lambda: moe.moe_linear_fp8(f8(2, 128), f32(1, 2), f8(64, 128), f32(1, 1))),
    ("offsets has shape", lambda: moe.moe_linear_grouped_fp8(
        f8(2, 128), f32(1, 2), t(4, dtype=torch.int32), f8(4, 64, 128), f32(4, 1, 1))),
    ("offsets is required", lambda: moe.moe_linear_grouped_fp8(
        f8(2, 128), f32(1, 2), None, f8(4, 64, 128), f32(4, 1, 1))),
    ("outside", lambda: moe.moe_linear_grouped_fp8(
        f8(2, 128), f32(1, 2), I5, f8(4, 64, 128), f32(4, 1, 1), rows=3)),
    ("without perm", lambda: moe.moe_linear_grouped_fp8(
        f8(2, 128), f32(1, 2), I5, f8(4, 64, 128), f32(4, 1, 1), rows=1)),
    ("perm must have at least", lambda: moe.moe_linear_grouped_fp8(
        f8(2, 128), f32(1, 2), I5, f8(4, 64, 128), f32(4, 1, 1), perm=t(3, dtype=torch.int32), k=2)),
    ("w_scale has shape", lambda: moe.moe_linear_grouped_fp8(
        f8(2, 128), f32(1, 2), I5, f8(4, 64, 128), f32(1, 1))),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_binding_refuses(i):
    text, call = BAD[i]
    with pytest.raises(ValueError, match=text.replace("(", r"\(")):
        call()
