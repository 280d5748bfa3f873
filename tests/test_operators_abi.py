"""Refusals of the operators around the layer (norms, grouped routing, products
with an epilogue): host validation only, nothing is launched. The C entry points
first, then the binding's checks, which see every mismatch before any pointer
reaches the library."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_05_amd as moe

P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(16)]  # far apart, never dereferenced
ODD = ctypes.c_void_p(0x10000008)
NAN, INF = float("nan"), float("inf")


def norm(x=P[0], w=P[1], b=P[2], rows=4, H=100, eps=1e-6, kind=1, dt=1, out=P[3]):
    return moe.lib().moe_norm(x, w, b, rows, H, eps, kind, dt, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(x=ODD), -1), (dict(w=ODD), -1),
    (dict(b=ODD), -1), (dict(out=ODD), -1), (dict(rows=0), -1), (dict(rows=-1), -1),
    (dict(H=0), -1), (dict(eps=-1e-6), -1), (dict(eps=NAN), -1), (dict(eps=INF), -1),
    (dict(kind=0), -1), (dict(kind=3), -1), (dict(dt=2), -1), (dict(H=16385), -2),
    (dict(rows=1000, H=4096, out=ctypes.c_void_p(P[0].value + 4096)), -1),  # out inside x
    (dict(rows=1000, H=4096, out=ctypes.c_void_p(P[0].value - 4096)), -1),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def residual(y=P[0], kind=1, w=P[1], b=None, res=P[2], gate=P[3], mode=2, scale=0.5, nkind=1,
             nw=P[4], nb=None, rows=4, H=100, eps=1e-6, dt=1, rout=P[5], nout=P[6]):
    return moe.lib().moe_norm_residual(y, kind, w, b, res, gate, mode, scale, nkind, nw, nb, rows, H,
                                       eps, dt, rout, nout, None)


@pytest.mark.parametrize("kw", [
    dict(y=None), dict(res=None), dict(rout=None), dict(nout=None), dict(gate=None), dict(mode=0),
    dict(mode=4), dict(mode=-1), dict(kind=0), dict(kind=5), dict(nkind=0), dict(nkind=-1),
    dict(nkind=0, nout=None), dict(scale=NAN), dict(scale=INF), dict(eps=-1.0), dict(rows=0),
    dict(H=-3), dict(dt=9), dict(y=ODD), dict(res=ODD), dict(gate=ODD), dict(nw=ODD), dict(nb=ODD),
    dict(rout=ODD), dict(nout=ODD), dict(rout=P[0]), dict(nout=P[2]), dict(nout=P[5]),
    dict(rout=ctypes.c_void_p(P[2].value + 16)), dict(nout=ctypes.c_void_p(P[0].value + 16)),
])
def test_norm_residual_refusals(kw):
    assert residual(**kw) == -1


def test_norm_residual_unsupported():
    assert residual(H=16385) == -2


def grouped(x=P[0], wg=P[1], bias=P[2], T=32, H=64, E=64, k=4, score=1, groups=8, tg=4, gt=2, rn=1,
            scale=2.5, dt=1, idx=P[3], w=P[4], ws=P[5], wsn=1 << 24):
    return moe.lib().moe_route_grouped(x, wg, bias, T, H, E, k, score, groups, tg, gt, rn, scale, dt,
                                       idx, w, ws, wsn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(wg=None), -1), (dict(idx=None), -1), (dict(w=None), -1),
    (dict(x=ODD), -1), (dict(wg=ODD), -1), (dict(ws=ODD), -1), (dict(dt=3), -1), (dict(T=0), -1),
    (dict(k=0), -1), (dict(score=2), -1), (dict(score=-1), -1), (dict(groups=0), -1),
    (dict(tg=0), -1), (dict(gt=0), -1), (dict(gt=3), -1), (dict(rn=2), -1), (dict(scale=NAN), -1),
    (dict(scale=INF), -1), (dict(groups=7), -2), (dict(tg=9), -2), (dict(E=256, groups=128), -2),
    (dict(E=16, tg=1, k=4), -2), (dict(E=257), -2), (dict(k=9), -2), (dict(H=96), -2), (dict(T=(1 << 27) + 1, k=1), -2),
    (dict(H=4096, ws=None), -3), (dict(H=4096, wsn=16), -3),
    (dict(dt=0, ws=None), -3), (dict(dt=0, wsn=16), -3),
])
def test_route_grouped_refusals(kw, status):
    assert grouped(**kw) == status


def test_route_grouped_workspace():
    L = moe.lib()
    assert L.moe_route_grouped_workspace_bytes(16, 4096, 128, 8, 1) >= 16 * 128 * 4
    assert L.moe_route_grouped_workspace_bytes(16, 4096, 257, 8, 1) == 0
    assert L.moe_route_grouped_workspace_bytes(16, 1024, 64, 8, 1) == 0  # one launch


def linear(x=P[0], w=P[1], b=P[2], act=2, res=P[3], M=32, N=64, K=64, dt=1, y=P[4], ws=P[5],
           wsn=1 << 40):
    return moe.lib().moe_linear(x, w, b, act, res, M, N, K, dt, y, ws, wsn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(act=5), -1),
    (dict(act=-1), -1), (dict(M=0), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(dt=4), -1),
    (dict(x=ODD), -1), (dict(w=ODD), -1), (dict(b=ODD), -1), (dict(res=ODD), -1), (dict(y=ODD), -1),
    (dict(ws=ODD), -1), (dict(N=96), -2), (dict(K=32), -2),
    (dict(M=2 ** 31 - 1, N=1 << 20), -2), (dict(M=1 << 22, N=1 << 14), -2),
    (dict(y=P[0]), -1), (dict(y=ctypes.c_void_p(P[0].value + 16)), -1),
    (dict(y=ctypes.c_void_p(P[3].value + 16)), -1),
])
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


def lgrouped(x=P[0], perm=P[6], k=2, T=16, off=P[7], E=8, rows=32, w=P[1], b=P[2], act=4,
             res=P[3], N=64, K=64, dt=1, y=P[4], ws=P[5], wsn=1 << 40):
    return moe.lib().moe_linear_grouped(x, perm, k, T, off, E, rows, w, b, act, res, N, K, dt, y, ws,
                                        wsn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(off=None), -1), (dict(x=None), -1), (dict(E=0), -1), (dict(rows=0), -1), (dict(T=0), -1),
    (dict(k=0), -1), (dict(k=9), -2), (dict(rows=33), -2), (dict(E=257), -2), (dict(N=32), -2),
    (dict(K=72), -2), (dict(y=P[0]), -1), (dict(act=7), -1),
])
def test_linear_grouped_refusals(kw, status):
    assert lgrouped(**kw) == status


# ---------------------------------------------------------------- the binding

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


BAD = [
    ("x must have 2 dimensions", lambda: moe.moe_norm(t(8))),
    ("weight has shape", lambda: moe.moe_norm(t(2, 8), t(9))),
    ("weight must be torch.bfloat16", lambda: moe.moe_norm(t(2, 8), t(8, dtype=torch.float32))),
    ("kind must be one of", lambda: moe.moe_norm(t(2, 8), kind="l2")),
    ("unsupported dtype", lambda: moe.moe_norm(t(2, 8, dtype=torch.float16))),
    ("out has shape", lambda: moe.moe_norm(t(2, 8), out=t(2, 9))),
    ("must be contiguous", lambda: moe.moe_norm(t(8, 2).t())),
    ("must be GPU tensors", lambda: moe.moe_norm(t(2, 8))),
    ("weight must be a torch tensor", lambda: moe.moe_norm(t(2, 8), 1.0)),
    ("res has shape", lambda: moe.moe_norm_residual(t(2, 8), t(3, 8))),
    ("gate must have shape", lambda: moe.moe_norm_residual(t(2, 8), t(2, 8), gate=t(2))),
    ("gate must have shape", lambda: moe.moe_norm_residual(t(2, 8), t(2, 8), gate=0.5)),
    ("needs a next_kind", lambda: moe.moe_norm_residual(t(2, 8), t(2, 8), next_out=t(2, 8))),
    ("next_kind must be one of", lambda: moe.moe_norm_residual(t(2, 8), t(2, 8), next_kind=None)),
    ("res is on meta", lambda: moe.moe_norm_residual(t(2, 8), t(2, 8).to("meta"))),
    ("wg has shape", lambda: moe.moe_route_grouped(t(2, 64), t(8, 128), None, 2)),
    ("bias must be torch.float32", lambda: moe.moe_route_grouped(t(2, 64), t(8, 64), t(8), 2)),
    ("score must be one of", lambda: moe.moe_route_grouped(t(2, 64), t(8, 64), None, 2, score="x")),
    ("topk_idx has shape", lambda: moe.moe_route_grouped(
        t(2, 64), t(8, 64), None, 2, topk_idx=t(2, 3, dtype=torch.int32))),
    ("w must have 3 dimensions", lambda: moe.moe_linear(t(2, 64), t(64, 64), act="swiglu")),
    ("w has shape", lambda: moe.moe_linear(t(2, 64), t(3, 64, 64), act="geglu")),
    ("w has shape", lambda: moe.moe_linear(t(2, 64), t(64, 128))),
    ("bias has shape", lambda: moe.moe_linear(t(2, 64), t(2, 64, 64), t(64), act="geglu")),
    ("residual has shape", lambda: moe.moe_linear(t(2, 64), t(64, 64), residual=t(1, 64))),
    ("act must be one of", lambda: moe.moe_linear(t(2, 64), t(64, 64), act="tanh")),
    ("offsets has shape", lambda: moe.moe_linear_grouped(
        t(2, 64), t(4, dtype=torch.int32), t(4, 64, 64))),
    ("outside", lambda: moe.moe_linear_grouped(
        t(2, 64), t(5, dtype=torch.int32), t(4, 64, 64), rows=3)),
    ("perm must have at least", lambda: moe.moe_linear_grouped(
        t(2, 64), t(5, dtype=torch.int32), t(4, 64, 64), perm=t(3, dtype=torch.int32), k=2)),
    ("perm must be torch.int32", lambda: moe.moe_linear_grouped(
        t(2, 64), t(5, dtype=torch.int32), t(4, 64, 64), perm=t(4, dtype=torch.int64), k=2)),
    ("y has shape", lambda: moe.moe_linear_grouped(
        t(2, 64), t(5, dtype=torch.int32), t(4, 64, 64), y=t(3, 64))),
    ("needs ws_up and ws_down", lambda: moe.moe_block_forward(
        t(2, 64), t(4, 64), t(4, 2, 64, 64), t(4, 64, 64), 2, ws_up=t(2, 64, 64))),
    ("must be GPU tensors", lambda: moe.moe_block_forward(
        t(2, 64), t(4, 64), t(4, 2, 64, 64), t(4, 64, 64), 2)),
    ("makes its own x", lambda: moe.MoEBlockGraph(
        2, t(4, 64), t(4, 2, 64, 64), t(4, 64, 64), 2, x=t(2, 64))),
    ("wg must be a GPU tensor", lambda: moe.MoEBlockGraph(
        2, t(4, 64), t(4, 2, 64, 64), t(4, 64, 64), 2)),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_binding_refuses(i):
    text, call = BAD[i]
    with pytest.raises(ValueError, match=text.replace("(", r"\(")):
        call()
