"""Outputs and workspaces that lie over what the same launch reads or writes: the
kernels would race with themselves, so the calls are refused (host validation only,
nothing is launched)."""
import ctypes

import pytest

import sparse_mixture_experts_05_amd as moe

P = [0x10000000 * (i + 1) for i in range(16)]  # far apart, never dereferenced
V = ctypes.c_void_p
INVALID = -1


# ---------------------------------------------------------------- products

M, N, K, E = 32, 128, 64, 8
X, W, B, RES, Y, WS, PERM, OFF = P[:8]
SIZE = {  # bytes of a bf16 call
    "x": (X, M * K * 2), "w": (W, 2 * N * K * 2), "bias": (B, 2 * N * 2), "residual": (RES, M * N * 2),
}


def linear(y=Y, ws=WS, act=4, dt=1, K=K, res=RES):
    return moe.lib().moe_linear(V(X), V(W), V(B), act, V(res), M, N, K, dt, V(y), V(ws), 1 << 40, None)


def grouped(y=Y, ws=WS, dt=1, K=K):
    return moe.lib().moe_linear_grouped(V(X), V(PERM), 2, M, V(OFF), E, 2 * M, V(W), V(B), 4, V(RES), N, K,
                                        dt, V(y), V(ws), 1 << 40, None)


@pytest.mark.parametrize("name", SIZE)
def test_linear_output_over_an_input(name):
    at, n = SIZE[name]
    assert linear(y=at + n - 16) == INVALID  # the last bytes of the input
    assert linear(y=at - M * N * 2 + 16) == INVALID  # its first


@pytest.mark.parametrize("name,at,n", [("w", W, E * 2 * N * K * 2), ("bias", B, E * 2 * N * 2),
                                       ("perm", PERM, 2 * M * 4), ("offsets", OFF, (E + 1) * 4)])
def test_linear_grouped_output_over_an_input(name, at, n):
    assert grouped(y=at) == INVALID
    assert grouped(y=(at + n - 1) // 16 * 16) == INVALID
    assert grouped(y=at - 2 * M * N * 2 + 16) == INVALID


def test_linear_workspace_over_an_operand():
    need = moe.lib().moe_linear_workspace_bytes(M, N, 4096, 4, 0)
    assert need > 0
    for at in (X, W, B, RES, Y):
        assert linear(ws=at, dt=0, K=4096) == INVALID
        assert linear(ws=at - need + 16, dt=0, K=4096) == INVALID
    need = moe.lib().moe_linear_grouped_workspace_bytes(E, 2 * M, N, 4096, 4, 0)
    assert need > 0
    for at in (PERM, OFF):
        assert grouped(ws=at, dt=0, K=4096) == INVALID
        assert grouped(ws=at - need + 16, dt=0, K=4096) == INVALID


# ---------------------------------------------------------------- norms

ROWS, H = 4, 96
NB = ROWS * H * 2  # bytes of bf16 rows


def norm(out):
    return moe.lib().moe_norm(V(X), V(W), V(B), ROWS, H, 1e-6, 1, 1, V(out), None)


@pytest.mark.parametrize("at", [W, B])
def test_norm_output_over_a_parameter(at):
    assert norm(at + H * 2 - 32) == INVALID
    assert norm(at - NB + 16) == INVALID


GATE, NW, NBIAS, ROUT, NOUT = P[8:13]


def residual(rout=ROUT, nout=NOUT, mode=2):
    return moe.lib().moe_norm_residual(V(X), 1, V(W), V(B), V(RES), V(GATE), mode, 0.5, 2, V(NW), V(NBIAS),
                                       ROWS, H, 1e-6, 1, V(rout), V(nout), None)


@pytest.mark.parametrize("at", [W, B, NW, NBIAS, GATE])
@pytest.mark.parametrize("which", ["rout", "nout"])
def test_norm_residual_output_over_a_parameter(at, which):
    assert residual(**{which: at + H * 2 - 32}) == INVALID
    assert residual(**{which: at - NB + 16}) == INVALID


@pytest.mark.parametrize("which", ["rout", "nout"])
def test_norm_residual_output_over_the_gate(which):
    assert residual(**{which: GATE}, mode=1) == INVALID  # a value a row: other rows still read it
    assert residual(**{which: GATE + 16}, mode=3) == INVALID
    assert residual(**{which: GATE - 16}, mode=3) == INVALID


# ---------------------------------------------------------------- grouped routing

T, RH, RE, RK = 32, 4096, 128, 8
IDX, TW = P[13:15]


def route(idx=IDX, w=TW, ws=WS):
    return moe.lib().moe_route_grouped(V(X), V(W), V(B), T, RH, RE, RK, 1, 8, 4, 2, 1, 2.5, 1, V(idx), V(w),
                                       V(ws), 1 << 40, None)


@pytest.mark.parametrize("at,n", [(X, T * RH * 2), (W, RE * RH * 2), (B, RE * 4)])
@pytest.mark.parametrize("which", ["idx", "w"])
def test_route_grouped_output_over_an_input(at, n, which):
    assert route(**{which: at + n - 4}) == INVALID
    assert route(**{which: at - T * RK * 4 + 4}) == INVALID


def test_route_grouped_outputs_and_workspace():
    assert route(w=IDX) == INVALID
    assert route(w=IDX + T * RK * 4 - 4) == INVALID
    need = moe.lib().moe_route_grouped_workspace_bytes(T, RH, RE, RK, 1)
    assert need > 0
    for at in (X, W, B, IDX, TW):
        assert route(ws=at) == INVALID
        assert route(ws=at - need + 16) == INVALID
