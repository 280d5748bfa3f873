"""GPU: moe_layer_few against the layer in float64, and against the separate calls.

Ids have to be the oracle's (rows are drawn again until the decisions are clear) and
weights within 2e-5 of its (tests/test_gpu_route_grouped.py). The output is held to the
experts in float64 with the call's own ids and weights (u = 2^-24, half = 2^-8 for bf16,
2^-24 for fp32). A product of K terms is off by at most d = K u sum|x w| + 2 u |a| in any
order; h = act(a) by 1.13 d + e |h| (e = 1e-4 for the bf16 gelu, else 8 u), with a gate as
tests/test_gpu_linear.py has it, and its rounding by half |h| more; out by the sum over
the experts of |w| times (those errors times |down| + F u sum|h down|), k + 2 roundings of
the sum, and its own rounding. Norms: the two roundings to bf16 are off by 2^-8 / sqrt(3) in
the mean each, so the error's norm is held to 2 * 2^-8 / sqrt(3) of out's; fp32 to 1e-5.
"""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_05_amd as moe
from tests.test_gpu_linear import HALF, U, act64, randn
from tests.test_gpu_route_grouped import RTOL_W, oracle

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
GATED = ("geglu", "swiglu")
SCALE = 2.5
REL = {BF16: 2 * 2.0 ** -8 / 3 ** 0.5, FP32: 1e-5}


def make(T, H, E, k, F, Fs, act, dtype, bias, mode, seed, **route):
    """(x, wg, bias, other tensors): rows whose decisions are clear."""
    two = (2,) if act in GATED else ()
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).to(dtype)
    wg = (torch.randn((E, H), generator=g) / H ** 0.5).to(dtype)
    b = np.float32(0.1) * np.random.default_rng(seed).standard_normal(E).astype(np.float32) if bias else None
    inside = b if mode == "score" and b is not None else np.zeros(E, np.float32)
    moves = b if mode == "choice" else None
    for _ in range(200):
        s = (x.double() @ wg.double().t()).numpy() + inside
        bad = [t for t in range(T) if oracle(s[t:t + 1], moves, k, **route)[2] < 4e-5]
        if not bad:
            break
        x[bad] = torch.randn((len(bad), H), generator=g).to(dtype)
    want = oracle(s, moves, k, **route)
    p = dict(w_up=randn((E, *two, F, H), dtype, seed + 1, H ** -0.5),
             w_down=randn((E, H, F), dtype, seed + 2, F ** -0.5),
             b_up=randn((E, *two, F), dtype, seed + 3, 0.3) if bias else None,
             b_down=randn((E, H), dtype, seed + 4, 0.3) if bias else None,
             ws_up=randn((*two, Fs, H), dtype, seed + 5, H ** -0.5) if Fs else None,
             ws_down=randn((H, Fs), dtype, seed + 6, Fs ** -0.5) if Fs else None)
    return x.cuda(), wg.cuda(), None if b is None else torch.tensor(b).cuda(), p, want


def expert64(x, up, down, b_up, b_down, act, dtype):
    """(y, error bound) of one expert's rows."""
    H, two = x.shape[1], act in GATED
    F = up.shape[-2]
    wf = up.double().reshape(-1, H)
    a = x.double() @ wf.t()
    d = H * U * (x.double().abs() @ wf.abs().t())
    if b_up is not None:
        a = a + b_up.double().reshape(1, -1)
    d = d + 2 * U * a.abs()
    e = 1e-4 if dtype == BF16 and act in ("gelu", "geglu") else 8 * U
    h = act64(a[:, :F], act)
    err = 1.13 * d[:, :F] + e * h.abs()
    if two:
        err = err * (a[:, F:].abs() + d[:, F:]) + h.abs() * d[:, F:]
        h = h * a[:, F:]
    err = err + HALF[dtype] * (h.abs() + err)
    w = down.double()
    y, dy = h @ w.t(), err @ w.abs().t() + F * U * ((h.abs() + err) @ w.abs().t())
    if b_down is not None:
        y = y + b_down.double()
    return y, dy + 2 * U * y.abs()


def layer64(x, p, idx, w, act, dtype):
    k = idx.shape[1]
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    err, size = torch.zeros_like(out), torch.zeros_like(out)
    get = lambda n, e: None if p[n] is None else p[n][e]  # noqa: E731
    for e in sorted(set(idx.flatten().tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        y, d = expert64(x[t], p["w_up"][e], p["w_down"][e], get("b_up", e), get("b_down", e), act, dtype)
        wt = w[t, j].double()[:, None]
        out[t] += wt * y
        err[t] += wt.abs() * d
        size[t] += (wt * y).abs()
    if p["ws_up"] is not None:
        y, d = expert64(x, p["ws_up"], p["ws_down"], None, None, act, dtype)
        out, err, size = out + y, err + d, size + y.abs()
    return out, err + (k + 2) * U * size


def near(got, want, err, dtype, name):
    got = got.double()
    off = (got - want).abs() - (err + HALF[dtype] * want.abs() * (1 + 2.0 ** -6) + 1e-38)
    assert not torch.isnan(got).any() and off.max() <= 0, f"{name}: {off.max():.3e} over"
    rel = (got - want).norm() / want.norm()
    assert rel <= REL[dtype], f"{name}: rel {rel:.3e}"


CASES = [  # T, H, E, k, F, Fs, act, score, mode, (groups, topk_groups, group_top), bias, renorm, dtype
    (1, 64, 1, 1, 64, 0, "none", "softmax", "choice", (1, 1, 1), False, True, BF16),
    (1, 4096, 128, 8, 1536, 1536, "gelu", "softmax", "score", (1, 1, 1), False, True, BF16),
    (5, 256, 8, 2, 512, 0, "gelu", "softmax", "score", (1, 1, 1), True, True, FP32),
    (2, 192, 40, 3, 64, 128, "silu", "sigmoid", "choice", (8, 4, 2), True, True, BF16),
    (16, 1024, 64, 8, 320, 64, "swiglu", "sigmoid", "choice", (8, 4, 2), True, True, BF16),
    (13, 2112, 255, 7, 192, 0, "geglu", "softmax", "choice", (5, 2, 1), True, False, BF16),
    (17, 512, 65, 8, 256, 576, "swiglu", "softmax", "score", (1, 1, 1), True, True, BF16),
    (32, 320, 16, 4, 448, 64, "gelu", "sigmoid", "score", (4, 2, 2), True, False, BF16),
    (33, 1024, 32, 4, 704, 0, "swiglu", "sigmoid", "choice", (4, 2, 2), True, True, BF16),
    (64, 2048, 256, 8, 128, 128, "geglu", "softmax", "choice", (8, 4, 2), False, True, BF16),
    (64, 64, 2, 2, 64, 64, "silu", "sigmoid", "choice", (1, 1, 1), True, True, BF16),
    (48, 8256, 3, 1, 64, 0, "none", "softmax", "choice", (1, 1, 1), True, False, BF16),
    (3, 320, 96, 8, 192, 320, "swiglu", "sigmoid", "choice", (6, 3, 1), True, True, FP32),
    (20, 256, 30, 4, 128, 0, "geglu", "softmax", "score", (1, 1, 1), True, True, FP32),
    (64, 448, 64, 8, 64, 192, "gelu", "softmax", "choice", (1, 1, 1), False, True, FP32),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_H%d_E%d_k%d_F%d_Fs%d_%s_%s_%s" % c[:9])
def test_against_float64(case):
    T, H, E, k, F, Fs, act, score, mode, (groups, tg, gt), bias, renorm, dtype = case
    print(f"\n[gpu] few {case}", flush=True)
    route = dict(score=score, groups=groups, topk_groups=tg, group_top=gt, renorm=renorm, scale=SCALE)
    x, wg, b, p, want = make(T, H, E, k, F, Fs, act, dtype, bias, mode, T + H, **route)
    whole = torch.full((T + 16, H), 3.0, dtype=dtype, device="cuda")
    idx, w = torch.full((T + 2, k), -9, dtype=torch.int32, device="cuda"), torch.full((T + 2, k), -9.0, device="cuda")
    ws = torch.full((moe.moe_layer_few_workspace_bytes(T, H, E, k, F, Fs, int(dtype == BF16)) + 4096,), 255,
                    dtype=torch.uint8, device="cuda")
    got, gi, gw = moe.moe_layer_few(x, wg, b, k=k, act=act, bias_mode=mode, out=whole[8:-8], topk_idx=idx[1:-1],
                                    topk_w=w[1:-1], ws=ws[:-4096], **route, **p)
    assert (gi.cpu().numpy() == want[0]).all()
    np.testing.assert_allclose(gw.cpu().numpy(), want[1], rtol=RTOL_W, atol=1e-30)
    near(got, *layer64(x, p, gi, gw, act, dtype), dtype, act)
    assert (whole[:8] == 3).all() and (whole[-8:] == 3).all() and (ws[-4096:] == 255).all()
    assert (idx[0] == -9).all() and (idx[-1] == -9).all() and (w[0] == -9).all() and (w[-1] == -9).all()
    for _ in range(3):  # equal calls, equal bits, whatever the workspace holds
        again = moe.moe_layer_few(x, wg, b, k=k, act=act, bias_mode=mode, **route, **p)
        assert all(torch.equal(u, v) for u, v in zip(again, (got, gi, gw)))


def test_is_the_layer_of_the_separate_calls():
    """moe_layer_forward's layer: the same ids, weights within rounding, and outputs within
    what the separate calls round more (each expert's row, to bf16)."""
    print("\n[gpu] few against moe_layer_forward", flush=True)
    route = dict(score="softmax", groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0)
    for T, Fs in ((1, 0), (7, 256), (40, 128)):
        x, wg, b, p, _ = make(T, 512, 32, 4, 256, Fs, "gelu", BF16, True, "score", T, **route)
        p["b_up"] = p["b_down"] = None
        want = moe.moe_layer_forward(x, wg, b, p["w_up"], p["w_down"], 4, ws1=p["ws_up"], ws2=p["ws_down"])
        out, idx, w = moe.moe_layer_few(x, wg, b, k=4, act="gelu", bias_mode="score", **p)
        assert torch.equal(idx, want["topk_idx"])
        assert torch.allclose(w, want["topk_w"], rtol=RTOL_W)
        ref, err = layer64(x, p, idx, w, "gelu", BF16)
        near(out, ref, err, BF16, "few")
        # both are within the bound of one rounding of h and out; the layer rounds ys too
        rel = (out.double() - want["out"].double()).norm() / ref.norm()
        assert rel <= 5 * 2.0 ** -8 / 3 ** 0.5


def test_ties_and_off_experts():
    """Equal scores go to the lower expert; experts that are off (-inf bias) weigh nothing
    and are chosen only when fewer than k are left."""
    print("\n[gpu] few ties", flush=True)
    T, H, E, F = 9, 64, 12, 64
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    x[torch.arange(T), torch.arange(T)] = 1
    wg = torch.zeros((E, H), dtype=BF16, device="cuda")
    wg[3:7] = 2
    up, down = randn((E, F, H), BF16, 1), randn((E, H, F), BF16, 2, F ** -0.5)
    _, idx, w = moe.moe_layer_few(x, wg, None, up, down, 6)
    assert (idx == torch.tensor([3, 4, 5, 6, 0, 1], device="cuda", dtype=torch.int32)).all()
    b = torch.full((E,), float("-inf"), device="cuda")
    b[5] = 0
    out, idx, w = moe.moe_layer_few(x, wg, b, up, down, 3)
    assert (idx == torch.tensor([5, 0, 1], device="cuda", dtype=torch.int32)).all()
    assert (w == torch.tensor([1.0, 0.0, 0.0], device="cuda")).all()
    y, d = expert64(x, up[5], down[5], None, None, "gelu", BF16)
    near(out, y, d, BF16, "one expert on")


def test_bad_tokens_stay_alone():
    """A token of NaNs or infinities reaches only its own row, and so does an expert's
    weight that is not finite."""
    print("\n[gpu] few nan", flush=True)
    route = dict(score="sigmoid", groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0)
    for T in (6, 24, 50):
        x, wg, b, p, want = make(T, 512, 32, 4, 256, 64, "swiglu", BF16, True, "choice", T, **route)
        p["ws_up"] = p["ws_down"] = None
        bad = int(want[0][3, 0])  # an expert of token 3
        p["w_down"][bad, 17, 5] = float("inf")
        x[2] = float("nan")
        x[4, 7] = float("-inf")
        out, idx, w = moe.moe_layer_few(x, wg, b, k=4, act="swiglu", **route, **p)
        assert torch.isnan(out[2]).all() and not torch.isfinite(out[4]).all()
        keep = [t for t in range(T) if t not in (2, 4)]
        assert (idx[keep].cpu().numpy() == want[0][keep]).all()
        p["w_down"][bad, 17, 5] = 0.0
        ref, err = layer64(x[keep], p, idx[keep], w[keep], "swiglu", BF16)
        hit = (idx[keep] == bad).any(1)
        cols = [c for c in range(512) if c != 17]
        near(out[keep][:, cols], ref[:, cols], err[:, cols], BF16, "other columns")
        assert not torch.isfinite(out[keep][hit][:, 17]).any()
        # the column of tokens without the expert: its weight times 0 is not added
        free = out[keep][~hit][:, 17].double()
        ok = (free - ref[~hit][:, 17]).abs() <= err[~hit][:, 17] + HALF[BF16] * 1.02 * ref[~hit][:, 17].abs()
        assert ok.all()


def test_graphs_streams_and_two_calls_at_once():
    """Captured graphs with workspaces of their own, replayed in turn with eager calls
    between; calls at the same time on two streams: each the same bits as alone."""
    print("\n[gpu] few graphs and streams", flush=True)
    route = dict(score="sigmoid", groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0)
    cases = []
    for T, F, act in ((1, 512, "gelu"), (16, 256, "swiglu"), (40, 128, "geglu")):
        x, wg, b, p, _ = make(T, 1024, 64, 8, F, 128, act, BF16, True, "choice", T, **route)
        call = lambda x=x, wg=wg, b=b, p=p, act=act, **kw: moe.moe_layer_few(  # noqa: E731
            x, wg, b, k=8, act=act, **route, **p, **kw)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        cases.append((x, call, g, out))
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for i, (x, call, g, out) in enumerate(cases):
            x.copy_(randn(tuple(x.shape), BF16, 90 + 3 * rep + i))
            g.replay()
        for x, call, g, out in cases:
            assert all(torch.equal(u, v) for u, v in zip(call(), out)), rep
        torch.cuda.synchronize()
        both = [[call(stream=s) for s in side for _ in range(5)] for x, call, g, out in cases]
        torch.cuda.synchronize()
        for (x, call, g, out), got in zip(cases, both):
            assert all(torch.equal(u, v) for one in got for u, v in zip(one, out)), rep
