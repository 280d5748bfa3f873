"""GPU: moe_block_forward with few=True and with 8-bit experts, against the block in
float64, against the separate calls, and captured.

few=True rounds less than the block's own steps and is held to their bounds. With 8-bit
experts the oracle has the weights and the normed x as the quantised ones multiply them
(their values are exact in float64) and the activated rows as they are before they are
quantised: an element then is off by half a step of e4m3, 2^-4 of it at most and
2^-4 / sqrt(3) in the mean over a step's ends, independently of the others, so a row of
their products is off by 2^-4 / sqrt(3) of its norm, besides the block's own roundings.
"""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe
from tests.test_gpu_block import KW, REL, block64, check, choose64, params, stream_rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
REL8 = REL[BF16] + 2.0 ** -4 / 3 ** 0.5


def dequant_rows(q, s):
    return q.double() * s.double().t().repeat_interleave(128, 1)


def dequant(q, s):
    N, K = q.shape[-2:]
    s = s.double().repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)
    return q.double() * s


def quantized(p, shared=True):
    """(the block's arguments with 8-bit experts, the parameters that those stand for)."""
    args, exact = dict(p), dict(p)
    for n in ("w_up", "w_down", "ws_up", "ws_down"):
        if n in p and (shared or n[1] == "_"):
            q, s = moe.moe_quantize_weight(p[n])
            args[n], args[n + "_scale"], exact[n] = q, s, dequant(q, s)
    return args, exact


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,E,H,F,Fs", [(1, 16, 256, 128, 0), (5, 64, 512, 192, 128), (64, 32, 320, 320, 64)])
def test_few(T, E, H, F, Fs, dtype):
    print(f"\n[gpu] block few T={T} E={E} H={H} F={F} Fs={Fs} {dtype}", flush=True)
    p = params(E, H, F, Fs, dtype)
    h = stream_rows(T, H, dtype, p, 1)
    got = moe.moe_block_forward(h, few=True, **p, **KW)
    check(h, p, got, dtype)
    assert "inv" not in got
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = moe.moe_block_forward(h, few=True, stream=side, **p, **KW)
    side.synchronize()
    assert torch.equal(other["res"], got["res"]) and torch.equal(other["next"], got["next"])


@pytest.mark.parametrize("T,E,H,F,Fs,cap,shared", [
    (1, 16, 256, 128, 0, None, True), (5, 64, 512, 384, 128, None, True), (64, 32, 384, 256, 128, None, False),
    (130, 8, 256, 256, 0, 40, True), (1500, 16, 512, 256, 256, None, True)])
def test_8bit(T, E, H, F, Fs, cap, shared):
    print(f"\n[gpu] block in 8 bits T={T} E={E} H={H} F={F} Fs={Fs} cap={cap}", flush=True)
    p = params(E, H, F, Fs, BF16, bias=cap is None)
    args, exact = quantized(p, shared)
    h = stream_rows(T, H, BF16, p, 1)
    junk = torch.full((1 << 24,), float("nan"), device="cuda")  # what unwritten rows may hold
    del junk
    got = moe.moe_block_forward(h, capacity=cap, **args, **KW)
    idx, w, _ = choose64(got["x"], p)
    assert torch.equal(got["topk_idx"].long(), idx)
    keep = None if cap is None else (got["inv"] >= 0).view(idx.shape)
    x64 = dequant_rows(*moe.moe_quantize(got["x"]))
    out, _, _, _ = block64(h, x64, {n: v for n, v in exact.items() if shared or not n.startswith("ws_")}, idx, w, keep)
    if not shared:  # the shared expert stays in bf16
        only = {n: v for n, v in exact.items() if n.startswith("ws_")}
        none = torch.full_like(idx, -1)
        out += block64(h, got["x"].double(), dict(exact, **only), none, w)[0]
    off = float((got["out"].double() - out).norm() / out.norm())
    assert off <= REL8, off
    # the steps one by one
    d = moe.moe_dispatch(got["topk_idx"], got["x"], E, capacity=cap, gather=False)
    q = moe.moe_quantize(got["x"])
    b = {n: args.get(n) for n in ("b_up", "b_down")}
    a = moe.moe_linear_grouped_fp8(*q, d["offsets"], args["w_up"], args["w_up_scale"], b["b_up"], "swiglu",
                                   perm=d["perm"], k=4)
    ys = moe.moe_linear_grouped_fp8(*moe.moe_quantize(a), d["offsets"], args["w_down"], args["w_down_scale"], b["b_down"])
    ysh = None
    if Fs and shared:
        ysh = moe.moe_linear_fp8(*q, args["ws_up"], args["ws_up_scale"], act="swiglu")
        ysh = moe.moe_linear_fp8(*moe.moe_quantize(ysh), args["ws_down"], args["ws_down_scale"])
    elif Fs:
        ysh = moe.moe_linear(moe.moe_linear(got["x"], args["ws_up"], act="swiglu"), args["ws_down"])
    assert torch.equal(moe.moe_combine(ys, d["inv"], got["topk_w"], ysh), got["out"])


@pytest.mark.parametrize("how", ["few", "8bit"])
@pytest.mark.parametrize("T", [1, 48])
def test_graphs(T, how):
    """Two graphs of one block, replayed in turn, with eager blocks between."""
    print(f"\n[gpu] block graph {how} T={T}", flush=True)
    H = 256
    p = params(16, H, 128, 128, BF16)
    args = dict(p, few=True) if how == "few" else quantized(p)[0]
    kw = {n: v for n, v in {**args, **KW}.items() if n not in ("wg", "w_up", "w_down", "k")}
    graphs = [moe.MoEBlockGraph(T, p["wg"], args["w_up"], args["w_down"], KW["k"], **kw) for _ in range(2)]
    for rep in range(4):
        hs = [stream_rows(T, H, BF16, p, 10 * rep + i) for i in range(2)]
        outs = [g.run(h) for g, h in zip(graphs, hs)]
        for h, (res, nxt) in zip(hs, outs):
            want = moe.moe_block_forward(h, **args, **KW)
            torch.cuda.synchronize()
            assert torch.equal(res, want["res"]) and torch.equal(nxt, want["next"]), rep
