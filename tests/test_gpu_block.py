"""GPU: moe_block_forward, the operators run together as a decoder block uses
them, against the whole block in float64, and its captured form.

The routed ids have to be the oracle's (rows are drawn again until the decisions
are clear, counting the bf16 rounding of the normed x, which the route reads and
the oracle is given). Values: norms, products, combine and the residual sum each
round to bf16 once (2^-8 at most, about 2^-8 / sqrt(3) in the mean), six such
steps in a row: the output's error norm is held to 6 * 2^-8 / sqrt(3) = 1.36e-2
of the block's own contribution, and fp32 to 1e-5.
"""
import pytest
import torch

import sparse_mixture_experts_05_amd as moe

pytestmark = pytest.mark.gpu
REL = {torch.bfloat16: 6 * 2.0 ** -8 / 3 ** 0.5, torch.float32: 1e-5}


def params(E, H, F, Fs, dtype, seed=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(dtype).cuda()  # noqa: E731
    p = dict(wg=r(E, H, std=H ** -0.5), w_up=r(E, 2, F, H, std=H ** -0.5),
             w_down=r(E, H, F, std=F ** -0.5), norm_weight=1 + r(H, std=0.1),
             route_bias=(torch.randn(E, generator=g) * 0.05).cuda(), out_weight=1 + r(H, std=0.1),
             next_weight=1 + r(H, std=0.1), gate=r(H))
    if bias:
        p.update(b_up=r(E, 2, F, std=0.1), b_down=r(E, H, std=0.1))
    if Fs:
        p.update(ws_up=r(2, Fs, H, std=H ** -0.5), ws_down=r(H, Fs, std=Fs ** -0.5))
    return p


KW = dict(k=4, groups=4, topk_groups=2, scale=2.5, out_norm="rms", next_norm="rms", res_scale=0.5)


def rms(v, w):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w.double()


def glu(x, up, down, bu=None, bd=None):
    a = torch.nn.functional.linear(x, up.double().reshape(-1, x.shape[1]))
    a = a + (0 if bu is None else bu.double().reshape(1, -1))
    F = up.shape[1]
    y = a[:, :F] * torch.sigmoid(a[:, :F]) * a[:, F:] @ down.double().t()
    return y if bd is None else y + bd.double()


def block64(h, x, p, idx, w, keep=None):
    """Everything behind the choice, in float64 (x: the normed rows)."""
    out = torch.zeros_like(x)
    for e in range(p["wg"].shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if keep is not None:
            t, j = t[keep[t, j]], j[keep[t, j]]
        if t.numel():
            y = glu(x[t], p["w_up"][e], p["w_down"][e],
                    *(p[n][e] if n in p else None for n in ("b_up", "b_down")))
            out.index_add_(0, t, w[t, j].double()[:, None] * y)
    if "ws_up" in p:
        out += glu(x, p["ws_up"], p["ws_down"])
    add = 0.5 * p["gate"].double() * rms(out, p["out_weight"])
    res = h.double() + add
    return out, add, res, rms(res, p["next_weight"])


def choose64(x, p):
    """(ids, weights, clear): sigmoid scores, choice bias, 2 of 4 groups by their two best."""
    s = x.double() @ p["wg"].double().t()
    sig = torch.sigmoid(s)
    v = sig + p["route_bias"].double()
    T, E = v.shape
    g = v.view(T, 4, E // 4).sort(dim=2, descending=True).values[:, :, :2].sum(2).sort(dim=1, descending=True)
    on = torch.zeros((T, 4), dtype=torch.bool, device=v.device).scatter_(1, g.indices[:, :2], True)
    o = v.masked_fill(~on.repeat_interleave(E // 4, 1), -1e9).sort(dim=1, descending=True)
    gap = torch.minimum(g.values[:, 1] - g.values[:, 2], (o.values[:, :4] - o.values[:, 1:5]).min(1).values)
    w = sig.gather(1, o.indices[:, :4])
    return o.indices[:, :4], w / w.sum(1, keepdim=True) * 2.5, gap > 4e-5


def stream_rows(T, H, dtype, p, seed):
    """Residual-stream rows whose routing decisions are clear on the x that the norm gives."""
    g = torch.Generator().manual_seed(seed)
    h = (2 * torch.randn((T, H), generator=g)).to(dtype).cuda()
    for _ in range(100):
        bad = (~choose64(moe.moe_norm(h, p["norm_weight"]), p)[2]).nonzero().flatten()
        if bad.numel() == 0:
            return h
        h[bad] = (2 * torch.randn((bad.numel(), H), generator=g)).to(dtype).cuda()
    raise RuntimeError("no clear rows")


def check(h, p, got, dtype, capacity=None):
    x = moe.moe_norm(h, p["norm_weight"])
    assert torch.equal(got["x"], x)
    idx, w, _ = choose64(x, p)
    assert torch.equal(got["topk_idx"].long(), idx)
    torch.testing.assert_close(got["topk_w"].double(), w, rtol=2e-5, atol=0)
    keep = None if capacity is None else (got["inv"] >= 0).view(idx.shape)
    if keep is not None:
        counts = torch.bincount(idx.flatten(), minlength=p["wg"].shape[0])
        assert int(keep.sum()) == int(counts.clamp(max=capacity).sum())
    out, add, res, nxt = block64(h, x.double(), p, idx, w, keep)
    rel = lambda a, b, n: float((a.double() - b).norm() / n.norm())  # noqa: E731
    live = (out.abs().sum(1) > 0)
    assert rel(got["out"], out, out) <= REL[dtype]
    # the residual row's own rounding, and the block's error on its part
    off = (got["res"].double() - res)[live]
    assert float(off.norm()) <= REL[dtype] * float(add[live].norm()) + 2.0 ** -8 * float(res.norm())
    assert rel(got["next"][live], nxt[live], nxt[live]) <= REL[dtype]


CASES = [  # (T, E, H, F, Fs, capacity)
    (1, 16, 256, 128, 0, None), (5, 64, 512, 192, 128, None), (64, 32, 320, 320, 64, None),
    (130, 8, 256, 256, 0, 40), (1500, 16, 512, 256, 256, None),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,E,H,F,Fs,cap", CASES)
def test_block(T, E, H, F, Fs, cap, dtype):
    print(f"\n[gpu] block T={T} E={E} H={H} F={F} Fs={Fs} cap={cap} {dtype}", flush=True)
    p = params(E, H, F, Fs, dtype, bias=cap is None)
    h = stream_rows(T, H, dtype, p, 1)
    got = moe.moe_block_forward(h, capacity=cap, **p, **KW)
    check(h, p, got, dtype, cap)
    # the next block takes the norm that this one made
    x = moe.moe_norm(got["res"], p["next_weight"])
    rel = (got["next"].double() - x.double()).norm() / x.double().norm()
    assert rel <= 3 * 2.0 ** -8
    again = moe.moe_block_forward(h, x=got["x"], capacity=cap, **p, **KW)
    assert torch.equal(again["res"], got["res"]) and torch.equal(again["next"], got["next"])


@pytest.mark.parametrize("T", [1, 48, 700])
def test_block_graphs(T):
    """Two graphs of one block, replayed in turn, with eager blocks between."""
    print(f"\n[gpu] block graph T={T}", flush=True)
    H, dtype = 256, torch.bfloat16
    p = params(16, H, 128, 64, dtype)
    kw = {n: v for n, v in {**p, **KW}.items() if n not in ("wg", "w_up", "w_down", "k")}
    graphs = [moe.MoEBlockGraph(T, p["wg"], p["w_up"], p["w_down"], KW["k"], **kw)]
    copies = {n: v.clone() for n, v in p.items()}
    kw2 = {n: copies.get(n, v) for n, v in kw.items()}
    graphs.append(moe.MoEBlockGraph(T, copies["wg"], copies["w_up"], copies["w_down"], KW["k"], **kw2))
    del copies, kw2  # a graph keeps the weights that it reads
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    with pytest.raises(ValueError, match="h has shape"):
        graphs[0].run(torch.zeros((1, 1), dtype=dtype, device="cuda"))
    for rep in range(4):
        hs = [stream_rows(T, H, dtype, p, 10 * rep + i) for i in range(2)]
        outs = [g.run(h) for g, h in zip(graphs, hs)]
        for h, (res, nxt), g in zip(hs, outs, graphs):
            want = moe.moe_block_forward(h, **p, **KW)
            torch.cuda.synchronize()
            assert torch.equal(res, want["res"]) and torch.equal(nxt, want["next"]), rep
            check(h, p, g.state, dtype)
    del junk
