"""GPU: a block of linear attention with its convs, norms, dropout, residual sum
and the next norm together, as training and serving run them, against the same
in 64 bits with autograd; captured and replayed, on streams, in two packs."""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck
from tests import delta_checks as dc
from tests.test_delta_block_gpu import conv, leaves, tree

pytestmark = pytest.mark.gpu

F32, BF, F64 = torch.float32, torch.bfloat16, torch.float64


def ssp():
    import selective_state_space_varlen_amd as m
    return m


def make(lens, Hk, Hv, Dk, Dv, W, carry, dtype=F32, seed=70):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T, n, C = sum(lens), len(lens), Hv * Dv
    widths = (Hk * Dk, Hk * Dk, Hv * Dv)
    states = lambda: {"decay": 0.3 * rnd(n, Hv, Dk, Dv), "conv": tuple(rnd(n, W - 1, c).to(dtype) for c in widths)}  # noqa: E731
    return {"x": tuple(rnd(T, c).to(dtype) for c in widths), "w": tuple(0.5 * rnd(c, W) for c in widths),
            "b": tuple(0.1 * rnd(c) for c in widths), "g": -torch.exp(rnd(T, Hv) - 3),
            "nw": (1 + 0.2 * rnd(Dk), 1 + 0.2 * rnd(Dk)), "ow": (1 + 0.2 * rnd(Hv, Dv), 0.2 * rnd(Hv, Dv)),
            "res": rnd(T, C).to(dtype), "lw": 1 + 0.2 * rnd(C), "lb": 0.2 * rnd(C), "dy": rnd(T, C).to(dtype),
            "dh": rnd(T, C).to(dtype), "states": states() if carry else None, "dstates": states() if carry else None}


RNG = [(5, 1), (5, 2)]  # of the block's result, and of what is added to the residual
P, OUT_EPS = 0.25, 0.01


def seeds(i):
    return torch.tensor(RNG[i], dtype=torch.int64, device="cuda")


def step(m, x, cu, Hk, Hv, rngs, inv_freq=None):
    """Block, residual sum with dropout, norm; and back. Everything a training step wants."""
    kw = dict(w=x["w"], b=x["b"], norm=m.SSMP_NORM_RMS, norm_weights=x["nw"], inv_freq=inv_freq, out_norm=x["ow"],
              out_eps=OUT_EPS, p=P, rng=rngs[0], initial_states=x["states"])
    F = m.decay_forward(x["x"], x["g"], cu, Hk, Hv, **kw)
    y, h = m.layer_norm_pack_fwd(F["out"].view(x["res"].shape), x["lw"], x["lb"], residual=x["res"], p=P, rng=rngs[1])
    L = m.layer_norm_pack_bwd(x["dy"], h, x["lw"], dh=x["dh"], p=P, rng=rngs[1], bias=True, residual=True)
    G = m.decay_backward(x["x"], x["g"], F, L["dx"].view(F["out"].shape), dfinal_states=x["dstates"])
    return F, y, h, L, G


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("carry", [False, True])
def test_block(carry, rotate):
    lens, Hk, Hv, Dk, Dv, W = [70, 1, 0, 153], 2, 4, 32, 24, 4
    d = make(lens, Hk, Hv, Dk, Dv, W, carry)
    inv = 0.5 ** torch.arange(8, dtype=F32) if rotate else None
    m, cu, T = ssp(), dc.cu_of(lens).cuda(), sum(lens)
    x = tree(d, lambda t: t.cuda())
    F, y, h, L, G = step(m, x, cu, Hk, Hv, [seeds(0), seeds(1)], None if inv is None else inv.cuda())
    torch.cuda.synchronize()

    r = tree(d, lambda t: t.to(F64).requires_grad_())
    st = r["states"] or {}
    u, last = zip(*(conv(r["x"][i], r["w"][i], r["b"][i], lens, st["conv"][i] if carry else None) for i in range(3)))
    pos = torch.cat([torch.arange(n) for n in lens])
    q, k = (dc.turn(dc.norm(u[i].view(T, Hk, Dk), None, None, None, False, 1e-6, False) * r["nw"][i], pos, inv, False)
            for i in range(2))
    o, hT = ck.attention(q, k, u[2].view(T, Hv, Dv), r["g"], lens, Dk ** -0.5, st.get("decay"))
    n = ck.layer_norm(o, *r["ow"], OUT_EPS)
    factor = [(lambda kb: kb[0].double().view(T, -1) * kb[1])(ck.keep(T * Hv * Dv, P, *s)) for s in RNG]
    out = n * factor[0].view(n.shape)
    hr = r["res"] + out.view(T, -1) * factor[1]
    yr = ck.layer_norm(hr, r["lw"], r["lb"], 1e-5)
    loss = (yr * r["dy"]).sum() + (hr * r["dh"]).sum()
    if carry:
        loss = loss + (hT * r["dstates"]["decay"]).sum() + sum((a * b).sum() for a, b in zip(last, r["dstates"]["conv"]))
    want = {"dx": r["x"], "dw": r["w"], "db": r["b"], "dg": r["g"], "dwq": r["nw"][0], "dwk": r["nw"][1],
            "dout_norm": r["ow"], "dresidual": r["res"], "dlw": r["lw"], "dlb": r["lb"]}
    if carry:
        want["dinitial_states"] = r["states"]
    grads = iter(torch.autograd.grad(loss, leaves(want)))
    want = tree(want, lambda t: next(grads))
    got = dict(G, dresidual=L["dresidual"], dlw=L["dw"], dlb=L["db"])
    # the chain's roundings: the attention's, a conv of W terms, a norm of Dk and one of Dv and of all
    # columns. Of what the attention errs by, relative to its largest value, the head norm makes r times that
    # value, which is largest where a row is small; 8 covers the other norms (rows of size 1).
    dev = o.detach() - o.detach().mean(-1, keepdim=True)
    root = float((1 / (dev.square().mean(-1) + OUT_EPS).sqrt()).max())
    tol = 8 * ck.tol32(max(lens), Dk + W, Dv) * max(1.0, root * float(o.detach().abs().max()))
    dc.check(F["out"], out, tol, "out")
    dc.check(h, hr, tol, "h")
    dc.check(y, yr, tol, "y")
    for name in want:
        for a, b in zip(leaves(got[name]), leaves(want[name])):
            # sums over tokens: T errors, independent of one another, of terms of which the sum may be small
            dc.check(a, b, tol * (T ** 0.5 if name in ("dw", "db", "dwq", "dwk", "dout_norm", "dlw", "dlb") else 1), name)
    if carry:
        dc.check(F["final_states"]["decay"], hT, tol, "state")
        for a, b in zip(F["final_states"]["conv"], last):
            dc.check(a, b, 0.0, "conv context")


def test_parts_left_out():
    """The attention alone is the entry point's; norms and dropout are theirs, one after the other."""
    lens, Hk, Hv, Dk, Dv = [90, 40], 1, 2, 64, 32
    d = tree(make(lens, Hk, Hv, Dk, Dv, 4, False, BF), lambda t: t.cuda())
    m, cu, T = ssp(), dc.cu_of(lens).cuda(), sum(lens)
    q, k, v = (t.view(T, n, -1) for t, n in zip(d["x"], (Hk, Hk, Hv)))
    F = m.decay_forward(d["x"], d["g"], cu, Hk, Hv)
    o, _ = m.decay_attn_pack_fwd(q, k, v, d["g"], cu)
    assert torch.equal(F["out"], o) and "final_states" not in F
    dout = d["dy"].view(o.shape)
    G, E = m.decay_backward(d["x"], d["g"], F, dout), m.decay_attn_pack_bwd(q, k, v, d["g"], cu, dout)
    for a, n in zip(G["dx"], ("dq", "dk", "dv")):
        assert torch.equal(a.view(E[n].shape), E[n])
    assert torch.equal(G["dg"], E["dg"]) and G["dw"] is None and G["db"] is None and G["dwq"] is None
    assert m.decay_backward(d["x"], d["g"], F, dout, want_dg=False)["dg"] is None
    F = m.decay_forward(d["x"], d["g"], cu, Hk, Hv, out_norm=(None, None), p=0.5, rng=seeds(0))
    n, _ = m.layer_norm_pack_fwd(o)
    assert torch.equal(F["out"], m.dropout_pack_fwd(n, 0.5, seeds(0))) and torch.equal(F["attn"], o)
    F = m.decay_forward(d["x"], d["g"], cu, Hk, Hv, p=0.5, rng=seeds(0))
    assert torch.equal(F["out"], m.dropout_pack_fwd(o, 0.5, seeds(0))) and torch.equal(F["attn"], o)


def flat(res):
    F, y, h, L, G = res
    return leaves({"o": F["out"], "y": y, "h": h, "L": {k: L[k] for k in sorted(L)}, "G": {k: G[k] for k in sorted(G)}})


def test_captured_and_replayed():
    """Other values, another division into sequences and other random numbers at each replay."""
    Hk, Hv, Dk, Dv, W = 2, 2, 64, 64, 4
    m = ssp()
    d = tree(make([700, 300], Hk, Hv, Dk, Dv, W, False, BF), lambda t: t.cuda())
    cu, rngs = dc.cu_of([700, 300]).cuda(), [seeds(0), seeds(1)]

    def once():
        return flat(step(m, d, cu, Hk, Hv, rngs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = once()
        for r in rngs:
            r[1:] += 2  # the next replay's stream
    for i, lens in enumerate(([700, 300], [1, 999], [1000, 0], [512, 488])):
        new = tree(make(lens, Hk, Hv, Dk, Dv, W, False, BF, seed=80 + i), lambda t: t.cuda())
        for a, b in zip(leaves(d), leaves(new)):
            a.copy_(b)
        cu.copy_(dc.cu_of(lens))
        before = [r.clone() for r in rngs]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        assert all(int(r[1]) == int(b[1]) + 2 for r, b in zip(rngs, before))
        for r, b in zip(rngs, before):
            r.copy_(b)
        want = once()
        for r in rngs:
            r[1:] += 2
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), lens


def test_two_graphs_on_one_scratch():
    Hk, Hv, Dk, Dv, T = 1, 2, 64, 128, 900
    m = ssp()
    need = (m.decay_attn_pack_fwd_scratch_bytes(T, 3, Hk, Hv, Dk, Dv), m.decay_attn_pack_bwd_scratch_bytes(T, 3, Hk, Hv, Dk, Dv))
    scratch = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    graphs = []
    for seed, lens in ((1, [900]), (2, [200, 300, 400])):
        x = {k: None if v is None else v.cuda() for k, v in ck.inputs(seed, lens, Hk, Hv, Dk, Dv, BF, True).items()}
        cu = dc.cu_of(lens).cuda()

        def call(x=x, cu=cu, s=None):
            o, hT = m.decay_attn_pack_fwd(x["q"], x["k"], x["v"], x["g"], cu, initial_state=x["h0"], final_state=True, scratch=s)
            G = m.decay_attn_pack_bwd(x["q"], x["k"], x["v"], x["g"], cu, x["dout"], initial_state=x["h0"],
                                      dfinal_state=x["dhT"], dinitial_state=True, scratch=s)
            return [o, hT] + [G[n] for n in sorted(G)]
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = call(s=scratch)
        graphs.append((g, res, want, x, cu))  # a graph reads its inputs where they were
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for i in order:
            scratch.fill_(255)
            g, res, want = graphs[i][:3]
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_streams():
    """Two steps at once, each with buffers of its own, give what each gives alone."""
    Hk, Hv, Dk, Dv, W = 2, 4, 64, 64, 4
    m = ssp()
    ds = [tree(make(lens, Hk, Hv, Dk, Dv, W, True, BF, seed=s), lambda t: t.cuda()) for lens, s in (([700, 40], 1), ([64, 900], 2))]
    cus = [dc.cu_of(lens).cuda() for lens in ([700, 40], [64, 900])]
    rngs = [seeds(0), seeds(1)]
    want = [[t.clone() for t in flat(step(m, d, cu, Hk, Hv, rngs))] for d, cu in zip(ds, cus)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, d, cu in zip(streams, ds, cus):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(flat(step(m, d, cu, Hk, Hv, rngs)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_without_tokens():
    Hk, Hv, Dk, Dv, W = 1, 2, 32, 24, 4
    d = tree(make([0, 0], Hk, Hv, Dk, Dv, W, True), lambda t: t.cuda())
    m, cu = ssp(), dc.cu_of([0, 0]).cuda()
    F, y, h, L, G = step(m, d, cu, Hk, Hv, [seeds(0), seeds(1)])
    torch.cuda.synchronize()
    assert F["out"].shape == (0, Hv, Dv) and y.shape == h.shape == (0, Hv * Dv)
    for a, b in zip(leaves(F["final_states"]), leaves(d["states"])):
        assert torch.equal(a, b)
    for a, b in zip(leaves(G["dinitial_states"]), leaves(d["dstates"])):
        assert torch.equal(a, b)
    for t in leaves(G["dw"]) + leaves(G["db"]) + leaves(G["dout_norm"]) + [G["dwq"], G["dwk"], L["dw"], L["db"]]:
        assert not bool(t.any())
    g = torch.zeros(Hv, device="cuda")
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    D = m.decay_attn_pack_bwd(e(0, Hk, Dk), e(0, Hk, Dk), e(0, Hv, Dv), g, cu, e(0, Hv, Dv),
                              out={"dq": e(0, Hk, Dk), "dk": e(0, Hk, Dk), "dv": e(0, Hv, Dv), "dg": torch.full_like(g, 7)})
    assert not bool(D["dg"].any())


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_on_a_device_that_is_not_current():
    lens, Hk, Hv, Dk, Dv, W = [70, 33], 1, 2, 32, 24, 4
    d, got = make(lens, Hk, Hv, Dk, Dv, W, False), []
    for dev in ("cuda:0", "cuda:1"):
        x = tree(d, lambda t: t.to(dev))
        got.append([t.cpu() for t in flat(step(ssp(), x, dc.cu_of(lens).to(dev), Hk, Hv, [seeds(0).to(dev), seeds(1).to(dev)]))])
    assert all(torch.equal(a, b) for a, b in zip(*got))
