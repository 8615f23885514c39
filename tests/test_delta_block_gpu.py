"""GPU: the calls of one gated delta rule block together (conv, head norms,
rule; forward, backward, carried states), as a training step makes them,
against the same block in 64 bits with torch's own conv1d and autograd."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc

pytestmark = pytest.mark.gpu

F32 = torch.float32


def ssp():
    import selective_state_space_varlen_amd as m
    return m


def make(lens, Hk, Hv, Dk, Dv, W, carry):
    gen = torch.Generator().manual_seed(60)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T, n = sum(lens), len(lens)
    widths = (Hk * Dk, Hk * Dk, Hv * Dv)
    return {"x": tuple(rnd(T, c) for c in widths), "w": tuple(0.5 * rnd(c, W) for c in widths),
            "b": tuple(0.1 * rnd(c) for c in widths), "g": -torch.exp(rnd(T, Hv) - 3), "beta": torch.sigmoid(rnd(T, Hv)),
            "dout": rnd(T, Hv, Dv),
            "states": {"delta": 0.3 * rnd(n, Hv, Dk, Dv), "conv": tuple(rnd(n, W - 1, c) for c in widths)} if carry
            else None,
            "dstates": {"delta": 0.3 * rnd(n, Hv, Dk, Dv), "conv": tuple(rnd(n, W - 1, c) for c in widths)} if carry
            else None}


def conv(x, w, b, lens, ctx):
    """SiLU of the causal depthwise conv of each sequence, and its last inputs."""
    W, outs, last, t = w.shape[1], [], [], 0
    for s, n in enumerate(lens):
        c = torch.zeros(W - 1, x.shape[1], dtype=x.dtype) if ctx is None else ctx[s]
        row = torch.cat([c, x[t:t + n]])
        y = torch.nn.functional.conv1d(row.t()[None], w[:, None], b, groups=x.shape[1])[0].t() if n else x[:0]
        outs.append(torch.nn.functional.silu(y))
        last.append(row[n:])
        t += n
    return torch.cat(outs), torch.stack(last)


def tree(t, f):
    if t is None:
        return None
    if isinstance(t, dict):
        return {k: tree(v, f) for k, v in t.items()}
    return tuple(tree(v, f) for v in t) if isinstance(t, tuple) else f(t)


def leaves(t):
    if isinstance(t, dict):
        return [x for v in t.values() for x in leaves(v)]
    return [x for v in t for x in leaves(v)] if isinstance(t, tuple) else [] if t is None else [t]


@pytest.mark.parametrize("carry", [False, True])
def test_block(carry):
    lens, Hk, Hv, Dk, Dv, W = [70, 1, 0, 33], 2, 4, 32, 24, 4
    d = make(lens, Hk, Hv, Dk, Dv, W, carry)
    m, cu = ssp(), dc.cu_of(lens).cuda()
    x = tree(d, lambda t: t.cuda())
    F = m.delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], cu, Hk, Hv, initial_states=x["states"])
    G = m.delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], F, x["dout"], dfinal_states=x["dstates"])
    torch.cuda.synchronize()

    r = tree(d, lambda t: t.to(dc.F64).requires_grad_())
    st = r["states"] or {}
    u, last = zip(*(conv(r["x"][i], r["w"][i], r["b"][i], lens, st["conv"][i] if carry else None) for i in range(3)))
    T = sum(lens)
    q, k = (dc.norm(u[i].view(T, Hk, Dk), None, None, None, True, 1e-6, False) for i in range(2))
    out, hT = dc.rule(q, k, u[2].view(T, Hv, Dv), r["g"], r["beta"], lens, Dk ** -0.5, st.get("delta"))
    loss = (out * r["dout"]).sum()
    if carry:
        loss = loss + (hT * r["dstates"]["delta"]).sum() + sum((a * b).sum() for a, b in zip(last, r["dstates"]["conv"]))
    want = {"dx": r["x"], "dw": r["w"], "db": r["b"], "dg": r["g"], "dbeta": r["beta"]}
    if carry:
        want["dinitial_states"] = r["states"]
    grads = iter(torch.autograd.grad(loss, leaves(want)))
    want = tree(want, lambda t: next(grads))
    # the chain's roundings: the rule's, a conv of W terms and a norm of Dk on
    # either side of it, each magnified by at most the norm's factor over the
    # smallest row (rows here are of size 1; 8 covers it)
    tol = 8 * dc.tol32(max(lens), Dk + W)
    dc.check(F["out"], out, tol, "out")
    for name in want:
        for a, b in zip(leaves(G[name]), leaves(want[name])):
            dc.check(a, b, tol, name)
    if carry:
        dc.check(F["final_states"]["delta"], hT, tol, "state")
        for a, b in zip(F["final_states"]["conv"], last):
            dc.check(a, b, 0.0, "conv context")


def test_block_in_two_packs():
    """Sequences cut at a pack's end: states forward, their gradients back."""
    Hk, Hv, Dk, Dv, W, lens, cut = 1, 2, 64, 64, 4, [90, 40], [50, 40]
    d = make(lens, Hk, Hv, Dk, Dv, W, False)
    m = ssp()
    x = tree(d, lambda t: t.cuda())
    whole = m.delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], dc.cu_of(lens).cuda(), Hk, Hv)
    gw = m.delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], whole, x["dout"])
    first = torch.cat([torch.arange(50), torch.arange(90, 130)]).cuda()
    second = torch.arange(50, 90).cuda()
    pick = lambda i: tree({"x": x["x"], "g": x["g"], "beta": x["beta"], "dout": x["dout"]}, lambda t: t[i])  # noqa: E731
    a, b = pick(first), pick(second)
    Fa = m.delta_forward(a["x"], x["w"], x["b"], a["g"], a["beta"], dc.cu_of(cut).cuda(), Hk, Hv, final_states=True)
    st = tree(Fa["final_states"], lambda t: t[:1].contiguous())
    Fb = m.delta_forward(b["x"], x["w"], x["b"], b["g"], b["beta"], dc.cu_of([40]).cuda(), Hk, Hv, initial_states=st)
    Gb = m.delta_backward(b["x"], x["w"], x["b"], b["g"], b["beta"], Fb, b["dout"])
    back = tree(Gb["dinitial_states"], lambda t: torch.cat([t, torch.zeros_like(t)]))
    Ga = m.delta_backward(a["x"], x["w"], x["b"], a["g"], a["beta"], Fa, a["dout"], dfinal_states=back)
    torch.cuda.synchronize()
    tol = 8 * dc.tol32(90, Dk + W)
    dc.check(Fa["out"], whole["out"].cpu()[first.cpu()], tol, "out")
    dc.check(Fb["out"], whole["out"].cpu()[second.cpu()], tol, "out")
    for i in range(3):
        dc.check(Ga["dx"][i], gw["dx"][i].cpu()[first.cpu()], tol, "dx")
        dc.check(Gb["dx"][i], gw["dx"][i].cpu()[second.cpu()], tol, "dx")
        dc.check(Ga["dw"][i] + Gb["dw"][i], gw["dw"][i].cpu(), tol, "dw")
    dc.check(Ga["dg"], gw["dg"].cpu()[first.cpu()], tol, "dg")
    dc.check(Gb["dbeta"], gw["dbeta"].cpu()[second.cpu()], tol, "dbeta")


def test_block_without_tokens():
    """No rows, two sequences: states go through as they are, weights get no gradient."""
    Hk, Hv, Dk, Dv, W = 1, 2, 32, 24, 4
    d = make([0, 0], Hk, Hv, Dk, Dv, W, True)
    m, cu = ssp(), dc.cu_of([0, 0]).cuda()
    x = tree(d, lambda t: t.cuda())
    F = m.delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], cu, Hk, Hv, initial_states=x["states"])
    G = m.delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], F, x["dout"], dfinal_states=x["dstates"])
    torch.cuda.synchronize()
    assert F["out"].shape == (0, Hv, Dv)
    for a, b in zip(leaves(F["final_states"]), leaves(x["states"])):
        assert torch.equal(a, b)
    for a, b in zip(leaves(G["dinitial_states"]), leaves(x["dstates"])):
        assert torch.equal(a, b)
    for t in G["dw"] + G["db"]:
        assert not bool(t.any())


def test_a_forward_that_kept_nothing_has_no_backward():
    Hk, Hv, Dk, Dv = 1, 1, 16, 8
    d = make([5], Hk, Hv, Dk, Dv, 4, False)
    x = tree(d, lambda t: t.cuda())
    F = ssp().delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], dc.cu_of([5]).cuda(), Hk, Hv, save=False)
    with pytest.raises(ValueError, match="save=True"):
        ssp().delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], F, x["dout"])
