"""GPU: the forms of a gated delta rule block: norms with weights, heads turned
in halves or in adjacent pairs, positions of the caller's, convs without
biases, states given in part, bf16; against the same block in 64 bits.

Tolerances. fp32 as in test_delta_block_gpu. In bf16 the block rounds what each
of its calls returns: forward the convs, the norms and the rule, backward the
rule, the norms and the convs. A rounding is at most 2^-8 of a value, hence of
the root of a tensor's summed squares; six of them lie on a gradient's way, which
is formed from values of both directions (twice), and the norm, SiLU and the
rule at these sizes magnify a relative error by less than two: 24 * 2^-8 of the
tensor's root of summed squares."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc
from tests.test_delta_block_gpu import conv, leaves, make, ssp, tree

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LENS, HK, HV, DK, DV, W = [70, 1, 0, 33], 2, 4, 32, 24, 4


def inputs(dtype, carry, bias, weights, l2):
    d = make(LENS, HK, HV, DK, DV, W, carry)
    gen = torch.Generator().manual_seed(61)
    # an RMS norm's rows are sqrt(Dk) long: its weights bring the keys back to 1
    d["nw"] = tuple((1 + 0.2 * torch.randn(DK, generator=gen)) * (1.0 if l2 else DK ** -0.5) if on else None
                    for on in weights)
    if not bias:
        d["b"] = None
    d["x"], d["dout"] = tree(d["x"], lambda t: t.to(dtype)), d["dout"].to(dtype)
    for s in ("states", "dstates"):
        if d[s] is not None:
            d[s]["conv"] = tree(d[s]["conv"], lambda t: t.to(dtype))
    return d


def reference(d, lens, pos, inv, l2, inter):
    """(values, gradients) of the block in 64 bits, in the layout of the calls' results."""
    r = tree(d, lambda t: t.to(dc.F64).requires_grad_())
    st = r["states"] or {}
    ctx = st.get("conv")
    b = r["b"] or (None,) * 3
    u, last = zip(*(conv(r["x"][i], r["w"][i], b[i], lens, None if ctx is None else ctx[i]) for i in range(3)))
    T = sum(lens)
    q, k = (dc.norm(u[i].view(T, HK, DK), r["nw"][i], pos, inv, l2, 1e-6, inter) for i in range(2))
    out, hT = dc.rule(q, k, u[2].view(T, HV, DV), r["g"], r["beta"], lens, DK ** -0.5, st.get("delta"))
    loss = (out * r["dout"]).sum()
    if r["dstates"] is not None:
        loss = loss + (hT * r["dstates"]["delta"]).sum() + sum((p * s).sum() for p, s in zip(last, r["dstates"]["conv"]))
    want = {"dx": r["x"], "dw": r["w"], "db": r["b"], "dg": r["g"], "dbeta": r["beta"], "dwq": r["nw"][0],
            "dwk": r["nw"][1], "dinitial_states": r["states"]}
    grads = iter(torch.autograd.grad(loss, leaves(want)))
    return {"out": out.detach(), "final_states": {"delta": hT.detach(), "conv": last}}, tree(want, lambda t: next(grads))


def near(got, want, dtype, name):
    if dtype == F32:
        return dc.check(got, want, 8 * dc.tol32(max(LENS), DK + W), name)
    g, r = got.detach().cpu().to(dc.F64), want.detach()
    assert g.shape == r.shape, name
    off, size = float((g - r).norm()), float(r.norm())
    assert off <= 24 * 2.0 ** -8 * size, f"{name}: {off:.3e} of {size:.3e}"


FORMS = [
    # l2, weights of q and k, rot, interleaved, caller's pos, biases, carried states
    (True, (True, True), 0, False, False, True, False),
    (True, (False, False), 32, False, False, True, False),
    (True, (True, False), 16, False, True, False, True),
    (True, (False, True), 32, True, False, True, True),
    (False, (True, True), 16, True, True, True, False),
    (False, (True, True), 32, False, False, False, False),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_forms(form, dtype):
    l2, weights, rot, inter, far, bias, carry = FORMS[form]
    d = inputs(dtype, carry, bias, weights, l2)
    inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None
    start = [0, 500, 3, 40] if far else [0] * 4
    pos = torch.cat([torch.arange(n) + s for n, s in zip(LENS, start)]).to(torch.int32)
    m, cu = ssp(), dc.cu_of(LENS).cuda()
    x = tree(d, lambda t: t.cuda())
    kw = {} if not inter else {"interleaved": True}
    F = m.delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], cu, HK, HV, pos=pos.cuda() if far else None,
                        norm=m.SSMP_NORM_L2 if l2 else m.SSMP_NORM_RMS, norm_weights=x["nw"],
                        inv_freq=None if inv is None else inv.cuda(), initial_states=x["states"], **kw)
    G = m.delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], F, x["dout"], dfinal_states=x["dstates"])
    torch.cuda.synchronize()
    values, grads = reference(d, LENS, pos, inv, l2, inter)
    near(F["out"], values["out"], dtype, "out")
    assert (G["db"] is None) == (not bias)
    assert (G["dwq"] is None, G["dwk"] is None) == (not weights[0], not weights[1])
    for name, want in grads.items():
        for a, b in zip(leaves(G.get(name)), leaves(want), strict=True):
            near(a, b, dtype, name)
    if carry:
        near(F["final_states"]["delta"], values["final_states"]["delta"], dtype, "state")
        for a, b in zip(F["final_states"]["conv"], values["final_states"]["conv"]):
            dc.check(a, b, 0.0, "conv context")  # the inputs themselves


@pytest.mark.parametrize("given", ["delta", "conv"])
def test_one_of_the_states_given(given):
    """The other one is zeros; gradients come back for both."""
    d = inputs(F32, True, True, (False, False), True)
    m, cu = ssp(), dc.cu_of(LENS).cuda()
    part = {given: d["states"][given]}
    d["states"] = {**tree(d["states"], torch.zeros_like), **part}
    x = tree(d, lambda t: t.cuda())
    F = m.delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], cu, HK, HV, initial_states=tree(part, lambda t: t.cuda()))
    G = m.delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], F, x["dout"], dfinal_states=x["dstates"])
    torch.cuda.synchronize()
    values, grads = reference(d, LENS, None, None, True, False)
    near(F["out"], values["out"], F32, "out")
    near(F["final_states"]["delta"], values["final_states"]["delta"], F32, "state")
    for name, want in grads.items():
        for a, b in zip(leaves(G.get(name)), leaves(want), strict=True):
            near(a, b, F32, name)


@pytest.mark.parametrize("inter", [False, True])
def test_turned_block_in_two_packs(inter):
    """A sequence cut at a pack's end: the second pack's positions go on."""
    n, cut = 90, 50
    d = make([n], HK, HV, DK, DV, W, False)
    m = ssp()
    x = tree(d, lambda t: t.cuda())
    inv = torch.tensor([1.0, 0.3, 0.05, 0.01, 0.9, 0.2, 0.002, 0.5]).cuda()

    def block(rows, st, pos, **kw):
        y = tree({n: x[n] for n in ("x", "g", "beta")}, lambda t: t[rows])
        return m.delta_forward(y["x"], x["w"], x["b"], y["g"], y["beta"], dc.cu_of([rows.stop - rows.start]).cuda(),
                               HK, HV, pos=pos, inv_freq=inv, interleaved=inter, initial_states=st, **kw)

    whole = block(slice(0, n), None, None)
    a = block(slice(0, cut), None, None, final_states=True)
    b = block(slice(cut, n), a["final_states"], torch.arange(cut, n, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    dc.check(torch.cat([a["out"], b["out"]]), whole["out"].cpu(), 8 * dc.tol32(n, DK + W), "out")


def test_block_captured_and_replayed():
    """Forward and backward in one graph, over other values and another division of the rows."""
    d = inputs(BF, True, True, (True, True), True)
    inv = torch.tensor([1.0, 0.3, 0.05, 0.01, 0.9, 0.2, 0.002, 0.5]).cuda()
    m, cu = ssp(), dc.cu_of(LENS).cuda()
    x = tree(d, lambda t: t.cuda())

    def once():
        F = m.delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], cu, HK, HV, norm_weights=x["nw"], inv_freq=inv,
                            interleaved=True, initial_states=x["states"])
        G = m.delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], F, x["dout"], dfinal_states=x["dstates"])
        return leaves({"out": F["out"], "states": F["final_states"], "G": G})

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once()
    for lens in ([70, 1, 0, 33], [5, 64, 35, 0], [0, 0, 0, 104], [70, 1, 0, 33]):
        cu.copy_(dc.cu_of(lens))
        x["x"][0].mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got]
        want = once()
        torch.cuda.synchronize()
        for a, b in zip(mine, want, strict=True):
            assert torch.equal(a, b)
