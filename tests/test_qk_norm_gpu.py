"""GPU: the head norms with rotation against their definition in 64 bits.

Tolerances: one row's norm is a sum of D squares and a few factors. Its
rounding, and that of the turned pair, is at most (D / 2 + 16) 2^-24 of the
row's largest component in 32 bits (the sum of squares errs by D 2^-24 of
itself at most, its root by half of that); a bf16 result by half a step more.
The gradient adds a second sum of D terms over the row: twice as much, of the
largest gradient times the largest normed component squared over the mean
square (one with unit rows). The weights' gradients are sums of N terms whose
roundings are independent: 4 sqrt(N) 2^-24 of the largest term."""
from __future__ import annotations

import math

import pytest
import torch

from tests import delta_checks as dc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def ssp():
    import selective_state_space_varlen_amd as m
    return m


def make(seed, T, Hq, Hk, D, rot, dtype, weights, far=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {"q": rnd(T, Hq, D).to(dtype), "k": (3 * rnd(T, Hk, D)).to(dtype), "dyq": rnd(T, Hq, D).to(dtype),
         "dyk": rnd(T, Hk, D).to(dtype), "wq": 1 + 0.2 * rnd(D) if weights else None,
         "wk": 1 + 0.2 * rnd(D) if weights else None, "pos": None, "inv_freq": None}
    if rot:
        d["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
        d["pos"] = (torch.randint(0, 4096, (T,), generator=gen) + far).to(torch.int32)
    return d


def reference(d, l2, eps, inter):
    res = {}
    for n in ("q", "k"):
        x = d[n].to(dc.F64).requires_grad_()
        w = None if d["w" + n] is None else d["w" + n].to(dc.F64).requires_grad_()
        y = dc.norm(x, w, d["pos"], d["inv_freq"], l2, eps, inter)
        res["y" + n] = y.detach()
        if y.numel():
            g = torch.autograd.grad((y * d["dy" + n].to(dc.F64)).sum(), [x] + ([] if w is None else [w]))
        else:
            g = [torch.zeros_like(x)] + ([] if w is None else [torch.zeros_like(w)])
        res["d" + n] = g[0]
        if w is not None:
            res["dw" + n] = g[1]
    return res


def run(d, l2, eps, inter, inplace=False):
    m = ssp()
    x = {n: None if t is None else t.cuda() for n, t in d.items()}
    kw = dict(wq=x["wq"], wk=x["wk"], pos=x["pos"], inv_freq=x["inv_freq"], eps=eps, interleaved=inter,
              norm=m.SSMP_NORM_L2 if l2 else m.SSMP_NORM_RMS)
    nan = lambda t: None if t is None else torch.full_like(t, float("nan"))  # noqa: E731
    if inplace:
        out = (x["q"].clone(), x["k"].clone())
        y = m.qk_norm_pack_fwd(*out, out=out, **kw)
        g = {"dq": x["dyq"].clone(), "dk": x["dyk"].clone(), "dwq": nan(x["wq"]), "dwk": nan(x["wk"])}
        G = m.qk_norm_pack_bwd(x["q"], x["k"], g["dq"], g["dk"], out=g, **kw)
    else:
        y = m.qk_norm_pack_fwd(x["q"], x["k"], out=(nan(x["q"]), nan(x["k"])), **kw)
        T, Hq, D = x["q"].shape
        ws = torch.full((max(m.qk_norm_pack_bwd_workspace_bytes(T, Hq, x["k"].shape[1], D), 1),), 255,
                        dtype=torch.uint8, device="cuda")
        G = m.qk_norm_pack_bwd(x["q"], x["k"], x["dyq"], x["dyk"], workspace=ws,
                               out={"dq": nan(x["q"]), "dk": nan(x["k"]), "dwq": nan(x["wq"]), "dwk": nan(x["wk"])},
                               **kw)
    torch.cuda.synchronize()
    return {"yq": y[0], "yk": y[1], **G}


def compare(got, ref, d, l2):
    D = d["q"].shape[2]
    tol = (D / 2 + 16) * 2.0 ** -24
    for n in ("q", "k"):
        if not ref["y" + n].numel():
            continue
        x = d[n].to(dc.F64)
        rows = x.square().sum(-1, keepdim=True).sqrt()
        r = (1.0 if l2 else math.sqrt(D)) / rows  # the norm's factor, eps aside
        dc.check(got["y" + n], ref["y" + n], tol, "y" + n)
        peak = float((x.abs() / rows).max()) ** 2 * D
        dc.check(got["d" + n], ref["d" + n], 2 * tol * max(peak, 1.0), "d" + n,
                 scale=float(r.max()) * float(d["dy" + n].abs().max()) * 2)
        if d["w" + n] is not None:
            N = x.shape[0] * x.shape[1]
            term = float(d["dy" + n].abs().max()) * float((x.abs() * r).max()) * 2
            dc.check(got["dw" + n], ref["dw" + n], (4 * math.sqrt(N) + D) * 2.0 ** -24, "dw" + n, scale=term)


CASES = [
    # T, Hq, Hk, D, rot, interleaved, l2, weights
    (1, 1, 1, 8, 0, False, True, False),
    (1, 16, 16, 128, 0, False, True, False),
    (3, 6, 2, 72, 48, True, False, True),
    (5, 3, 1, 80, 80, False, False, True),
    (17, 4, 4, 128, 64, False, True, True),
    (33, 5, 0, 64, 64, False, False, True),
    (33, 0, 3, 64, 32, True, True, False),
    (70, 2, 1, 256, 256, False, False, False),
    (9, 7, 7, 512, 128, False, False, True),
    (130, 1, 1, 40, 2, True, False, True),
    (64, 33, 31, 16, 16, False, True, True),
    (0, 2, 2, 64, 32, False, False, True),
    (700, 8, 2, 128, 128, False, False, True),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_definition(case, dtype):
    T, Hq, Hk, D, rot, inter, l2, weights = CASES[case]
    d = make(case, T, Hq, Hk, D, rot, dtype, weights)
    ref = reference(d, l2, 1e-6, inter)
    got = run(d, l2, 1e-6, inter)
    compare(got, ref, d, l2)
    if T == 0 and weights:
        assert not bool(got["dwq"].any()) and not bool(got["dwk"].any())
    same = run(d, l2, 1e-6, inter, inplace=True)
    for n, t in got.items():
        assert t is None or torch.equal(t, same[n]), n


@pytest.mark.parametrize("far", [-4096, 1000000, 2 ** 31 - 4096])
def test_far_positions(far):
    d = make(50, 40, 2, 1, 64, 64, F32, False, far=far)
    got, ref = run(d, False, 1e-6, False), reference(d, False, 1e-6, False)
    compare(got, ref, d, False)


def test_many_workgroups_add_weight_gradients():
    d = make(51, 9000, 3, 1, 64, 0, F32, True)
    compare(run(d, False, 1e-6, False), reference(d, False, 1e-6, False), d, False)


def test_only_one_weight():
    d = make(52, 30, 2, 2, 64, 32, BF, True)
    d["wk"] = None
    got = run(d, True, 1e-6, False)
    assert got["dwk"] is None
    compare(got, reference(d, True, 1e-6, False), d, True)


def test_zero_rows_and_bad_rows():
    """A zero row gives zeros (eps > 0); NaN and infinities stay in their row,
    and no lane without a row adds to the weights' gradients when eps = 0."""
    d = make(53, 20, 3, 1, 72, 32, F32, True)
    clean = run(d, False, 1e-6, False)
    d["q"][4, 1] = 0.0
    d["q"][7, 2, 5] = float("nan")
    d["k"][9, 0, 70] = float("inf")
    got = run(d, False, 1e-6, False)
    assert not bool(got["yq"][4, 1].any())
    keep = torch.ones(20, 3, dtype=torch.bool)
    keep[4, 1] = keep[7, 2] = False
    for n in ("yq", "dq"):
        assert torch.equal(got[n].cpu()[keep], clean[n].cpu()[keep])
    keep = torch.ones(20, 1, dtype=torch.bool)
    keep[9] = False
    for n in ("yk", "dk"):
        assert torch.equal(got[n].cpu()[keep], clean[n].cpu()[keep])
    d = make(54, 3, 3, 2, 72, 0, F32, True)
    compare(run(d, False, 0.0, False), reference(d, False, 0.0, False), d, False)


def test_gradients_against_differences():
    d = make(55, 6, 2, 1, 24, 16, F32, True)
    got = run(d, True, 1e-6, False)
    gen = torch.Generator().manual_seed(56)
    for n in ("q", "k"):
        for leaf, gname in ((n, "d" + n), ("w" + n, "dw" + n)):
            x = d[leaf].to(dc.F64)
            v = torch.randn(x.shape, generator=gen, dtype=dc.F64)

            def loss(h):
                e = {**d, leaf: x + h * v}
                y = dc.norm(e[n], e["w" + n], d["pos"], d["inv_freq"], True, 1e-6, False)
                return float((y * d["dy" + n].to(dc.F64)).sum())

            diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
            mine = got[gname].cpu().to(dc.F64)
            assert abs(float((mine * v).sum()) - diff) <= 64 * 2.0 ** -24 * float(mine.abs().max()) * float(v.norm()) + 1e-9, gname


def test_captured_and_replayed():
    m = ssp()
    d = {n: None if t is None else t.cuda() for n, t in make(57, 50, 4, 2, 64, 32, BF, True).items()}
    kw = dict(wq=d["wq"], wk=d["wk"], pos=d["pos"], inv_freq=d["inv_freq"])

    def work():
        y = m.qk_norm_pack_fwd(d["q"], d["k"], **kw)
        return [*y, *m.qk_norm_pack_bwd(d["q"], d["k"], d["dyq"], d["dyk"], **kw).values()]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(4):
        d["q"].add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        ref = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
