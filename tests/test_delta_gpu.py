"""GPU: the gated delta rule (chunked forward and backward, single-token step)
against its definition in 64 bits. Buffers start as NaN, so that a value that
was not written, or was read before it was written, shows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import delta_checks as dc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def ssp():
    import selective_state_space_varlen_amd as m
    return m


def dev(d):
    return {n: None if t is None else t.cuda() for n, t in d.items()}


def poison(nbytes):
    return torch.full((max(nbytes, 1),), 255, dtype=torch.uint8, device="cuda")


def nan_like(t):
    return torch.full_like(t, float("nan"))


def run(d, cu, carry, scale=None):
    """Forward and backward on poisoned buffers."""
    m = ssp()
    T, Hk, Dk = d["q"].shape
    Hv, Dv = d["v"].shape[1:]
    n = cu.numel() - 1
    state = (n, Hv, Dk, Dv)
    nan_state = lambda: torch.full(state, float("nan"), device="cuda") if carry else False  # noqa: E731
    out, saved, hT = m.gated_delta_pack_fwd(
        d["q"], d["k"], d["v"], d["g"], d["beta"], cu, scale=scale, initial_state=d["h0"], final_state=nan_state(),
        saved=poison(m.gated_delta_pack_saved_bytes(T, n, Hk, Hv, Dk, Dv)), out=nan_like(d["v"]),
        scratch=poison(m.gated_delta_pack_fwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, d["q"].dtype)))
    G = m.gated_delta_pack_bwd(
        d["q"], d["k"], d["g"], d["beta"], cu, d["dout"], saved, scale=scale, dfinal_state=d["dhT"],
        dinitial_state=nan_state(),
        scratch=poison(m.gated_delta_pack_bwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, d["q"].dtype)),
        out={"dq": nan_like(d["q"]), "dk": nan_like(d["k"]), "dv": nan_like(d["v"]), "dg": nan_like(d["g"]),
             "dbeta": nan_like(d["beta"])})
    torch.cuda.synchronize()
    return {"out": out, "hT": hT, "dh0": G.pop("dinitial_state"), **G}


def compare(got, ref, d, lens, carry, Dk):
    T = sum(lens)
    tol = dc.tol32(max(lens, default=0), Dk)
    r = d["v"].shape[1] // d["q"].shape[1]
    for n in ("out", "dq", "dk", "dv", "dbeta"):
        # dq and dk add r heads
        dc.check(got[n][:T], ref[n], (tol + dc.tol_parts(n, got[n].dtype)) * (r if n in ("dq", "dk") else 1), n)
    # dg sums what reads and writes a state, dq.q and dk.k, with both signs
    terms = sum(float((ref[a].abs() * d[b][:T].to(dc.F64).abs()).sum(-1).max()) if T else 0.0
                for a, b in (("dq", "q"), ("dk", "k")))
    dc.check(got["dg"][:T], ref["dg"], tol, "dg", scale=max(terms, float(ref["dg"].abs().max()) if T else 0.0))
    if carry:
        dc.check(got["hT"], ref["hT"], tol, "hT")
        dc.check(got["dh0"], ref["dh0"], tol, "dh0")


CASES = [
    # lens, Hk, Hv, Dk, Dv
    ([1], 1, 1, 8, 8),
    ([2, 1], 1, 2, 64, 64),
    ([63, 64, 65], 2, 2, 64, 32),
    ([130], 1, 1, 128, 128),
    ([0, 5, 0, 0, 70, 1, 0], 2, 4, 72, 40),
    ([0, 0], 1, 1, 64, 64),
    ([200, 129], 1, 3, 40, 136),
    ([3, 300], 2, 2, 128, 64),
    ([64] * 5, 1, 2, 128, 24),
    ([17] * 9, 3, 3, 120, 72),
]


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_chunked_matches_definition(case, dtype, carry):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    d = dc.rule_inputs(100 + case, lens, Hk, Hv, Dk, Dv, dtype, carry)
    ref = dc.rule_reference(d, lens, Dk ** -0.5)
    compare(run(dev(d), dc.cu_of(lens).cuda(), carry), ref, d, lens, carry, Dk)


@pytest.mark.parametrize("what", ["beta0", "beta_some0", "beta1_same_keys", "reset", "lowest", "fast", "slow", "k0"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_limits_of_gates_and_decays(what, dtype):
    lens, Hk, Hv, Dk, Dv = [150, 70], 1, 2, 64, 40
    d = dc.rule_inputs(7, lens, Hk, Hv, Dk, Dv, dtype, True)
    T = sum(lens)
    if what == "beta0":
        d["beta"].zero_()
    elif what == "beta_some0":
        d["beta"][::3] = 0.0
    elif what == "beta1_same_keys":  # the inverse of the all-ones triangle
        d["beta"].fill_(1.0)
        d["k"][:] = d["k"][:1]
        d["g"].zero_()
    elif what == "reset":
        d["g"][5::17] = float("-inf")
        d["g"][64] = float("-inf")
        d["g"][0] = float("-inf")
    elif what == "lowest":
        d["g"][5::17] = torch.finfo(F32).min
    elif what == "fast":  # large decays before small ones: differences of far running sums
        d["g"][:] = -30.0
        d["g"][32:64] = -0.01
        d["g"][100:120] = -0.001
    elif what == "slow":
        d["g"].zero_()
    elif what == "k0":
        d["k"][10:90] = 0.0
    ref = dc.rule_reference(d, lens, 0.3)
    compare(run(dev(d), dc.cu_of(lens).cuda(), True, scale=0.3), ref, d, lens, True, Dk)
    assert T == ref["out"].shape[0]


def test_gradients_against_differences():
    """The kernels' gradients along a random direction against central
    differences of the 64-bit definition."""
    lens, Hk, Hv, Dk, Dv = [70, 9], 1, 2, 16, 24
    d = dc.rule_inputs(3, lens, Hk, Hv, Dk, Dv, F32, True)
    got = run(dev(d), dc.cu_of(lens).cuda(), True)
    gen = torch.Generator().manual_seed(4)
    names = {"q": "dq", "k": "dk", "v": "dv", "g": "dg", "beta": "dbeta", "h0": "dh0"}
    for n, gn in names.items():
        x = {m: d[m].to(dc.F64) for m in names}
        dirn = torch.randn(x[n].shape, generator=gen, dtype=dc.F64)

        def loss(step):
            y = dict(x)
            y[n] = x[n] + step * dirn
            o, h = dc.rule(y["q"], y["k"], y["v"], y["g"], y["beta"], lens, Dk ** -0.5, y["h0"])
            return float((o * d["dout"].to(dc.F64)).sum() + (h * d["dhT"].to(dc.F64)).sum())

        h = 1e-5  # truncation h^2, rounding 2^-53 / h: both far below the 32-bit gradients' own error
        diff = (loss(h) - loss(-h)) / (2 * h)
        mine = got[gn].cpu().to(dc.F64)
        # independent errors of tol32 of the largest entry each, along the direction
        room = dc.tol32(70, Dk) * float(mine.abs().max()) * float(dirn.norm()) * 4
        assert abs(float((mine * dirn).sum()) - diff) <= room, n


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_behind_the_last_sequence(dtype):
    lens, Hk, Hv, Dk, Dv, tail = [70, 33], 1, 2, 64, 40, 50
    d = dc.rule_inputs(11, lens, Hk, Hv, Dk, Dv, dtype, True, tail=tail)
    ref = dc.rule_reference(d, lens, Dk ** -0.5)
    for n in ("q", "k", "v", "g", "beta", "dout"):
        d[n][sum(lens):] = float("nan")
    got = run(dev(d), dc.cu_of(lens).cuda(), True)
    compare(got, ref, d, lens, True, Dk)
    for n in ("out", "dq", "dk", "dv", "dg", "dbeta"):
        assert bool(got[n][sum(lens):].isnan().all()), n  # as they were


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_sequence(bad):
    lens, Hk, Hv, Dk, Dv = [40, 100, 30], 1, 2, 64, 64
    d = dc.rule_inputs(12, lens, Hk, Hv, Dk, Dv, BF, True)
    ref = run(dev(d), dc.cu_of(lens).cuda(), True)
    d["v"][90], d["k"][60] = bad, bad
    got = run(dev(d), dc.cu_of(lens).cuda(), True)
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[40:140] = False
    for n in ("out", "dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[n].cpu()[keep], ref[n].cpu()[keep]), n
    for n in ("hT", "dh0"):
        assert torch.equal(got[n][[0, 2]], ref[n][[0, 2]]), n


def test_later_tokens_do_not_reach_earlier_outputs():
    lens, Hk, Hv, Dk, Dv = [150], 1, 1, 64, 64
    d = dc.rule_inputs(13, lens, Hk, Hv, Dk, Dv, BF, False)
    cu = dc.cu_of(lens).cuda()
    a = run(dev(d), cu, False)["out"]
    for n in ("q", "k", "v", "g", "beta"):
        d[n][100:] = d[n][100:].flip(0)
    b = run(dev(d), cu, False)["out"]
    assert torch.equal(a[:100], b[:100]) and not torch.equal(a[100:], b[100:])


def test_a_sequence_in_pieces():
    """A sequence cut in three, its state handed on, and its gradients handed back."""
    Hk, Hv, Dk, Dv, T = 1, 2, 64, 40, 190
    d = dc.rule_inputs(14, [T], Hk, Hv, Dk, Dv, F32, True)
    ref = dc.rule_reference(d, [T], Dk ** -0.5)
    x = dev(d)
    m = ssp()
    cuts = [0, 50, 114, T]
    h, kept = x["h0"], []
    parts = {n: [] for n in ("out", "dq", "dk", "dv", "dg", "dbeta")}
    sl = lambda t, i: t[cuts[i]:cuts[i + 1]].contiguous()  # noqa: E731
    for i in range(3):
        cu = dc.cu_of([cuts[i + 1] - cuts[i]]).cuda()
        o, saved, h = m.gated_delta_pack_fwd(*(sl(x[n], i) for n in ("q", "k", "v", "g", "beta")), cu,
                                             initial_state=h, final_state=True, save=True)
        kept.append((cu, saved))
        parts["out"].append(o)
    dh = x["dhT"]
    for i in (2, 1, 0):
        cu, saved = kept[i]
        G = m.gated_delta_pack_bwd(sl(x["q"], i), sl(x["k"], i), sl(x["g"], i), sl(x["beta"], i), cu,
                                   sl(x["dout"], i), saved, dfinal_state=dh, dinitial_state=True)
        dh = G["dinitial_state"]
        for n in parts:
            if n != "out":
                parts[n].insert(0, G[n])
    got = {n: torch.cat(v) for n, v in parts.items()}
    compare({**got, "hT": h, "dh0": dh}, ref, d, [T], True, Dk)


def test_repeats_bit_for_bit_on_other_streams():
    lens, Hk, Hv, Dk, Dv = [90, 200, 5], 2, 4, 128, 64
    d = dev(dc.rule_inputs(15, lens, Hk, Hv, Dk, Dv, BF, True))
    cu = dc.cu_of(lens).cuda()
    ref = run(d, cu, True)
    torch.cuda.synchronize()
    m, got = ssp(), []
    streams = [torch.cuda.Stream() for _ in range(3)]
    for st in streams:  # in flight together
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            o, saved, h = m.gated_delta_pack_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu,
                                                 initial_state=d["h0"], final_state=True, save=True)
            G = m.gated_delta_pack_bwd(d["q"], d["k"], d["g"], d["beta"], cu, d["dout"], saved,
                                       dfinal_state=d["dhT"], dinitial_state=True)
            got.append({"out": o, "hT": h, "dh0": G.pop("dinitial_state"), **G})
    torch.cuda.synchronize()
    for g in got:
        for n, t in g.items():
            assert torch.equal(t, ref[n]), n


def test_captured_and_replayed():
    """One graph for any division of its T rows: cu_seqlens is read on the device."""
    Hk, Hv, Dk, Dv, T, n = 1, 2, 64, 64, 256, 4
    m = ssp()
    batches = []
    for i, lens in enumerate(([64, 64, 64, 64], [1, 200, 0, 55], [100, 30, 20, 10])):
        d = dc.rule_inputs(20 + i, lens, Hk, Hv, Dk, Dv, BF, False, tail=T - sum(lens))
        batches.append((dev(d), dc.cu_of(lens).cuda(), sum(lens)))
    static = {k: torch.empty_like(v) for k, v in batches[0][0].items() if v is not None}
    cu = torch.empty_like(batches[0][1])

    def load(b):
        for k in static:
            static[k].copy_(b[0][k])
        cu.copy_(b[1])

    def work():
        o, saved, h = m.gated_delta_pack_fwd(static["q"], static["k"], static["v"], static["g"], static["beta"], cu,
                                             final_state=True, save=True)
        G = m.gated_delta_pack_bwd(static["q"], static["k"], static["g"], static["beta"], cu, static["dout"], saved)
        return {"out": o, "hT": h, **{k: v for k, v in G.items() if v is not None}}

    load(batches[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for b in (0, 1, 2, 1, 0):
        load(batches[b])
        graph.replay()
        torch.cuda.synchronize()
        mine = {k: v.clone() for k, v in got.items()}
        ref = work()
        torch.cuda.synchronize()
        used = batches[b][2]
        for k in mine:
            rows = slice(None) if k == "hT" else slice(0, used)
            assert torch.equal(mine[k][rows], ref[k][rows]), (b, k)


def test_any_cu_seqlens_stays_in_bounds():
    """Boundaries that decrease or leave [0, T]: values mean nothing, but what
    lies around the buffers is as it was. Every index the kernels form from
    them is clamped first."""
    Hk, Hv, Dk, Dv, T = 1, 1, 64, 64, 200
    m = ssp()
    d = dev(dc.rule_inputs(21, [T], Hk, Hv, Dk, Dv, BF, False))
    for cu in ([0, 150, 100, 200], [-5, 70, 70, 900], [200, 0, 200, 0], [0, 0, 0, 0], [2 ** 31 - 1, -2 ** 31, 7, 9]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        big = torch.full((3 * T, Hv, Dv), 7.0, dtype=BF, device="cuda")
        o, saved, h = m.gated_delta_pack_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, final_state=True,
                                             save=True, out=big[T:2 * T])
        m.gated_delta_pack_bwd(d["q"], d["k"], d["g"], d["beta"], cu, d["dout"], saved)
        torch.cuda.synchronize()
        assert bool((big[:T] == 7).all()) and bool((big[2 * T:] == 7).all())


def test_no_tokens():
    m = ssp()
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    h0 = torch.randn(2, 2, 64, 8, device="cuda")
    q, v, g = e(0, 1, 64), e(0, 2, 8), e(0, 2)
    o, saved, h = m.gated_delta_pack_fwd(q, q, v, g, g, cu, initial_state=h0, final_state=True, save=True)
    assert o.shape == v.shape and torch.equal(h, h0)
    G = m.gated_delta_pack_bwd(q, q, g, g, cu, v, saved, dfinal_state=h0, dinitial_state=True)
    assert torch.equal(G["dinitial_state"], h0)


# ---------------------------------------------------------------------------
def step_reference(d, state, slots, scale):
    state = state.to(dc.F64).clone()
    outs = []
    for b, s in enumerate(slots):
        if not 0 <= s < state.shape[0]:
            outs.append(None)
            continue
        o, h = dc.rule(*(d[n][b:b + 1].to(dc.F64) for n in ("q", "k", "v", "g", "beta")), [1], scale, state[s:s + 1])
        state[s] = h[0]
        outs.append(o[0])
    return outs, state


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", [
    # B, slots of the pool, Hk, Hv, Dk, Dv, slot choice
    (1, 1, 1, 1, 8, 8, "none"), (1, 3, 2, 4, 128, 128, "perm"), (5, 5, 1, 3, 72, 40, "none"),
    (6, 9, 1, 2, 64, 24, "perm"), (9, 4, 1, 2, 128, 136, "twice"), (7, 5, 2, 2, 40, 32, "outside"),
    (300, 3, 1, 1, 16, 8, "twice"),
])
def test_step(case, dtype):
    B, pool, Hk, Hv, Dk, Dv, how = case
    d = dc.rule_inputs(30, [1] * B, Hk, Hv, Dk, Dv, dtype, False)
    gen = torch.Generator().manual_seed(31)
    state = 0.3 * torch.randn(pool, Hv, Dk, Dv, generator=gen)
    if how == "none":
        slots = list(range(B))
    elif how == "perm":
        slots = torch.randperm(pool, generator=gen)[:B].tolist()
    else:
        slots = torch.randint(0, pool, (B,), generator=gen).tolist()
        if how == "outside":
            slots[1], slots[4] = -1, pool
    outs, ref = step_reference(d, state, slots, Dk ** -0.5)
    x, st = dev(d), state.cuda()
    out = nan_like(x["v"])
    ssp().gated_delta_pack_step(x["q"], x["k"], x["v"], x["g"], x["beta"], st, out=out,
                                slots=None if how == "none" else torch.tensor(slots, dtype=torch.int32).cuda())
    # rows of one slot follow one another as the tokens of a sequence do
    tol = dc.tol32(max(np.bincount([s for s in slots if 0 <= s < pool])), Dk)
    dc.check(st, ref, tol, "state")
    top = max(float(o.abs().max()) for o in outs if o is not None)
    for b, o in enumerate(outs):
        if o is None:
            assert bool(out[b].isnan().all())
        else:
            dc.check(out[b], o, tol, f"out[{b}]", scale=top)
    for s in range(pool):
        if s not in slots:
            assert torch.equal(st[s].cpu(), state[s])


def test_step_continues_the_chunked_form():
    """A prompt through the chunks, then tokens one by one on its state."""
    Hk, Hv, Dk, Dv, P, N = 1, 2, 128, 64, 100, 6
    d = dc.rule_inputs(40, [P + N], Hk, Hv, Dk, Dv, BF, False)
    ref, hT = dc.rule(*(d[n].to(dc.F64) for n in ("q", "k", "v", "g", "beta")), [P + N], Dk ** -0.5)
    x, m = dev(d), ssp()
    part = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, _, h = m.gated_delta_pack_fwd(*(t[:P] for t in part), dc.cu_of([P]).cuda(), final_state=True)
    outs = [o]
    for t in range(P, P + N):
        outs.append(m.gated_delta_pack_step(*(y[t:t + 1] for y in part), h))
    tol = dc.tol32(P + N, Dk)
    dc.check(torch.cat(outs), ref, tol, "out")
    dc.check(h, hT, tol, "state")


def test_step_captured():
    B, Hk, Hv, Dk, Dv = 4, 1, 2, 64, 32
    m = ssp()
    x = dev(dc.rule_inputs(41, [1] * B, Hk, Hv, Dk, Dv, BF, False))
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    slots = torch.tensor([2, 0, 5, 1], dtype=torch.int32, device="cuda")
    st = torch.randn(6, Hv, Dk, Dv, device="cuda") * 0.3
    eager, out = st.clone(), torch.zeros_like(x["v"])
    m.gated_delta_pack_step(*args, st.clone(), slots=slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.gated_delta_pack_step(*args, st, slots=slots, out=out)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        ref = m.gated_delta_pack_step(*args, eager, slots=slots)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(st, eager)
