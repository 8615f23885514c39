"""GPU: the gated delta rule on few long sequences, whose chunks are split into
parts that are walked at once and joined."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc
from tests.test_delta_gpu import BF, F32, compare, dev, nan_like, run, ssp
from tests.test_delta_many_gpu import reference

pytestmark = pytest.mark.gpu

CASES = [
    # lens, Hk, Hv, Dk, Dv
    ([2100], 1, 2, 128, 72),              # one sequence, parts that do not divide it
    ([2048], 2, 2, 64, 64),               # parts that do
    ([3000, 0, 4200], 1, 1, 40, 24),      # an empty sequence between
    ([5, 9000, 0, 70], 1, 2, 24, 136),    # short ones beside a long one; three blocks of columns
]


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_split_matches_definition(case, dtype, carry):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    d = dc.rule_inputs(500 + case, lens, Hk, Hv, Dk, Dv, dtype, carry)
    # slow decays, so that what enters a part still counts when it leaves
    d["g"] *= 0.02
    ref = reference(d, lens, Dk ** -0.5)
    compare(run(dev(d), dc.cu_of(lens).cuda(), carry), ref, d, lens, carry, Dk)


@pytest.mark.parametrize("what", ["reset", "lowest", "slow", "beta1_same_keys", "beta0"])
def test_split_limits_of_gates_and_decays(what):
    lens, Hk, Hv, Dk, Dv = [2300], 1, 1, 32, 24
    d = dc.rule_inputs(520, lens, Hk, Hv, Dk, Dv, F32, True)
    d["g"] *= 0.02
    if what == "reset":
        d["g"][700] = float("-inf")
        d["g"][1024] = float("-inf")
    elif what == "lowest":
        d["g"][::400] = torch.finfo(F32).min
    elif what == "slow":
        d["g"].zero_()
    elif what == "beta1_same_keys":
        d["beta"].fill_(1.0)
        d["k"][:] = d["k"][:1]
        d["g"].zero_()
    elif what == "beta0":
        d["beta"].zero_()
    ref = reference(d, lens, 0.3)
    compare(run(dev(d), dc.cu_of(lens).cuda(), True, scale=0.3), ref, d, lens, True, Dk)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_split_bad_values_stay_in_their_sequence(bad):
    lens = [2400, 3000]
    d = dc.rule_inputs(530, lens, 1, 1, 32, 24, F32, True)
    good = run(dev(d), dc.cu_of(lens).cuda(), True)
    for n in ("v", "k", "dout"):
        d[n][1500] = bad
    got = run(dev(d), dc.cu_of(lens).cuda(), True)
    for n in ("out", "dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[n][2400:], good[n][2400:]), n
    assert torch.equal(got["out"][:1472], good["out"][:1472])  # whole chunks before the bad one
    assert torch.equal(got["hT"][1], good["hT"][1]) and torch.equal(got["dh0"][1], good["dh0"][1])


def test_split_rows_behind_the_last_sequence():
    lens, tail = [2500], 900
    d = dc.rule_inputs(531, lens, 1, 2, 64, 40, BF, False, tail=tail)
    d["g"] *= 0.02
    ref = reference(d, lens, 64 ** -0.5)
    got = run(dev(d), dc.cu_of(lens).cuda(), False)
    compare(got, ref, d, lens, False, 64)
    for n in ("out", "dq", "dk", "dv", "dg", "dbeta"):
        assert bool(got[n][2500:].isnan().all()), n


def test_split_any_cu_seqlens_stays_in_bounds():
    """Buffers between guards; values mean nothing, other memory keeps its own."""
    m = ssp()
    T, Hk, Hv, Dk, Dv = 4200, 1, 1, 16, 24
    d = dev(dc.rule_inputs(532, [T], Hk, Hv, Dk, Dv, F32, False))
    gen = torch.Generator().manual_seed(533)
    for _ in range(12):
        cu = torch.randint(-3000, 9000, (3,), generator=gen, dtype=torch.int32).cuda()
        nb = m.gated_delta_pack_fwd_scratch_bytes(T, 2, Hk, Hv, Dk, Dv, F32)
        room = torch.full((nb + 8192,), 77, dtype=torch.uint8, device="cuda")
        hold = torch.full((T + 128, Hv, Dv), 5.0, device="cuda")
        m.gated_delta_pack_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, final_state=True,
                               scratch=room[4096:4096 + nb], out=hold[64:64 + T])
        torch.cuda.synchronize()
        assert bool((room[:4096] == 77).all()) and bool((room[4096 + nb:] == 77).all())
        assert bool((hold[:64] == 5.0).all()) and bool((hold[64 + T:] == 5.0).all())


def test_split_in_pieces_and_captured():
    """A sequence in two calls, the state handed on, against one call; and both
    captured, replayed over other values and lengths."""
    m = ssp()
    T, Hk, Hv, Dk, Dv = 4608, 1, 2, 64, 64
    d = dev(dc.rule_inputs(540, [T], Hk, Hv, Dk, Dv, F32, False))
    d["g"] *= 0.02
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    cu = dc.cu_of([T]).cuda()
    out, hT = nan_like(d["v"]), torch.empty(1, Hv, Dk, Dv, device="cuda")
    ws = torch.empty(m.gated_delta_pack_fwd_scratch_bytes(T, 1, Hk, Hv, Dk, Dv, F32), dtype=torch.uint8, device="cuda")

    def once():
        m.gated_delta_pack_fwd(*args, cu, final_state=hT, out=out, scratch=ws)

    once()
    torch.cuda.synchronize()
    whole, state = out.clone(), hT.clone()
    cut = 2304
    half = dc.cu_of([cut]).cuda()
    a, _, s = m.gated_delta_pack_fwd(*[x[:cut].contiguous() for x in args], half, final_state=True)
    b, _, s = m.gated_delta_pack_fwd(*[x[cut:].contiguous() for x in args], half, initial_state=s, final_state=True)
    tol = dc.tol32(T, Dk)
    dc.check(torch.cat([a, b]), whole.cpu(), tol, "out")
    dc.check(s, state.cpu(), tol, "hT")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for i, n in enumerate((T, 2100, 0, 4000, T)):
        cu.copy_(dc.cu_of([n]))
        args[2].mul_(-1.0)
        out.fill_(float("nan"))
        hT.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        g_out, g_hT = out.clone(), hT.clone()
        out.fill_(float("nan"))
        once()
        torch.cuda.synchronize()
        assert torch.equal(g_out[:n], out[:n]) and bool(g_out[n:].isnan().all()), (i, n)
        assert torch.equal(g_hT, hT), (i, n)
        if n == T:  # v's sign has turned once, or five times; both sides are within tol of the exact values
            dc.check(g_out, -whole.cpu(), 2 * tol, "out")
            dc.check(g_hT, -state.cpu(), 2 * tol, "hT")


def test_two_graphs_share_a_scratch():
    """A split pack and a short one, captured on the same scratch and replayed
    in turn on one stream: each call leaves nothing there that the next reads."""
    m = ssp()
    Hk, Hv, Dk, Dv = 1, 2, 64, 40
    calls, outs, size = [], [], 0
    for lens in ([2304], [70, 0, 130]):
        d = dev(dc.rule_inputs(550 + len(lens), lens, Hk, Hv, Dk, Dv, BF, True))
        T, n = sum(lens), len(lens)
        size = max(size, m.gated_delta_pack_fwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, BF),
                   m.gated_delta_pack_bwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, BF))
        kept = torch.empty(m.gated_delta_pack_saved_bytes(T, n, Hk, Hv, Dk, Dv), dtype=torch.uint8, device="cuda")
        out = {"out": nan_like(d["v"]), "hT": nan_like(d["h0"]), "dh0": nan_like(d["h0"]),
               "grads": {"dq": nan_like(d["q"]), "dk": nan_like(d["k"]), "dv": nan_like(d["v"]),
                         "dg": nan_like(d["g"]), "dbeta": nan_like(d["beta"])}}
        calls.append((d, dc.cu_of(lens).cuda(), kept, out))
    scratch = torch.empty(size, dtype=torch.uint8, device="cuda")

    def call(d, cu, kept, out):
        m.gated_delta_pack_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, initial_state=d["h0"],
                               final_state=out["hT"], saved=kept, scratch=scratch, out=out["out"])
        m.gated_delta_pack_bwd(d["q"], d["k"], d["g"], d["beta"], cu, d["dout"], kept, dfinal_state=d["dhT"],
                               dinitial_state=out["dh0"], scratch=scratch, out=out["grads"])

    flat = lambda out: {"out": out["out"], "hT": out["hT"], "dh0": out["dh0"], **out["grads"]}  # noqa: E731
    graphs = []
    for c in calls:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(*c)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        outs.append({n: t.clone() for n, t in flat(c[3]).items()})
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(*c)
        graphs.append(graph)
    for turn in range(3):
        scratch.fill_(255)
        for c in calls:
            for t in flat(c[3]).values():
                t.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, want in zip(calls, outs):
            for n, t in flat(c[3]).items():
                assert torch.equal(t, want[n]), (turn, n)
