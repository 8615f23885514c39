"""GPU: linear attention with a decay (chunked forward and backward, single-token
step) against its definition in 64 bits. Buffers start as NaN, so that a value
that was not written, or was read before it was written, shows."""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck
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


def run(d, cu, carry, scale=None, dg=True):
    """Forward and backward on poisoned buffers."""
    m = ssp()
    T, Hk, Dk = d["q"].shape
    Hv, Dv = d["v"].shape[1:]
    n = cu.numel() - 1
    sizes = (T, n, Hk, Hv, Dk, Dv)
    nan_state = lambda: torch.full((n, Hv, Dk, Dv), float("nan"), device="cuda") if carry else False  # noqa: E731
    out, hT = m.decay_attn_pack_fwd(d["q"], d["k"], d["v"], d["g"], cu, scale=scale, initial_state=d["h0"],
                                    final_state=nan_state(), out=nan_like(d["v"]),
                                    scratch=poison(m.decay_attn_pack_fwd_scratch_bytes(*sizes)))
    G = m.decay_attn_pack_bwd(d["q"], d["k"], d["v"], d["g"], cu, d["dout"], scale=scale, initial_state=d["h0"],
                              dfinal_state=d["dhT"], dinitial_state=nan_state(),
                              scratch=poison(m.decay_attn_pack_bwd_scratch_bytes(*sizes)),
                              out={"dq": nan_like(d["q"]), "dk": nan_like(d["k"]), "dv": nan_like(d["v"]),
                                   "dg": nan_like(d["g"]) if dg else None})
    torch.cuda.synchronize()
    return {"out": out, "hT": hT, "dh0": G.pop("dinitial_state"), **G}


def compare(got, ref, d, lens, carry, dg=True):
    T, L = sum(lens), max(lens, default=0)
    Dk, (Hv, Dv) = d["q"].shape[2], d["v"].shape[1:]
    tol = ck.tol32(L, Dk, Dv)
    r = Hv // d["q"].shape[1]
    for n in ("out", "dq", "dk", "dv"):
        # dq and dk add r heads
        dc.check(got[n][:T], ref[n], (tol + ck.tol_parts(n, got[n].dtype, dg)) * (r if n in ("dq", "dk") else 1), n)
    if dg:
        top = max(ck.meets(d, ref, lens), float(ref["dg"].abs().max()) if ref["dg"].numel() else 0.0)
        if d["g"].dim() == 2:
            dc.check(got["dg"][:T], ref["dg"], tol * ck.rms_sum(L), "dg", scale=top)
        else:  # the sum of T such errors, those of 256 tokens alike
            dc.check(got["dg"], ref["dg"], tol * ck.rms_sum(L) * (max(T, 1) * min(max(T, 1), 256)) ** 0.5, "dg", scale=top)
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
    ([257, 256, 255, 513, 1], 1, 2, 16, 24),   # segments of 256, and pieces of them
    ([700], 1, 1, 64, 264),                    # value heads wider than a walk's state, twice
    ([1, 520], 2, 6, 24, 200),
]


@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_chunked_matches_definition(case, dtype, carry, per_token):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    d = ck.inputs(200 + case, lens, Hk, Hv, Dk, Dv, dtype, carry, per_token)
    ref = ck.reference(d, lens, Dk ** -0.5)
    compare(run(dev(d), dc.cu_of(lens).cuda(), carry), ref, d, lens, carry)


# More workgroups than the card has at a time: then the value heads of a key
# head that has two share one in dq's and dk's walks.
SHORT = [1, 0, 5, 64, 3, 17, 2, 40]


@pytest.mark.parametrize("dg", [True, False])
@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [
    (SHORT * 5 + [65, 300], 4, 8, 128, 128),
    (SHORT * 5 + [257], 4, 8, 64, 64),
    (SHORT * 5 + [64, 129], 6, 12, 128, 40),
    (SHORT * 5 + [200], 4, 8, 40, 128),
    (SHORT * 5, 6, 12, 8, 8),
    (SHORT * 3 + [70, 1], 3, 6, 72, 136),      # wide value heads, in slices: each alone
    (SHORT * 5 + [66], 2, 8, 72, 64),          # four
])
@pytest.mark.parametrize("carry,per_token", [(True, True), (False, False)])
def test_heads_in_pairs(lens, Hk, Hv, Dk, Dv, carry, per_token, dg):
    assert 2 * len(lens) * Hv * -(-Dv // 128) > 512
    d = ck.inputs(9, lens, Hk, Hv, Dk, Dv, BF, carry, per_token)
    ref = ck.reference(d, lens, 0.4)
    compare(run(dev(d), dc.cu_of(lens).cuda(), carry, scale=0.4, dg=dg), ref, d, lens, carry, dg)


@pytest.mark.parametrize("what", ["reset", "lowest", "fast", "slow", "none", "k0", "long_then_reset"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_limits_of_decays(what, dtype):
    lens, Hk, Hv, Dk, Dv = [350, 70], 1, 2, 64, 40
    d = ck.inputs(7, lens, Hk, Hv, Dk, Dv, dtype, True)
    if what == "reset":
        for t in (0, 5, 63, 64, 65, 255, 256, 257, 300, 349, 350, 419):
            d["g"][t] = float("-inf")
    elif what == "lowest":
        d["g"][5::17] = torch.finfo(F32).min
    elif what == "fast":  # large decays before small ones: differences of far running sums
        d["g"][:] = -30.0
        d["g"][32:64] = -0.01
        d["g"][100:120] = -0.001
    elif what == "slow":
        d["g"][:] = -1e-6
    elif what == "none":
        d["g"].zero_()
    elif what == "k0":
        d["k"][::2] = 0
    elif what == "long_then_reset":
        d["g"][:] = -1e-4
        d["g"][340] = float("-inf")
    x = dict(d, g=d["g"].clamp(min=-1e4))  # e^-1e4 = 0; -inf * 0 would be NaN in the reference's product rule
    ref = ck.reference(x, lens, 0.37)
    got = run(dev(d), dc.cu_of(lens).cuda(), True, scale=0.37)
    compare(got, ref, d, lens, True)
    gone = d["g"] < -100
    assert not bool(got["dg"].cpu()[gone].any())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_without_dg(dtype):
    lens, Hk, Hv, Dk, Dv = [300, 41], 2, 4, 72, 136
    d = ck.inputs(31, lens, Hk, Hv, Dk, Dv, dtype, True)
    got = run(dev(d), dc.cu_of(lens).cuda(), True, dg=False)
    assert got["dg"] is None
    compare(got, ck.reference(d, lens, Dk ** -0.5), d, lens, True, dg=False)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_behind_the_last_sequence_stay(dtype):
    lens, Hk, Hv, Dk, Dv = [70, 30, 290], 1, 3, 32, 48
    d = ck.inputs(5, lens, Hk, Hv, Dk, Dv, dtype, False, tail=77)
    T = sum(lens)
    for n in ("q", "k", "v", "g", "dout"):
        d[n][T:] = float("nan")
    got = run(dev(d), dc.cu_of(lens).cuda(), False)
    compare(got, ck.reference(d, lens, Dk ** -0.5), d, lens, False)
    for n in ("out", "dq", "dk", "dv", "dg"):
        assert bool(got[n][T:].isnan().all()), n


def test_sequences_do_not_meet():
    """A NaN stays in its sequence, and results do not depend on the neighbours."""
    lens, Hk, Hv, Dk, Dv = [100, 300, 90], 1, 2, 64, 64
    d = ck.inputs(3, lens, Hk, Hv, Dk, Dv, BF, True)
    cu = dc.cu_of(lens).cuda()
    a = run(dev(d), cu, True)
    for n in ("q", "k", "v", "g", "dout"):
        d[n][150] = float("nan")
    d["h0"][1] = d["dhT"][1] = float("inf")
    b = run(dev(d), cu, True)
    for n in ("out", "dq", "dk", "dv", "dg"):
        for s in (slice(0, 100), slice(400, 490)):
            assert torch.equal(a[n][s], b[n][s]), n
    for n in ("hT", "dh0"):
        assert torch.equal(a[n][0], b[n][0]) and torch.equal(a[n][2], b[n][2]), n


@pytest.mark.parametrize("cut", [1, 64, 100, 256])
def test_a_sequence_continued_in_another_pack(cut):
    lens, Hk, Hv, Dk, Dv = [400], 2, 2, 64, 32
    d = dev(ck.inputs(9, lens, Hk, Hv, Dk, Dv, F32, True))
    m = ssp()
    whole = run(d, dc.cu_of(lens).cuda(), True)
    part = lambda s: {n: d[n][s].contiguous() for n in ("q", "k", "v", "g", "dout")}  # noqa: E731
    x, y = part(slice(0, cut)), part(slice(cut, 400))
    cx, cy = dc.cu_of([cut]).cuda(), dc.cu_of([400 - cut]).cuda()
    o1, h1 = m.decay_attn_pack_fwd(x["q"], x["k"], x["v"], x["g"], cx, initial_state=d["h0"], final_state=True)
    o2, h2 = m.decay_attn_pack_fwd(y["q"], y["k"], y["v"], y["g"], cy, initial_state=h1, final_state=True)
    g2 = m.decay_attn_pack_bwd(y["q"], y["k"], y["v"], y["g"], cy, y["dout"], initial_state=h1, dfinal_state=d["dhT"],
                               dinitial_state=True)
    g1 = m.decay_attn_pack_bwd(x["q"], x["k"], x["v"], x["g"], cx, x["dout"], initial_state=d["h0"],
                               dfinal_state=g2["dinitial_state"], dinitial_state=True)
    tol = 2 * ck.tol32(400, Dk, Dv)  # both sides err
    dc.check(torch.cat([o1, o2]), whole["out"].cpu(), tol, "out")
    dc.check(h2, whole["hT"].cpu(), tol, "hT")
    dc.check(g1["dinitial_state"], whole["dh0"].cpu(), tol, "dh0")
    for n in ("dq", "dk", "dv"):
        dc.check(torch.cat([g1[n], g2[n]]), whole[n].cpu(), tol, n)


@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 1, 1, 8, 8), (5, 2, 4, 128, 128), (3, 1, 3, 72, 40), (2, 1, 1, 32, 264)])
def test_step_is_the_recurrence(B, Hk, Hv, Dk, Dv, dtype, per_token):
    lens = [1] * B
    d = ck.inputs(11, lens, Hk, Hv, Dk, Dv, dtype, True, per_token)
    out, hT = ck.attention(*(d[n].to(ck.F64) for n in ("q", "k", "v", "g")), lens, Dk ** -0.5, d["h0"].to(ck.F64))
    pool = torch.full((B + 3, Hv, Dk, Dv), float("nan"), device="cuda")
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    pool[slots.long().cuda()] = d["h0"].cuda()
    x = dev(d)
    got = ssp().decay_attn_pack_step(x["q"], x["k"], x["v"], x["g"], pool, slots=slots.cuda(), out=nan_like(x["v"]))
    tol = ck.tol32(1, Dk, Dv)
    dc.check(got, out, tol, "out")
    dc.check(pool[slots.long().cuda()], hT, tol, "state")
    rest = [i for i in range(B + 3) if i not in slots.tolist()]
    assert bool(pool[rest].isnan().all())


def test_step_slots_named_twice_and_outside_the_pool():
    Hk, Hv, Dk, Dv = 1, 2, 40, 72
    rows = [2, -1, 0, 2, 7, 2]
    d = ck.inputs(12, [1] * 6, Hk, Hv, Dk, Dv, F32, False)
    pool = torch.randn(3, Hv, Dk, Dv, generator=torch.Generator().manual_seed(2))
    order = [0, 3, 5]  # the rows of slot 2, a sequence of three
    ref, hT = ck.attention(*(d[n][order].to(ck.F64) for n in ("q", "k", "v", "g")), [3], 0.5, pool[2:3].to(ck.F64))
    one, h0 = ck.attention(*(d[n][2:3].to(ck.F64) for n in ("q", "k", "v", "g")), [1], 0.5, pool[0:1].to(ck.F64))
    x, p = dev(d), pool.cuda()
    got = ssp().decay_attn_pack_step(x["q"], x["k"], x["v"], x["g"], p, slots=torch.tensor(rows, dtype=torch.int32).cuda(),
                                     scale=0.5, out=nan_like(x["v"]))
    tol = ck.tol32(3, Dk, Dv)
    dc.check(got[order], ref, tol, "out")
    dc.check(got[2:3], one, tol, "out")
    dc.check(p[2:3], hT, tol, "state")
    dc.check(p[0:1], h0, tol, "state")
    assert torch.equal(p[1].cpu(), pool[1]) and bool(got[[1, 4]].isnan().all())


def test_steps_follow_a_prompt():
    """The states that a prompt leaves, and then tokens one by one, as the whole sequence."""
    lens, Hk, Hv, Dk, Dv = [90, 300], 2, 2, 64, 64
    d = dev(ck.inputs(13, lens, Hk, Hv, Dk, Dv, BF, False))
    m, n = ssp(), 5
    whole, hT = m.decay_attn_pack_fwd(d["q"], d["k"], d["v"], d["g"], dc.cu_of(lens).cuda(), final_state=True)
    ends = [90, 390]
    keep = torch.cat([torch.arange(0, 85), torch.arange(90, 385)])
    x = {k: d[k][keep.cuda()].contiguous() for k in ("q", "k", "v", "g")}
    _, state = m.decay_attn_pack_fwd(x["q"], x["k"], x["v"], x["g"], dc.cu_of([85, 295]).cuda(), final_state=True)
    tol = 2 * ck.tol32(300, Dk, Dv)
    for i in range(n):
        at = torch.tensor([e - n + i for e in ends], device="cuda")
        y = m.decay_attn_pack_step(*(d[k][at].contiguous() for k in ("q", "k", "v", "g")), state)
        dc.check(y, whole[at].cpu().to(ck.F64), tol + 2.0 ** -13 + 2.0 ** -8, "out")  # both are rounded to bf16
    dc.check(state, hT.cpu(), tol, "state")


def test_offsets_past_32_bits():
    """2.3e9 elements of v (4.6e9 bytes): the last three sequences as alone. 768
    workgroups or more walk sequences whole, so that both take the same steps."""
    m = ssp()
    L, n, Hv, Dk, Dv, few = 2000, 35, 256, 8, 128, 3
    T = L * n
    assert T * Hv * Dv > 1 << 31 and few * Hv >= 768
    gen = torch.Generator("cuda").manual_seed(6)
    o = dict(device="cuda", generator=gen)
    q, k = torch.randn(T, 1, Dk, **o).to(BF), torch.randn(T, 1, Dk, **o).to(BF)
    v, dout = (torch.randn(T, Hv, Dv, dtype=BF, **o) for _ in range(2))
    g = -torch.rand(T, Hv, **o) * 0.1
    h0, dhT = (torch.randn(n, Hv, Dk, Dv, **o) for _ in range(2))

    def run_(s, states):
        t = [x[s] for x in (q, k, v, g)]
        count = t[0].shape[0] // L
        cu = dc.cu_of([L] * count).cuda()
        out, hT = m.decay_attn_pack_fwd(*t, cu, initial_state=h0[states].clone(), final_state=True)
        G = m.decay_attn_pack_bwd(*t, cu, dout[s], initial_state=h0[states].clone(), dfinal_state=dhT[states].clone(),
                                  dinitial_state=True)
        return dict(G, out=out, hT=hT)

    whole = run_(slice(0, T), slice(0, n))
    alone = run_(slice(T - few * L, T), slice(n - few, n))
    for name, t in alone.items():
        assert torch.equal(whole[name][-t.shape[0]:], t), name


def test_step_on_a_pool_past_32_bits():
    m = ssp()
    Hv, D, slots = 32, 128, 8200
    assert slots * Hv * D * D > 1 << 32
    d = dev(ck.inputs(8, [3], Hv, Hv, D, D, BF, False, True))
    state = torch.empty(slots, Hv, D, D, device="cuda")
    at = torch.tensor([8199, 0, 8192], dtype=torch.int32, device="cuda")
    small = torch.randn(3, Hv, D, D, device="cuda", generator=torch.Generator("cuda").manual_seed(9))
    state[at.long()] = small
    a = m.decay_attn_pack_step(d["q"], d["k"], d["v"], d["g"], state, at)
    b = m.decay_attn_pack_step(d["q"], d["k"], d["v"], d["g"], small)
    assert torch.equal(a, b) and torch.equal(state[at.long()], small)


def test_many_sequences_without_tokens():
    """Nothing to walk, in more workgroups than the card has at a time: states and gradients go through."""
    m, n, Hk, Hv, D = ssp(), 300, 2, 4, 64
    q, v = (torch.empty(0, h, D, dtype=BF, device="cuda") for h in (Hk, Hv))
    g, cu = torch.empty(0, Hv, device="cuda"), torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    h = torch.randn(n, Hv, D, D, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    _, hT = m.decay_attn_pack_fwd(q, q, v, g, cu, initial_state=h, final_state=True)
    G = m.decay_attn_pack_bwd(q, q, v, g, cu, v, initial_state=h, dfinal_state=h, dinitial_state=True)
    assert torch.equal(hT, h) and torch.equal(G["dinitial_state"], h)


def test_heads_in_pairs_captured_and_replayed():
    m, n, Hk, Hv, D = ssp(), 80, 2, 4, 64
    lens = [1 + 7 * i % 90 for i in range(n)]
    assert 2 * n * Hv > 512
    d = dev(ck.inputs(12, lens, Hk, Hv, D, D, BF, False, True))
    cu = dc.cu_of(lens).cuda()
    args = (d["q"], d["k"], d["v"], d["g"], cu, d["dout"])
    want = m.decay_attn_pack_bwd(*args)
    ws = poison(m.decay_attn_pack_bwd_scratch_bytes(sum(lens), n, Hk, Hv, D, D))
    out = {k: nan_like(want[k]) for k in ("dq", "dk", "dv", "dg")}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.decay_attn_pack_bwd(*args, scratch=ws, out=out)
    for _ in range(3):
        ws.fill_(255)
        for t in out.values():
            t.fill_(float("nan"))
        graph.replay()
        eager = m.decay_attn_pack_bwd(*args)
        torch.cuda.synchronize()
        for k, t in out.items():
            assert torch.equal(t, want[k]) and torch.equal(eager[k], want[k]), k
