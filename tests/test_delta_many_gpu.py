"""GPU: the gated delta rule where its launches take other forms than for a few
short sequences: many chains at once (128 columns a workgroup, the longest
sequences first), more sequences than are ordered, and packs whose elements
need more than 32 bits to count."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc
from tests.test_delta_gpu import BF, F32, compare, dev, nan_like, run, ssp

pytestmark = pytest.mark.gpu


def reference(d, lens, scale):
    """dc.rule_reference with the sequences side by side, padded by tokens that
    leave the state as it is (a = 1, beta = 0); 64 bits, products and sums only."""
    n, L, T = len(lens), max(lens), sum(lens)
    start = torch.tensor([0] + lens).cumsum(0)[:-1]
    at = start[:, None] + torch.arange(L)
    on = torch.arange(L) < torch.tensor(lens)[:, None]
    at = torch.where(on, at, torch.zeros_like(at)).cuda()
    on = on.cuda()
    x = {m: d[m][:T].cuda().to(dc.F64).requires_grad_() for m in ("q", "k", "v", "g", "beta")}
    h0 = None if d["h0"] is None else d["h0"].cuda().to(dc.F64).requires_grad_()
    Hv, Dk, Dv = d["v"].shape[1], d["q"].shape[2], d["v"].shape[2]
    r = Hv // d["q"].shape[1]
    S = torch.zeros(n, Hv, Dk, Dv, dtype=dc.F64, device="cuda") if h0 is None else h0
    outs = []
    for t in range(L):
        i, m = at[:, t], on[:, t, None].to(dc.F64)
        q, k = x["q"][i].repeat_interleave(r, 1), x["k"][i].repeat_interleave(r, 1)
        S = S * (x["g"][i] * m).exp()[..., None, None]
        e = x["v"][i] - (S * k[..., None]).sum(2)
        S = S + k[..., None] * ((x["beta"][i] * m)[..., None] * e)[:, :, None]
        outs.append(scale * (S * q[..., None]).sum(2))
    out = torch.stack(outs, 1)[on]
    loss = (out * d["dout"][:T].cuda().to(dc.F64)).sum()
    if d["dhT"] is not None:
        loss = loss + (S * d["dhT"].cuda().to(dc.F64)).sum()
    leaves = list(x.values()) + ([] if h0 is None else [h0])
    res = {"out": out.detach(), "hT": S.detach()}
    res.update(zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), torch.autograd.grad(loss, leaves)))
    return {m: t.cpu() for m, t in res.items()}


def lengths(seed, n, top):
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, top + 1, (n,), generator=gen)
    lens[torch.randperm(n, generator=gen)[:n // 8]] = 0
    return lens.tolist()


CASES = [
    # lens, Hk, Hv, Dk, Dv
    (lengths(0, 130, 80), 1, 2, 72, 72),        # 128 columns in bf16, keys over 64
    (lengths(1, 70, 150), 2, 4, 40, 128),       # 128 columns, keys to 64
    (lengths(2, 45, 140), 1, 3, 128, 136),      # two workgroups a head, the second nearly empty
    (lengths(3, 300, 70), 1, 1, 64, 24),        # 64 columns, ordered
    ([300, 0, 2, 420], 2, 64, 24, 72),          # a few long ones over many heads
    (lengths(4, 4500, 3), 1, 1, 16, 72),        # more than are ordered
]


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_many_chains(case, dtype, carry):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    d = dc.rule_inputs(300 + case, lens, Hk, Hv, Dk, Dv, dtype, carry)
    ref = reference(d, lens, Dk ** -0.5)
    compare(run(dev(d), dc.cu_of(lens).cuda(), carry), ref, d, lens, carry, Dk)


def test_the_two_references_agree():
    lens = [3, 0, 70]
    d = dc.rule_inputs(5, lens, 1, 2, 16, 8, F32, True)
    a, b = reference(d, lens, 0.25), dc.rule_reference(d, lens, 0.25)
    for n in b:
        # the same sums in 64 bits, in other orders
        dc.check(a[n], b[n], dc.tol32(70, 16) * 2.0 ** -29, n)


def test_many_chains_captured():
    """One graph, replayed over other lengths in the same buffers: the order of
    the sequences is made anew in each replay."""
    m = ssp()
    Hk, Hv, Dk, Dv, T = 1, 2, 72, 72, 130 * 40
    packs = []
    for seed in (10, 11, 12):
        lens = lengths(seed, 130, 70)
        while sum(lens) > T:
            lens[lens.index(max(lens))] = 0
        packs.append(dc.cu_of(lens).cuda())
    d = dev(dc.rule_inputs(9, [T], Hk, Hv, Dk, Dv, BF, False))
    d["h0"] = 0.3 * torch.randn(130, Hv, Dk, Dv, generator=torch.Generator().manual_seed(13)).cuda()
    d["dhT"] = d["h0"].flip(0).contiguous()
    cu = packs[0].clone()
    eager = []
    for p in packs:
        eager.append(run(d, p, True))
    state = nan_like(d["h0"])
    out = nan_like(d["v"])
    saved = torch.empty(m.gated_delta_pack_saved_bytes(T, 130, Hk, Hv, Dk, Dv), dtype=torch.uint8, device="cuda")
    ws = torch.empty(m.gated_delta_pack_fwd_scratch_bytes(T, 130, Hk, Hv, Dk, Dv, BF), dtype=torch.uint8, device="cuda")
    wb = torch.empty(m.gated_delta_pack_bwd_scratch_bytes(T, 130, Hk, Hv, Dk, Dv, BF), dtype=torch.uint8, device="cuda")
    grads = {"dq": nan_like(d["q"]), "dk": nan_like(d["k"]), "dv": nan_like(d["v"]), "dg": nan_like(d["g"]),
             "dbeta": nan_like(d["beta"])}
    dh0 = nan_like(d["h0"])

    def once():
        m.gated_delta_pack_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, initial_state=d["h0"],
                               final_state=state, saved=saved, out=out, scratch=ws)
        m.gated_delta_pack_bwd(d["q"], d["k"], d["g"], d["beta"], cu, d["dout"], saved, dfinal_state=d["dhT"],
                               dinitial_state=dh0, scratch=wb, out=grads)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    got = {"out": out, "hT": state, "dh0": dh0, **grads}
    for i in (1, 2, 0, 1):
        cu.copy_(packs[i])
        for t in got.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        n = int(packs[i][-1])
        for name, t in got.items():
            rows = 130 if name in ("hT", "dh0") else n
            assert torch.equal(t[:rows], eager[i][name][:rows]), name
            assert bool(t[rows:].isnan().all()), name


def test_more_elements_than_32_bits_count():
    """Equal sequences, equal to the bit wherever they lie: values, outputs and
    gradients of 2.4e9 elements, 10 GB of kept states."""
    m = ssp()
    n, L, Hk, Hv, Dk, Dv = 280, 1037, 1, 64, 8, 128
    one = dc.rule_inputs(21, [L], Hk, Hv, Dk, Dv, BF, False)
    small = run(dev(one), dc.cu_of([L]).cuda(), False)
    d = {k: None if t is None else t.cuda().repeat(n, *[1] * (t.dim() - 1)) for k, t in one.items()}
    assert d["v"].numel() > 1 << 31
    cu = dc.cu_of([L] * n).cuda()
    big = run(d, cu, False)
    del d
    for name in ("out", "dq", "dk", "dv", "dg", "dbeta"):
        rows = big[name].view(n, L, *big[name].shape[1:])
        for s in range(n):
            assert torch.equal(rows[s], rows[0]), (name, s)
        # few chains are split otherwise, in columns that do not meet
        assert torch.equal(rows[0], small[name]), name
    assert m.gated_delta_pack_saved_bytes(n * L, n, Hk, Hv, Dk, Dv) > 1 << 32
