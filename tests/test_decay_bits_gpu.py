"""GPU: a bf16 result of the linear attention is the nearest bf16 to a value that
errs as 32-bit sums do, with and without dg: nothing on the way is held in fewer
bits. Short sequences, where 32-bit sums err least and a part left out shows
most: 2^-14 of a term moves 5 results in 1000 to their neighbours. The count
of results that may lie beside the nearest value is that of the delta rule's test
(`off`), whose errors are of the same kind: a state's product, decayed products
and 32-bit roundings of each. (What tests/decay_checks.py allows for two cut
parts, `tol_parts`, is more than any result needs.)"""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck
from tests import delta_checks as dc
from tests.test_decay_gpu import BF, dev, run
from tests.test_delta_bits_gpu import off

pytestmark = pytest.mark.gpu

CASES = [
    # lens, Hk, Hv, Dk, Dv
    ([1] * 150 + [2] * 20, 1, 2, 64, 40),     # both value heads of a key head in a workgroup
    ([1, 2, 3] * 30, 2, 2, 128, 128),
    ([1, 3] * 70, 1, 1, 72, 136),
    ([2, 1, 3] * 12, 1, 3, 40, 64),
    ([3, 2] * 40, 4, 8, 128, 128),            # the same, of the largest heads
]


@pytest.mark.parametrize("dg", [True, False])
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_bf16_results_are_rounded_once(case, carry, dg):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    d = ck.inputs(800 + case, lens, Hk, Hv, Dk, Dv, BF, carry)
    ref = ck.reference(d, lens, Dk ** -0.5)
    got = run(dev(d), dc.cu_of(lens).cuda(), carry, dg=dg)
    heads = {"dq": Hv // Hk, "dk": Hv // Hk}  # whose gradients are added
    seen = {n: off(got[n], ref[n], ck.tol32(max(lens), Dk, Dv) * heads.get(n, 1)) for n in ("out", "dq", "dk", "dv")}
    assert all(outside == 0 and moved <= most for outside, moved, most in seen.values()), seen


@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [
    ([70, 300, 1, 0, 129], 1, 3, 64, 40),
    ([64, 17] * 40, 2, 4, 128, 128),          # more workgroups than the card has at a time
    ([200, 90], 2, 2, 72, 200),
])
def test_results_within_their_own_size(lens, Hk, Hv, Dk, Dv):
    """Rows of very different sizes: v and dout of a sequence are 2^-30 to 2^20 of another's, and
    so are its results. Each sequence's error is held to its own largest value."""
    d = ck.inputs(31, lens, Hk, Hv, Dk, Dv, BF, False)
    t = 0
    for i, n in enumerate(lens):
        d["v"][t:t + n] *= 2.0 ** (10 * (i % 6) - 30)
        d["dout"][t:t + n] *= 2.0 ** (-7 * (i % 4))
        t += n
    ref = ck.reference(d, lens, Dk ** -0.5)
    for dg in (True, False):
        got = run(dev(d), dc.cu_of(lens).cuda(), False, dg=dg)
        t = 0
        for n in lens:
            for name in ("out", "dq", "dk", "dv"):
                r = Hv // Hk if name in ("dq", "dk") else 1
                dc.check(got[name][t:t + n], ref[name][t:t + n], r * ck.tol32(n, Dk, Dv), f"{name} of {n} tokens")
            t += n


@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [
    ([70, 300, 1, 0, 129], 1, 3, 64, 40),
    ([64, 17] * 40, 2, 4, 128, 128),
    ([200, 90], 2, 2, 72, 200),
    ([33], 1, 2, 16, 64),
])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_gradients_do_not_depend_on_whether_dg_is_asked_for(lens, Hk, Hv, Dk, Dv, dtype):
    d = dev(ck.inputs(33, lens, Hk, Hv, Dk, Dv, dtype, True))
    a, b = (run(d, dc.cu_of(lens).cuda(), True, dg=dg) for dg in (True, False))
    for n in ("dq", "dk", "dv", "dh0"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [
    ([1, 64, 600], 1, 2, 128, 128),
    ([257, 0, 300], 2, 2, 40, 72),
    ([520], 1, 1, 64, 264),
    ([300, 7] * 25, 4, 8, 128, 64),           # both value heads of a key head in a workgroup
])
def test_what_dg_starts_from(lens, Hk, Hv, Dk, Dv, dtype):
    """Queries and keys of zero and no decay: every token's dg is (dfinal_state . initial_state), a sum of
    Dk Dv products that nearly cancel. It is formed in 64 bits and rounded once, whatever it starts from in the sequence."""
    d = ck.inputs(50, lens, Hk, Hv, Dk, Dv, dtype, True)
    d["q"].zero_(), d["k"].zero_(), d["g"].zero_()
    want = (d["h0"].double() * d["dhT"].double()).sum((-1, -2))
    size = (d["h0"].double() * d["dhT"].double()).abs().sum((-1, -2))
    got = run(dev(d), dc.cu_of(lens).cuda(), True)["dg"].cpu().double()
    one = run(dev(dict(d, g=torch.zeros(Hv))), dc.cu_of(lens).cuda(), True)["dg"].cpu().double()
    t = 0
    for s, n in enumerate(lens):
        off_by = (got[t:t + n] - want[s]).abs()
        assert bool((off_by <= 2.0 ** -24 * want[s].abs() + 2.0 ** -45 * size[s]).all()), (s, float(off_by.max()), want[s])
        t += n
    n = torch.tensor(lens, dtype=torch.float64)[:, None]
    room = 2.0 ** -24 * (n * want).sum(0).abs() + 2.0 ** -40 * (n * size).sum(0)
    assert bool(((one - (n * want).sum(0)).abs() <= room).all())
