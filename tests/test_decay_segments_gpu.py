"""GPU: linear attention over long and over many sequences, which are walked in
segments, against 64-bit values: every length of a segment, states between them
that are added up by the walks and by a join over more than one batch of eight,
pieces of dg's anchors (256 tokens) that straddle segment ends, and more
sequences than a wave has lanes."""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck
from tests import decay_pairs as pairs
from tests import delta_checks as dc
from tests.test_decay_cpu import segment
from tests.test_decay_gpu import BF, F32, dev, run

pytestmark = pytest.mark.gpu

MIXED = [0, 1, 5, 130, 64, 0, 63, 3, 17, 65, 2, 0, 300, 128, 9]

CASES = [
    # lens, Hk, Hv, Dk, Dv, tokens of a segment, states between segments (T / segment)
    ([1300], 1, 1, 16, 24, 128, 10),
    ([2500, 3, 700], 1, 2, 40, 64, 128, 25),
    ([1500, 900, 1600], 14, 56, 8, 8, 256, 15),
    ([1500, 900, 1600], 28, 56, 8, 16, 256, 15),        # pairs of value heads
    ([1500, 901, 1599], 20, 80, 8, 8, 384, 10),
    ([1500, 901, 1599], 40, 80, 16, 8, 384, 10),
    ([1500, 901, 1599], 32, 128, 8, 8, 640, 6),
    ([1500, 901, 1599], 64, 128, 8, 8, 640, 6),
    ([1400, 1600], 41, 164, 8, 8, 640, 4),              # few states: added up by the walks
    ([2600], 40, 160, 8, 8, 512, 5),
    ([2600], 160, 160, 8, 8, 512, 5),
    ([2500, 2300, 2100], 64, 256, 8, 8, 2048, 3),
    ([2100, 2060, 2048, 2049, 2100, 2300], 32, 128, 8, 8, 2048, 6),
    (MIXED * 5, 1, 2, 72, 40, 128, 30),
    (MIXED * 5, 2, 4, 64, 64, 128, 30),                 # pairs of value heads
    (MIXED * 5 + [2300], 3, 12, 16, 24, 2048, 3),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_segments_match_definition(case, per_token, dtype):
    lens, Hk, Hv, Dk, Dv, seg, states = CASES[case]
    T, n, L = sum(lens), len(lens), max(lens)
    assert segment(T, n, Hv) == seg and T // seg == states and Dv <= 128
    d = ck.inputs(300 + case, lens, Hk, Hv, Dk, Dv, dtype, True, per_token)
    ref = pairs.reference(d, lens, Dk ** -0.5, "cuda")
    got = run(dev(d), dc.cu_of(lens).cuda(), True)
    tol, r = ck.tol32(L, Dk, Dv), Hv // Hk
    for name in ("out", "dv", "hT", "dh0"):
        dc.check(got[name], ref[name], tol, name)
    for name in ("dq", "dk"):
        dc.check(got[name], ref[name], tol * r, name)
    if not per_token:  # the sum over the tokens is the sum of what they have: test_sum_of_dg
        d = dict(d, g=d["g"].expand(T, Hv).contiguous())
        ref = pairs.reference(d, lens, Dk ** -0.5, "cuda")
        got = run(dev(d), dc.cu_of(lens).cuda(), True)
    pairs.check_dg(got["dg"], ref["dg"], pairs.meets_of_heads(d, ref), tol * ck.rms_sum(L))


def sum_of_dg(d, lens):
    """One decay for a head, and the same decays given by token: the same walks, and the
    first's dg is the 64-bit sum of the second's, of which each was rounded to 32 bits
    (2^-24 of it) before it stood here, as the sum was: each head by itself."""
    T, Hv = d["v"].shape[:2]
    cu = dc.cu_of(lens).cuda()
    head = run(dev(d), cu, d["h0"] is not None)
    token = run(dev(dict(d, g=d["g"].expand(T, Hv).contiguous())), cu, d["h0"] is not None)
    for name in ("out", "dq", "dk", "dv"):
        assert torch.equal(head[name], token[name]), name
    each, got = token["dg"].cpu().double(), head["dg"].cpu().double()
    room = (each.abs().sum(0) + got.abs()) * (2.0 ** -24 + 2.0 ** -40)  # 2^-40: of the sums in 64 bits
    assert bool(((each.sum(0) - got).abs() <= room).all()), (each.sum(0), got, room)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_sum_of_dg(case, dtype):
    lens, Hk, Hv, Dk, Dv, _, _ = CASES[case]
    sum_of_dg(ck.inputs(300 + case, lens, Hk, Hv, Dk, Dv, dtype, True, False), lens)


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [
    ([1], 1, 1, 8, 8), ([2, 1], 1, 2, 64, 64), ([63, 64, 65], 2, 2, 64, 32), ([0, 5, 0, 0, 70, 1, 0], 2, 4, 72, 40),
    ([200, 129], 1, 3, 40, 136), ([3, 300], 2, 2, 128, 64), ([257, 256, 255, 513, 1], 1, 2, 16, 24),
    ([700], 1, 1, 64, 264), ([1, 520], 2, 6, 24, 200)])
def test_one_decay_for_a_head(lens, Hk, Hv, Dk, Dv, dtype, carry):
    d = ck.inputs(60, lens, Hk, Hv, Dk, Dv, dtype, carry, False)
    sum_of_dg(d, lens)
    T, L = sum(lens), max(lens)
    d = dict(d, g=d["g"].expand(T, Hv).contiguous())
    ref = pairs.reference(d, lens, Dk ** -0.5, "cuda")
    got = run(dev(d), dc.cu_of(lens).cuda(), carry)
    pairs.check_dg(got["dg"], ref["dg"], pairs.meets_of_heads(d, ref), ck.tol32(L, Dk, Dv) * ck.rms_sum(L))
