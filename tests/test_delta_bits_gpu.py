"""GPU: a bf16 result of the gated delta rule is the nearest bf16 to a value that
errs as 32-bit sums do, whatever its tensor: nothing on the way is held in fewer
bits. Short sequences, where 32-bit sums err least and a part left out shows
most: 2^-14 of a term moves one result in a hundred to its neighbour."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc
from tests.test_delta_gpu import BF, dev, run

pytestmark = pytest.mark.gpu

CASES = [
    # lens, Hk, Hv, Dk, Dv
    ([1] * 150 + [2] * 20, 1, 2, 64, 40),
    ([1, 2, 3] * 30, 2, 2, 128, 128),
    ([1, 3] * 70, 1, 1, 72, 136),
]


def off(got, ref, err):
    """Entries outside the bf16 values nearest to ref - err and ref + err."""
    g, r = got.cpu(), ref.detach()
    return int((~((g >= (r - err).to(BF)) & (g <= (r + err).to(BF)))).sum())


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_bf16_results_are_rounded_once(case, carry):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    d = dc.rule_inputs(700 + case, lens, Hk, Hv, Dk, Dv, BF, carry)
    ref = dc.rule_reference(d, lens, Dk ** -0.5)
    got = run(dev(d), dc.cu_of(lens).cuda(), carry)
    heads = {"dq": Hv // Hk, "dk": Hv // Hk}  # whose gradients are added
    bad = {n: off(got[n], ref[n], dc.tol32(max(lens), Dk) * heads.get(n, 1) * float(ref[n].abs().max()))
           for n in ("out", "dq", "dk", "dv")}
    assert not any(bad.values()), bad
