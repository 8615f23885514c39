"""GPU: many chains over more than three chunks each, with keys over 64: eight
waves a workgroup, whose two sets of operands in LDS take turns from chunk to
chunk."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc
from tests.test_delta_gpu import BF, F32, compare, dev, run
from tests.test_delta_many_gpu import reference

pytestmark = pytest.mark.gpu

CASES = [
    # lens, Hk, Hv, Dk, Dv: more than 256 chains of 64 columns
    ([330, 0, 261, 70], 4, 44, 128, 72),
    ([449], 2, 130, 72, 128),
    ([64 * 5, 64 * 6, 64 * 4 + 1], 24, 24, 120, 200),
]


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_long_chains(case, dtype, carry):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    assert len(lens) * Hv * -(-Dv // 64) > 256
    d = dc.rule_inputs(800 + case, lens, Hk, Hv, Dk, Dv, dtype, carry)
    # slow decays, so that the first chunks still count in the last
    d["g"] *= 0.05
    ref = reference(d, lens, Dk ** -0.5)
    torch.cuda.empty_cache()
    compare(run(dev(d), dc.cu_of(lens).cuda(), carry), ref, d, lens, carry, Dk)
