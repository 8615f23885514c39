"""GPU: how far a NaN or an infinity of one token reaches in the delta rule's
backward: earlier tokens by the formula, later ones only to its chunk's end."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc
from tests.test_delta_gpu import BF, F32, dev, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("name", ["dout", "q"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens, Hv", [([40, 230], 2), ([2200], 1)])  # whole, and split in parts
def test_bad_values_in_the_backward(lens, Hv, bad, name, dtype):
    d = dc.rule_inputs(740, lens, 1, Hv, 64, 40, dtype, True)
    cu = dc.cu_of(lens).cuda()
    clean = run(dev(d), cu, True)
    start = sum(lens) - lens[-1]
    at, end = start + 100, start + 128  # a token of the second chunk, and that chunk's end
    d[name][at] = bad
    got = run(dev(d), cu, True)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(got[n][end:], clean[n][end:]), n
        assert torch.equal(got[n][:start], clean[n][:start]), n
    keep = torch.arange(sum(lens)) != at
    assert torch.equal(got["out"].cpu()[keep], clean["out"].cpu()[keep])  # of a query only its own
    assert torch.equal(got["hT"], clean["hT"])
