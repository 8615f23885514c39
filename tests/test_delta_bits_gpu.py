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


def off(got, ref, rel):
    """(entries outside the bf16 values nearest to ref - err and ref + err, err being
    rel of the largest; those that are not the one nearest to ref; how many of these
    there may be). rel is four times an error's rms, for an entry of the size that the
    sums have on the way: on average over the entries, the rms of all. A value
    anywhere in the interval of width u that is rounded to one bf16 leaves it with an
    error e with probability |e| / u, so rms / u bounds what is expected of each
    entry; five times the count's own deviation is allowed on top."""
    g, r = got.cpu(), ref.detach()
    err = rel * float(r.abs().max())
    outside = int((~((g >= (r - err).to(BF)) & (g <= (r + err).to(BF)))).sum())
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp_min(1e-30))) - 7)
    expected = float((rel / 4 * float(r.square().mean().sqrt()) / step).clamp_max(1.0).sum())
    return outside, int((g != r.to(BF)).sum()), int(expected + 5 * expected ** 0.5 + 1)


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_bf16_results_are_rounded_once(case, carry):
    lens, Hk, Hv, Dk, Dv = CASES[case]
    d = dc.rule_inputs(700 + case, lens, Hk, Hv, Dk, Dv, BF, carry)
    ref = dc.rule_reference(d, lens, Dk ** -0.5)
    got = run(dev(d), dc.cu_of(lens).cuda(), carry)
    heads = {"dq": Hv // Hk, "dk": Hv // Hk}  # whose gradients are added
    seen = {n: off(got[n], ref[n], dc.tol32(max(lens), Dk) * heads.get(n, 1)) for n in ("out", "dq", "dk", "dv")}
    assert all(outside == 0 and moved <= most for outside, moved, most in seen.values()), seen
