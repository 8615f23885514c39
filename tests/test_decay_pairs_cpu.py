"""CPU: the closed form by pairs of tokens agrees with the recurrence, both in 64 bits."""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck
from tests import decay_pairs as pairs


@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [([0, 5, 70, 1, 0], 2, 4, 8, 16), ([130], 1, 9, 16, 8), ([3, 33], 3, 3, 8, 8)])
def test_closed_form_is_the_recurrence(lens, Hk, Hv, Dk, Dv, per_token, carry):
    d = ck.inputs(40, lens, Hk, Hv, Dk, Dv, torch.float32, carry, per_token)
    a, b = ck.reference(d, lens, 0.3), pairs.reference(d, lens, 0.3)
    for n, t in a.items():
        assert float((t - b[n]).abs().max()) <= 1e-12 * (1.0 + float(t.abs().max())), n
    assert pairs.meets_of_heads(d, b).shape == (Hv,)


@pytest.mark.parametrize("lens,Hk,Hv,Dk,Dv", [([200, 129], 1, 3, 40, 136), ([3, 300], 2, 2, 128, 64), ([257, 256, 255, 513, 1], 1, 2, 16, 24),
                                              ([700], 1, 1, 64, 264), ([1, 520], 2, 6, 24, 200)])
def test_a_wrong_dg_is_seen_in_each_head(lens, Hk, Hv, Dk, Dv):
    """Zeros, a tenth too much, or a piece of 64 tokens without its part, of one head alone, are over what
    the check by token allows; of a sum over the tokens, they are over what test_sum_of_dg allows."""
    d = ck.inputs(60, lens, Hk, Hv, Dk, Dv, torch.float32, True, False)
    d["g"] = d["g"].expand(sum(lens), Hv).contiguous()
    ref = pairs.reference(d, lens, Dk ** -0.5)
    meets, rel = pairs.meets_of_heads(d, ref), ck.tol32(max(lens), Dk, Dv) * ck.rms_sum(max(lens))
    pairs.check_dg(ref["dg"].float(), ref["dg"], meets, rel)
    for h in range(Hv):
        for rows, by in ((slice(None), 0.0), (slice(None), 1.1), (slice(128, 192), 0.0)):
            bad = ref["dg"].clone()
            bad[rows, h] *= by
            with pytest.raises(AssertionError, match=f"head {h}"):
                pairs.check_dg(bad.float(), ref["dg"], meets, rel)
            room = (ref["dg"].abs().sum(0) + bad.sum(0).abs()) * (2.0 ** -24 + 2.0 ** -40)
            assert float((bad - ref["dg"]).sum(0)[h].abs()) > float(room[h])
