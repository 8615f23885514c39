"""CPU tests of the delta-rule block helper: what it refuses before any call."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_varlen_amd as m


def test_gradients_of_states_that_were_not_given_are_refused():
    """Neither dropped nor used in part: the convs of a forward without states take none."""
    fwd = {"cu_seqlens": None, "carry": False, "initial_states": {}}
    t = torch.zeros(1)
    for d in ({"delta": t}, {"conv": (t, t, t)}, {"delta": None, "conv": (t, t, t)}):
        with pytest.raises(ValueError, match="final states"):
            m.delta_backward((t, t, t), (t, t, t), None, t, t, fwd, t, dfinal_states=d)
