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


def test_the_tensors_device_is_current_during_a_call(monkeypatch):
    """The rule and the norms see to it themselves; the convs and the positions take the current device."""
    t, seen = torch.zeros(4, 8), []

    class Record:
        def __init__(self, x):
            seen.append(x)

        def __enter__(self):
            seen.append("in")

        def __exit__(self, *e):
            seen.append("out")

    monkeypatch.setattr(torch.cuda, "device_of", Record)
    with pytest.raises(ValueError, match="device tensor"):
        m.delta_forward((t, t, t), (t, t, t), None, t, t, torch.zeros(2, dtype=torch.int32), 1, 1)
    assert seen[0] is t and seen[1:] == ["in", "out"]
    seen.clear()
    with pytest.raises(KeyError):  # an empty forward's result, found out inside
        m.delta_backward(x=(t, t, t), w=(t, t, t), b=None, g=t, beta=t, dout=t, fwd={})
    assert seen[0] is t and seen[1:] == ["in", "out"]


@pytest.mark.gpu
@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_on_a_device_that_is_not_current():
    from tests.test_delta_block_gpu import make, tree
    lens, Hk, Hv, Dk, Dv, W = [70, 33], 1, 2, 32, 24, 4
    d = make(lens, Hk, Hv, Dk, Dv, W, False)
    cu, got = torch.tensor([0, 70, 103], dtype=torch.int32), []
    for dev in ("cuda:0", "cuda:1"):
        x = tree(d, lambda t: t.to(dev))
        F = m.delta_forward(x["x"], x["w"], x["b"], x["g"], x["beta"], cu.to(dev), Hk, Hv)
        G = m.delta_backward(x["x"], x["w"], x["b"], x["g"], x["beta"], F, x["dout"])
        torch.cuda.synchronize(dev)
        got.append([F["out"].cpu(), *(t.cpu() for t in G["dx"] + G["dw"])])
    assert all(torch.equal(a, b) for a, b in zip(*got))
