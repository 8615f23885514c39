"""GPU: whatever cu_seqlens holds, the delta rule's calls write inside their
buffers: every output, both scratches and what the forward keeps lie between
guards. (tests/test_delta_sizes_cpu.py goes through the same index arithmetic
on the host.)"""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc
from tests.test_delta_gpu import BF, F32, dev, ssp

pytestmark = pytest.mark.gpu

GUARD, FILL = 8192, 0x4B


class Guarded:
    """Buffers between guards of GUARD bytes in one allocation."""

    def __init__(self, sizes):
        self.at, end = {}, GUARD
        for name, n in sizes.items():
            self.at[name] = (end, n)
            end += -(-n // 16) * 16 + GUARD
        self.mem = torch.full((end,), FILL, dtype=torch.uint8, device="cuda")

    def bytes(self, name):
        a, n = self.at[name]
        return self.mem[a:a + n]

    def view(self, name, like):
        return self.bytes(name).view(like.dtype).view(like.shape)

    def broken(self):
        """Names of buffers that something was written before or behind."""
        torch.cuda.synchronize()
        bad, free = [], torch.ones(self.mem.numel(), dtype=torch.bool, device="cuda")
        for a, n in self.at.values():
            free[a:a + n] = False
        hit = ((self.mem != FILL) & free).nonzero()
        if hit.numel():
            bad = [(name, int(hit[0])) for name, (a, n) in self.at.items()
                   if bool(((hit >= a - GUARD) & (hit < a + n + GUARD)).any())]
        return bad


def calls(T, n, Hk, Hv, Dk, Dv, dtype, seed):
    """run(cu): forward and backward on guarded buffers; what was overrun."""
    m = ssp()
    d = dev(dc.rule_inputs(seed, [T], Hk, Hv, Dk, Dv, dtype, False))
    state = torch.empty(n, Hv, Dk, Dv, device="cuda")
    h0 = torch.randn(n, Hv, Dk, Dv, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    like = {"out": d["v"], "dq": d["q"], "dk": d["k"], "dv": d["v"], "dg": d["g"], "dbeta": d["beta"], "hT": state,
            "dh0": state}
    sizes = {name: t.numel() * t.element_size() for name, t in like.items()}
    sizes["saved"] = m.gated_delta_pack_saved_bytes(T, n, Hk, Hv, Dk, Dv)
    sizes["fwd"] = m.gated_delta_pack_fwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, dtype)
    sizes["bwd"] = m.gated_delta_pack_bwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, dtype)
    room = Guarded(sizes)
    t = {name: room.view(name, x) for name, x in like.items()}

    def run(cu):
        for name in ("saved", "fwd", "bwd"):
            room.bytes(name).fill_(255)
        m.gated_delta_pack_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu, initial_state=h0, final_state=t["hT"],
                               saved=room.bytes("saved"), scratch=room.bytes("fwd"), out=t["out"])
        m.gated_delta_pack_bwd(d["q"], d["k"], d["g"], d["beta"], cu, d["dout"], room.bytes("saved"), dfinal_state=h0,
                               dinitial_state=t["dh0"], scratch=room.bytes("bwd"),
                               out={name: t[name] for name in ("dq", "dk", "dv", "dg", "dbeta")})
        return room.broken()

    return run


FORMS = [
    # T, nseq, Hk, Hv, Dk, Dv
    (200, 3, 1, 2, 64, 40),      # a few sequences
    (131, 1, 1, 1, 8, 8),        # one
    (700, 9, 2, 24, 128, 72),    # many chains, by length, eight waves
    (300, 140, 1, 2, 72, 24),    # many chains, four waves
    (4200, 2, 1, 1, 16, 24),     # split
    (2113, 1, 1, 2, 128, 136),   # split, parts that do not divide it
]


def boundaries(T, n, seed):
    """Ordered ones (which may end early or late), then any."""
    gen = torch.Generator().manual_seed(seed)
    yield torch.linspace(0, T, n + 1).to(torch.int32)
    yield torch.zeros(n + 1, dtype=torch.int32)
    for k in range(3):
        cu = torch.randint(0, T + 1, (n + 1,), generator=gen).sort().values
        cu[0] = 0
        yield cu.to(torch.int32)
    yield torch.randint(0, T + 1, (n + 1,), generator=gen).sort(descending=True).values.to(torch.int32)
    for k in range(6):
        yield torch.randint(-T, 3 * T, (n + 1,), generator=gen).to(torch.int32)
    ends = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, T], dtype=torch.int32)
    for k in range(2):
        yield ends[torch.randint(0, 4, (n + 1,), generator=gen)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_writes_stay_inside(form, dtype):
    T, n = FORMS[form][:2]
    run = calls(*FORMS[form], dtype, 900 + form)
    for i, cu in enumerate(boundaries(T, n, 910 + form)):
        bad = run(cu.cuda())
        assert not bad, (i, cu.tolist()[:8], bad)
