"""GPU: how near to the 64-bit cosines and sines the head norms' rotation turns."""
from __future__ import annotations

import pytest
import torch

from tests import delta_checks as dc

pytestmark = pytest.mark.gpu

def ssp():
    import selective_state_space_varlen_amd as m
    return m


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("first", [True, False])
def test_turns_to_the_last_bits(first, inter):
    """One component of each pair is 1 and the others 0, so that y holds the
    cosines and sines themselves: each within 8 * 2^-24 of its value (2 ulp, or
    4 * 2^-24, of the library's cosine and sine, 2 of the norm's root, and the
    correction's and the result's roundings), the small ones too. Angles of up to
    4096 in 64 bits err by 4096 * 2^-51, far less."""
    T, rot = 60, 64
    m = ssp()
    inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
    gen = torch.Generator().manual_seed(70)
    pos = torch.randint(0, 4096, (T,), generator=gen).to(torch.int32)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    x = torch.zeros(T, rot // 2, rot)
    at = a if first else b
    for i in range(rot // 2):  # head i shows pair i
        x[:, i, range(rot)[at][i]] = 1.0
    y, _ = m.qk_norm_pack_fwd(x.cuda(), x[:, :0].cuda(), pos=pos.cuda(), inv_freq=inv.cuda(), eps=0.0, interleaved=inter)
    # back: turned the other way
    g = m.qk_norm_pack_bwd(x.cuda(), x[:, :0].cuda(), x.cuda(), x[:, :0].cuda(), wq=torch.ones(rot).cuda(),
                           pos=pos.cuda(), inv_freq=inv.cuda(), eps=0.0, interleaved=inter)
    torch.cuda.synchronize()
    ang = pos.to(dc.F64)[:, None] * inv.to(dc.F64)
    cos, sin = torch.cos(ang), torch.sin(ang)
    head = torch.arange(rot // 2)
    ya, yb = y.cpu().to(dc.F64)[..., a], y.cpu().to(dc.F64)[..., b]
    got = {"a": ya[:, head, head], "b": yb[:, head, head]}
    want = {"a": cos, "b": sin} if first else {"a": -sin, "b": cos}
    for n in got:
        off = (got[n] - want[n]).abs() / want[n].abs().clamp_min(1e-30)
        assert float(off.max()) <= 8 * 2.0 ** -24, (n, float(off.max()) * 2 ** 24)
    # dw of the shown component: the sum of the cosines over the tokens
    shown = g["dwq"].cpu().to(dc.F64)[at]
    assert float((shown - cos.sum(0)).abs().max()) <= T * 8 * 2.0 ** -24
