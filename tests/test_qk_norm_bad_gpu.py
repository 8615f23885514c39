"""GPU: what an infinite component of a head reaches through the head norms."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def ssp():
    import selective_state_space_varlen_amd as m
    return m


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D, rot, inter", [(40, 2, True), (24, 10, True), (72, 14, True), (40, 16, False)])
def test_infinite_components_that_are_not_turned(D, rot, inter, dtype):
    """By the formula an infinity makes its row's factor zero: the component
    itself is NaN, the others zero. A gradient's reaches the weight of its own
    component alone."""
    T, H, bad = 5, 3, rot + 1
    gen = torch.Generator().manual_seed(71)
    x, dy = (torch.randn(T, H, D, generator=gen).to(dtype) for _ in range(2))
    pos = torch.arange(7, 7 + T, dtype=torch.int32).cuda()
    inv, w = (10.0 ** -torch.linspace(0, 3, rot // 2)).cuda(), (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    m = ssp()
    kw = dict(wq=w, pos=pos, inv_freq=inv, interleaved=inter, norm=m.SSMP_NORM_RMS)
    z = x.clone()
    z[2, 1, bad] = INF
    none = x[:, :0].cuda()
    y = m.qk_norm_pack_fwd(z.cuda(), none, **kw)[0].cpu()
    row = y[2, 1].tolist()
    assert row[bad] != row[bad] and all(v == 0.0 for i, v in enumerate(row) if i != bad), row
    dz = dy.clone()
    dz[2, 1, bad] = INF
    clean = m.qk_norm_pack_bwd(x.cuda(), none, dy.cuda(), none, **kw)
    got = m.qk_norm_pack_bwd(x.cuda(), none, dz.cuda(), none, **kw)
    keep = torch.arange(D) != bad
    assert torch.equal(got["dwq"].cpu()[keep], clean["dwq"].cpu()[keep])
    assert not bool(got["dwq"].cpu()[bad].isfinite())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_squares_out_of_range(dtype):
    """Components of 2e19, whose squares pass 32 bits' range: zeros, in that row alone."""
    x = torch.ones(4, 2, 64, dtype=dtype)
    x[2, 1] = 2e19
    y = ssp().qk_norm_pack_fwd(x.cuda(), x[:, :0].cuda(), eps=0.0)[0].cpu()
    assert not bool(y[2, 1].any())
    y[2, 1] = 0.125
    assert bool((y == 0.125).all())  # 1 / sqrt 64
