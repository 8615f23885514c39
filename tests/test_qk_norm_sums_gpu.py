"""GPU: the weights' gradients of the head norms over very many equal rows."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.mark.parametrize("T, H, D", [(1 << 20, 8, 8), (600000, 3, 16), (300000, 2, 64)])
def test_equal_rows_add_up(T, H, D):
    """Equal terms, whose rounded sums in 32 bits would drift one way. Each term
    errs by its factors' roundings: the sum of squares by D / 2 * 2^-24 of itself at
    most and the root by half of that, the root's own 2 * 2^-24 and two products:
    D / 4 + 4 of 2^-24. A lane adds up to 8 rows (of 8 tokens) in 32 bits, whose sums
    so far are rounded, 9 / 2 in all, then up to 6 times those of other lanes, 6; the
    rest is added in 64 bits and rounded twice, 2: D / 4 + 17."""
    import selective_state_space_varlen_amd as m
    gen = torch.Generator().manual_seed(80)
    x, dy = torch.randn(D, generator=gen), torch.randn(D, generator=gen)
    q = x.cuda().expand(T, H, D).contiguous()
    g = dy.cuda().expand(T, H, D).contiguous()
    none = q[:, :0].contiguous()
    w = torch.ones(D, device="cuda")
    got = m.qk_norm_pack_bwd(q, none, g, none, wq=w, norm=m.SSMP_NORM_RMS, eps=1e-6)["dwq"].cpu().to(F64)
    want = T * H * (dy.to(F64) * x.to(F64) / (x.to(F64).square().mean() + 1e-6).sqrt())
    off = ((got - want) / want).abs()
    assert float(off.max()) <= (D / 4 + 17) * 2.0 ** -24, (off * 2 ** 24).tolist()
