"""GPU: rows whose squares, or whose sum, pass the range of 32 bits, beside rows that do not."""
from __future__ import annotations

import pytest
import torch

from tests.test_layer_norm_gpu import nan_like, ssp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [8, 65, 520, 4096, 8200])
def test_rows_out_of_range(D, dtype):
    m = ssp()
    gen = torch.Generator("cuda").manual_seed(D)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, dy, dh, w, b = rnd(7, D).to(dtype), rnd(7, D).to(dtype), rnd(7, D).to(dtype), rnd(D), rnd(D)
    run = lambda x: (m.layer_norm_pack_fwd(x, w, b, out=(nan_like(x), None))[0],  # noqa: E731
                     m.layer_norm_pack_bwd(dy, x, w, dh=dh, bias=True))
    y0, G0 = run(x)
    big = x.clone()
    big[2] = torch.where(rnd(D) > 0, 1e21, -1e21).to(dtype)
    big[2, 0] = 2e21  # (not all equal)
    y, G = run(big)
    assert torch.equal(y[2], b.to(dtype)) and torch.equal(G["dx"][2], dh[2])
    others = [0, 1, 3, 4, 5, 6]
    assert torch.equal(y[others], y0[others]) and torch.equal(G["dx"][others], G0["dx"][others])
    assert bool(G["dw"].isfinite().all()) and torch.equal(G["db"], G0["db"])
    over = x.clone()
    over[2] = 3.2e38
    y, G = run(over)
    assert bool(y[2].isnan().all()) and bool(G["dx"][2].isnan().all())
    assert torch.equal(y[others], y0[others]) and torch.equal(G["dx"][others], G0["dx"][others])
