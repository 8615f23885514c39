"""GPU: the layer norm of the most heads, wider than its weights' gradients are
formed for, against the definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck
from tests.test_layer_norm_gpu import nan_like, ssp

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF])
def test_most_heads(dtype):
    m, T, H, D, eps = ssp(), 2, 65536, 1032, 1e-5
    gen = torch.Generator("cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, dy, w, b = rnd(T, H, D).to(dtype), rnd(T, H, D).to(dtype), 1.0 + 0.3 * rnd(H, D), rnd(H, D)
    y, _ = m.layer_norm_pack_fwd(x, w, b, eps=eps, out=(nan_like(x), None))
    dx = m.layer_norm_pack_bwd(dy, x, w, eps=eps, out={"dx": nan_like(x), "dresidual": None, "dw": None, "db": None})["dx"]
    with pytest.raises(RuntimeError, match="out of range"):
        m.layer_norm_pack_bwd(dy, x, w, eps=eps, bias=True)
    for heads in (slice(0, 40), slice(32700, 32800), slice(H - 40, H)):
        h, W = x[:, heads].double(), w[heads].double()
        leaf = h.clone().requires_grad_()
        out = ck.layer_norm(leaf, W, b[heads].double(), eps)
        ck.near(y[:, heads], out.detach().cpu(), ck.ln_tol(h.cpu(), W.cpu(), eps), "y")
        (G,) = torch.autograd.grad((out * dy[:, heads].double()).sum(), leaf)
        # as in the tests of fewer heads: r |dy w| in place of |w|, three terms, n's own error
        dev = h - h.mean(-1, keepdim=True)
        r = 1.0 / ((dev * dev).mean(-1, keepdim=True) + eps).sqrt()
        cw = (dy[:, heads].double() * W).abs().amax(-1, keepdim=True)
        n_top = (dev * r).abs().amax(-1, keepdim=True).clamp(min=1.0)
        ck.near(dx[:, heads], G.cpu(), (3 * r * cw * n_top).cpu() * ck.ln_tol(h.cpu(), None, eps), "dx")
    for t in (y, dx):
        assert not bool(t.isnan().any())
