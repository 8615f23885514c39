"""GPU: whatever cu_seqlens holds, the linear attention's calls write inside
their buffers: every output and both scratches lie between guards. So do those
of the layer norm and of dropout, for rows that no wide piece divides."""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck
from tests.test_decay_gpu import BF, F32, dev, ssp
from tests.test_delta_guards_gpu import Guarded

pytestmark = pytest.mark.gpu

FORMS = [
    # T, nseq, Hk, Hv, Dk, Dv
    (200, 3, 1, 2, 64, 40),      # a few sequences
    (131, 1, 1, 1, 8, 8),        # one, over a segment
    (700, 9, 2, 4, 128, 72),
    (1500, 70, 1, 2, 32, 136),   # more sequences than lanes; wide value heads
    (600, 140, 1, 2, 128, 72),   # both value heads in a workgroup
]


@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form", FORMS)
def test_any_cu_seqlens(form, dtype, per_token):
    T, n, Hk, Hv, Dk, Dv = form
    m = ssp()
    d = dev(ck.inputs(1, [T], Hk, Hv, Dk, Dv, dtype, False, per_token))
    state = torch.empty(n, Hv, Dk, Dv, device="cuda")
    h0 = torch.randn(n, Hv, Dk, Dv, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    like = {"out": d["v"], "dq": d["q"], "dk": d["k"], "dv": d["v"], "dg": d["g"], "hT": state, "dh0": state}
    sizes = {name: t.numel() * t.element_size() for name, t in like.items()}
    sizes["fwd"] = m.decay_attn_pack_fwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv)
    sizes["bwd"] = m.decay_attn_pack_bwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv)
    room = Guarded(sizes)
    t = {name: room.view(name, x) for name, x in like.items()}
    gen = torch.Generator().manual_seed(3)
    cus = [torch.linspace(0, T, n + 1).to(torch.int32)]
    cus += [torch.randint(-2 * T, 3 * T, (n + 1,), generator=gen, dtype=torch.int32) for _ in range(6)]
    cus += [torch.full((n + 1,), v, dtype=torch.int32) for v in (0, T, -5, T + 9, (1 << 31) - 1, -(1 << 31))]
    cus.append(torch.tensor([0, T] * (n + 1), dtype=torch.int32)[:n + 1])  # all sequences the same one, or none
    for cu in cus:
        cu = cu.cuda().contiguous()
        for name in ("fwd", "bwd"):
            room.bytes(name).fill_(255)
        m.decay_attn_pack_fwd(d["q"], d["k"], d["v"], d["g"], cu, initial_state=h0, final_state=t["hT"],
                              scratch=room.bytes("fwd"), out=t["out"])
        m.decay_attn_pack_bwd(d["q"], d["k"], d["v"], d["g"], cu, d["dout"], initial_state=h0, dfinal_state=h0,
                              dinitial_state=t["dh0"], scratch=room.bytes("bwd"),
                              out={name: t[name] for name in ("dq", "dk", "dv", "dg")})
        assert not room.broken(), cu.tolist()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,row", [(1, (1,)), (3, (5,)), (7, (72,)), (5, (3, 33)), (2, (1025,)), (3, (4104,)), (2, (16383,))])
def test_rows(T, row, dtype):
    m = ssp()
    gen = torch.Generator("cuda").manual_seed(4)
    x, res, dy = (torch.randn(T, *row, device="cuda", generator=gen).to(dtype) for _ in range(3))
    w, b = torch.randn(*row, device="cuda", generator=gen), torch.randn(*row, device="cuda", generator=gen)
    rng = torch.tensor([1, 2], device="cuda")
    like = {"y": x, "h": x, "dx": x, "dr": x, "dw": w, "db": w, "z": x}
    sizes = {name: t.numel() * t.element_size() for name, t in like.items()}
    sizes["ws"] = m.layer_norm_pack_bwd_workspace_bytes(T, row[0] if len(row) > 1 else 1, row[-1])
    room = Guarded(sizes)
    t = {name: room.view(name, v) for name, v in like.items()}
    m.layer_norm_pack_fwd(x, w, b, residual=res, p=0.2, rng=rng, out=(t["y"], t["h"]))
    m.layer_norm_pack_bwd(dy, t["h"], w, dh=res, p=0.2, rng=rng, workspace=room.bytes("ws"),
                          out={"dx": t["dx"], "dresidual": t["dr"], "dw": t["dw"], "db": t["db"]})
    m.dropout_pack_fwd(x, 0.2, rng, residual=res, out=t["z"])
    assert not room.broken()
