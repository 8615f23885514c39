"""CPU tests of the delta-rule and head-norm entry points: sizes, refusals
(made on the host before anything is launched), and the 64-bit references that
the GPU tests compare with."""
from __future__ import annotations

import ctypes

import pytest
import torch

from tests import delta_checks as dc

NULL, FAKE = None, ctypes.c_void_p(0x1000)  # FAKE is never dereferenced: every call fails validation first
ODD = ctypes.c_void_p(0x1008)
BIG = 1 << 40
OK, E_NULL, E_SHAPE, E_UNSUP, E_WS, E_ALIGN = 0, 1, 2, 4, 6, 8


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_varlen_amd import binding
    return binding.load()


def norm_fwd(lib, q=FAKE, k=FAKE, wq=NULL, wk=NULL, pos=FAKE, inv=FAKE, yq=FAKE, yk=FAKE, T=4, Hq=2, Hk=1, D=64, rot=32,
             dtype=1, norm=0, inter=0):
    return lib.qk_norm_pack_fwd(q, k, wq, wk, pos, inv, yq, yk, T, Hq, Hk, D, rot, dtype, norm, 1e-6, inter, NULL)


def test_norm_refusals(lib):
    for kw, st in (({"T": -1}, E_SHAPE), ({"T": 1 << 31}, E_SHAPE), ({"Hq": -1}, E_SHAPE), ({"Hq": 0, "Hk": 0}, E_SHAPE),
                   ({"D": 0}, E_SHAPE), ({"rot": -2}, E_SHAPE), ({"rot": 66}, E_SHAPE), ({"D": 12, "rot": 0}, E_UNSUP),
                   ({"D": 520, "rot": 0}, E_UNSUP), ({"rot": 8}, E_UNSUP), ({"rot": 3, "inter": 1}, E_UNSUP),
                   ({"dtype": 2}, E_UNSUP), ({"norm": 2}, E_UNSUP), ({"pos": NULL}, E_NULL), ({"inv": NULL}, E_NULL),
                   ({"q": NULL}, E_NULL), ({"yk": NULL}, E_NULL), ({"q": ODD}, E_ALIGN), ({"yk": ODD}, E_ALIGN)):
        assert norm_fwd(lib, **kw) == st, kw
    assert norm_fwd(lib, T=0, q=NULL, k=NULL, yq=NULL, yk=NULL) == OK  # nothing to do, nothing launched

    def bwd(dwq=FAKE, wq=FAKE, ws=FAKE, nb=BIG, dyk=FAKE):
        return lib.qk_norm_pack_bwd(FAKE, FAKE, wq, NULL, NULL, NULL, FAKE, dyk, FAKE, FAKE, dwq, NULL, ws, nb, 4, 2, 1,
                                    64, 0, 1, 0, 1e-6, 0, NULL)
    assert bwd(wq=NULL) == E_NULL and bwd(dyk=NULL) == E_NULL
    need = lib.qk_norm_pack_bwd_workspace_bytes(4, 2, 1, 64)
    assert need > 0 and bwd(ws=NULL) == E_WS and bwd(nb=need - 1) == E_WS and bwd(ws=ODD) == E_ALIGN
    assert lib.qk_norm_pack_bwd_workspace_bytes(0, 2, 1, 64) == 0
    assert lib.qk_norm_pack_bwd_workspace_bytes(4, 2, 1, 1024) == 0


def rule_fwd(lib, q=FAKE, v=FAKE, g=FAKE, cu=FAKE, nseq=2, out=FAKE, T=100, Hk=1, Hv=2, Dk=64, Dv=64, dtype=1, h0=NULL,
             saved=NULL, nsaved=0, scratch=FAKE, nscratch=BIG):
    return lib.gated_delta_pack_fwd(q, FAKE, v, g, FAKE, cu, nseq, out, T, Hk, Hv, Dk, Dv, dtype, 0.1, h0, NULL, saved,
                                    nsaved, scratch, nscratch, NULL)


def rule_bwd(lib, dout=FAKE, saved=FAKE, nsaved=BIG, scratch=FAKE, nscratch=BIG, dg=FAKE, dq=FAKE, Hk=1, dh0=NULL):
    return lib.gated_delta_pack_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, 2, dout, 100, Hk, 2, 64, 64, 1, 0.1, NULL, dh0, dq, FAKE,
                                    FAKE, dg, FAKE, saved, nsaved, scratch, nscratch, NULL)


def test_rule_refusals(lib):
    for kw, st in (({"T": -1}, E_SHAPE), ({"T": 1 << 31}, E_SHAPE), ({"nseq": 0}, E_SHAPE), ({"Hk": 0}, E_SHAPE),
                   ({"Hk": 3}, E_SHAPE), ({"Dv": 0}, E_SHAPE), ({"Dk": 12}, E_UNSUP), ({"Dv": 4}, E_UNSUP),
                   ({"Dk": 136}, E_UNSUP), ({"dtype": 3}, E_UNSUP), ({"cu": NULL}, E_NULL), ({"q": NULL}, E_NULL),
                   ({"g": NULL}, E_NULL), ({"out": NULL}, E_NULL), ({"v": ODD}, E_ALIGN), ({"h0": ODD}, E_ALIGN),
                   ({"scratch": ODD}, E_ALIGN), ({"scratch": NULL}, E_WS), ({"nscratch": 100}, E_WS),
                   ({"saved": FAKE, "nsaved": 100}, E_WS)):
        assert rule_fwd(lib, **kw) == st, kw
    for kw, st in (({"dout": NULL}, E_NULL), ({"dg": NULL}, E_NULL), ({"saved": NULL}, E_WS), ({"nsaved": 64}, E_WS),
                   ({"scratch": NULL}, E_WS), ({"nscratch": 64}, E_WS), ({"dq": ODD}, E_ALIGN), ({"Hk": 3}, E_SHAPE),
                   ({"dh0": ODD}, E_ALIGN)):
        assert rule_bwd(lib, **kw) == st, kw
    assert rule_fwd(lib, T=0, q=NULL, out=NULL, scratch=NULL, nscratch=0) == OK  # nothing to do


def test_more_threads_than_a_launch_takes_are_refused(lib):
    assert norm_fwd(lib, T=1 << 26) == E_SHAPE
    assert rule_fwd(lib, T=1 << 30, Hk=1, Hv=1, Dk=8, Dv=8) == E_SHAPE       # chunks
    assert rule_fwd(lib, T=100, nseq=1 << 23, Hk=1, Hv=1, Dk=8, Dv=8) == E_SHAPE  # chunks, of which each sequence has a slot
    assert rule_fwd(lib, T=100, nseq=1 << 14, Hv=2, Dv=1 << 19) == E_SHAPE   # chains
    assert lib.gated_delta_pack_step(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 19, 8, 1, 32, 64, 32, 1, 0.1,
                                     NULL) == E_SHAPE
    assert lib.qk_norm_pack_bwd_workspace_bytes(1 << 26, 2, 1, 64) == 0
    assert lib.gated_delta_pack_saved_bytes(1 << 30, 2, 1, 1, 8, 8) == 0


def test_rule_sizes(lib):
    T, n, Hk, Hv, Dk, Dv = 1000, 3, 1, 2, 64, 40
    slots = T // 64 + n
    assert lib.gated_delta_pack_saved_bytes(T, n, Hk, Hv, Dk, Dv) >= slots * Hv * (Dk * Dv + 64 * Dv) * 4
    for dt in (0, 1):
        assert lib.gated_delta_pack_fwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, dt) > 0
        assert (lib.gated_delta_pack_bwd_scratch_bytes(T, n, Hk, Hv, Dk, Dv, dt)
                >= slots * Hv * (Dk * Dv + 64 * Dv) * 4)
    for bad in ((T, 0, 1, 2, 64, 40), (T, 3, 2, 3, 64, 40), (T, 3, 1, 2, 60, 40), (0, 3, 1, 2, 64, 40)):
        assert lib.gated_delta_pack_saved_bytes(*bad) == 0
        assert lib.gated_delta_pack_fwd_scratch_bytes(*bad, 1) == 0
        assert lib.gated_delta_pack_bwd_scratch_bytes(*bad, 1) == 0


def test_step_refusals(lib):
    def step(q=FAKE, state=FAKE, slots=FAKE, out=FAKE, B=4, nslots=8, Hk=1, Hv=2, Dk=64, Dv=64, dtype=1):
        return lib.gated_delta_pack_step(q, FAKE, FAKE, FAKE, FAKE, state, slots, out, B, nslots, Hk, Hv, Dk, Dv, dtype,
                                         0.1, NULL)
    for kw, st in (({"B": -1}, E_SHAPE), ({"B": 9, "slots": NULL}, E_SHAPE), ({"Hk": 3}, E_SHAPE), ({"Dk": 136}, E_UNSUP),
                   ({"Dv": 12}, E_UNSUP), ({"dtype": 2}, E_UNSUP), ({"q": NULL}, E_NULL), ({"state": NULL}, E_NULL),
                   ({"out": ODD}, E_ALIGN), ({"state": ODD}, E_ALIGN), ({"B": 1 << 30, "slots": FAKE}, E_SHAPE)):
        assert step(**kw) == st, kw
    assert step(B=0, q=NULL) == OK


def test_binding_refuses_host_and_misshapen_tensors():
    import selective_state_space_varlen_amd as m
    q, g = torch.zeros(4, 1, 64), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="device tensor"):
        m.gated_delta_pack_fwd(q, q, q, g, g, dc.cu_of([4]))
    with pytest.raises(ValueError, match="device tensor"):
        m.qk_norm_pack_fwd(q, q)
    with pytest.raises(ValueError, match="heads"):
        m.gated_delta_pack_step(q[0], q, q, g, g, torch.zeros(1, 1, 64, 64))
    with pytest.raises(ValueError, match="heads"):
        m.qk_norm_pack_fwd(q[0], q)


def test_slots_of_sequences_never_meet():
    """floor(cu[s] / 64) + s + c is another slot for every chunk, below T / 64 + nseq."""
    gen = torch.Generator().manual_seed(1)
    for _ in range(200):
        n = int(torch.randint(1, 12, (1,), generator=gen))
        lens = [int(x) for x in torch.randint(0, 200, (n,), generator=gen)]
        seen, start = set(), 0
        for s, m in enumerate(lens):
            for c in range(-(-m // 64)):
                slot = start // 64 + s + c
                assert slot not in seen and slot < sum(lens) // 64 + n
                seen.add(slot)
            start += m


def test_reference_gradients_against_differences():
    lens, Hk, Hv, Dk, Dv = [3, 4], 1, 2, 8, 8
    d = dc.rule_inputs(1, lens, Hk, Hv, Dk, Dv, torch.float32, True)
    x = [d[n].to(dc.F64).requires_grad_() for n in ("q", "k", "v", "g", "beta", "h0")]
    assert torch.autograd.gradcheck(lambda *a: dc.rule(*a[:5], lens, 0.4, a[5]), x)
    y = torch.randn(3, 2, 16, dtype=dc.F64, requires_grad=True)
    w = torch.randn(16, dtype=dc.F64, requires_grad=True)
    pos, inv = torch.tensor([0, 5, 9], dtype=torch.int32), torch.tensor([1.0, 0.1, 0.01, 0.5])
    for l2 in (False, True):
        for inter in (False, True):
            assert torch.autograd.gradcheck(lambda a, b: dc.norm(a, b, pos, inv, l2, 1e-3, inter), (y, w))


def test_reference_rotation_keeps_lengths_and_counts_positions():
    x = torch.randn(5, 1, 8, dtype=dc.F64)
    inv = torch.tensor([1.0, 0.3])
    for inter in (False, True):
        y = dc.turn(x, torch.arange(5), inv, inter)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1)) and torch.equal(y[0], x[0])
        z = dc.turn(dc.turn(x, torch.full((5,), 3), inv, inter), torch.full((5,), -3), inv, inter)
        assert torch.allclose(z, x)
