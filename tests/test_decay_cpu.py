"""CPU tests of the linear attention, layer norm and dropout entry points:
sizes, refusals (made on the host before anything is launched), the index
arithmetic of segments, and the 64-bit references that the GPU tests compare
with."""
from __future__ import annotations

import ctypes
import random

import pytest
import torch

from tests import decay_checks as ck
from tests import delta_checks as dc

NULL, FAKE = None, ctypes.c_void_p(0x1000)  # FAKE is never dereferenced: every call fails validation first
ODD = ctypes.c_void_p(0x1008)
BIG = 1 << 40
OK, E_NULL, E_SHAPE, E_UNSUP, E_WS, E_ALIGN = 0, 1, 2, 4, 6, 8


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_varlen_amd import binding
    return binding.load()


def fwd(lib, q=FAKE, k=FAKE, v=FAKE, g=FAKE, cu=FAKE, nseq=2, out=FAKE, T=300, Hk=1, Hv=2, Dk=64, Dv=64, dtype=1, per=1,
        h0=NULL, hT=NULL, scratch=FAKE, nscratch=BIG):
    return lib.decay_attn_pack_fwd(q, k, v, g, cu, nseq, out, T, Hk, Hv, Dk, Dv, dtype, per, 0.1, h0, hT, scratch, nscratch,
                                   NULL)


def bwd(lib, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, h0=NULL, dhT=NULL, dh0=NULL, scratch=FAKE, nscratch=BIG, T=300,
        Hk=1, Hv=2, Dk=64, Dv=64, nseq=2):
    return lib.decay_attn_pack_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, nseq, dout, T, Hk, Hv, Dk, Dv, 1, 1, 0.1, h0, dhT, dh0, dq,
                                   dk, dv, dg, scratch, nscratch, NULL)


def test_attention_refusals(lib):
    for kw, st in (({"T": -1}, E_SHAPE), ({"T": 1 << 31}, E_SHAPE), ({"nseq": 0}, E_SHAPE), ({"Hk": 0}, E_SHAPE),
                   ({"Hk": 3}, E_SHAPE), ({"Dv": 0}, E_SHAPE), ({"Dk": 12}, E_UNSUP), ({"Dv": 4}, E_UNSUP),
                   ({"Dk": 136}, E_UNSUP), ({"dtype": 3}, E_UNSUP), ({"cu": NULL}, E_NULL), ({"q": NULL}, E_NULL),
                   ({"k": NULL}, E_NULL), ({"v": NULL}, E_NULL), ({"g": NULL}, E_NULL), ({"out": NULL}, E_NULL),
                   ({"v": ODD}, E_ALIGN), ({"h0": ODD}, E_ALIGN), ({"hT": ODD}, E_ALIGN), ({"scratch": ODD}, E_ALIGN),
                   ({"scratch": NULL}, E_WS), ({"nscratch": 100}, E_WS)):
        assert fwd(lib, **kw) == st, kw
    for kw, st in (({"dout": NULL}, E_NULL), ({"dq": NULL}, E_NULL), ({"dv": NULL}, E_NULL), ({"scratch": NULL}, E_WS),
                   ({"nscratch": 64}, E_WS), ({"dq": ODD}, E_ALIGN), ({"Hk": 3}, E_SHAPE), ({"dh0": ODD}, E_ALIGN),
                   ({"dhT": ODD}, E_ALIGN), ({"Dk": 136}, E_UNSUP)):
        assert bwd(lib, **kw) == st, kw
    assert fwd(lib, T=0, q=NULL, k=NULL, v=NULL, g=NULL, out=NULL, scratch=NULL, nscratch=0) == OK  # nothing to do


def test_one_buffer_for_two_states_is_refused(lib):
    """Segments of a sequence run beside each other: one would read what another has written."""
    assert fwd(lib, h0=FAKE, hT=FAKE) == E_UNSUP
    assert bwd(lib, h0=FAKE, dh0=FAKE) == E_UNSUP
    assert bwd(lib, dhT=FAKE, dh0=FAKE) == E_UNSUP


def test_more_than_a_launch_takes_is_refused(lib):
    assert fwd(lib, T=1 << 30, Hv=1, Dk=8, Dv=8) == E_SHAPE
    assert fwd(lib, T=100, nseq=1 << 23, Hv=1, Dk=8, Dv=8) == E_SHAPE
    assert fwd(lib, T=100, nseq=1 << 14, Hv=2, Dv=1 << 19) == E_SHAPE
    assert fwd(lib, T=100, Hv=7000, Dk=128, Dv=136) == E_SHAPE  # a row of dq's parts
    assert bwd(lib, T=100, Hv=7000, Dk=128, Dv=136) == E_SHAPE
    assert lib.decay_attn_pack_fwd_scratch_bytes(1 << 30, 2, 1, 1, 8, 8) == 0


def test_step_refusals(lib):
    def step(q=FAKE, g=FAKE, state=FAKE, slots=FAKE, out=FAKE, B=4, nslots=8, Hk=1, Hv=2, Dk=64, Dv=64, dtype=1):
        return lib.decay_attn_pack_step(q, FAKE, FAKE, g, state, slots, out, B, nslots, Hk, Hv, Dk, Dv, dtype, 1, 0.1, NULL)
    for kw, st in (({"B": -1}, E_SHAPE), ({"B": 9, "slots": NULL}, E_SHAPE), ({"Hk": 3}, E_SHAPE), ({"Dk": 136}, E_UNSUP),
                   ({"Dv": 12}, E_UNSUP), ({"dtype": 2}, E_UNSUP), ({"q": NULL}, E_NULL), ({"g": NULL}, E_NULL),
                   ({"state": NULL}, E_NULL), ({"out": ODD}, E_ALIGN), ({"state": ODD}, E_ALIGN), ({"B": 1 << 30}, E_SHAPE)):
        assert step(**kw) == st, kw
    assert step(B=0, q=NULL) == OK


def test_layer_norm_refusals(lib):
    def f(x=FAKE, res=NULL, w=FAKE, b=FAKE, rng=FAKE, y=FAKE, h=FAKE, T=4, H=1, D=64, dtype=1, p=0.1):
        return lib.layer_norm_pack_fwd(x, res, w, b, rng, y, h, T, H, D, dtype, p, 1e-5, NULL)
    for kw, st in (({"T": -1}, E_SHAPE), ({"T": 1 << 31}, E_SHAPE), ({"H": 0}, E_SHAPE), ({"H": 1 << 17}, E_SHAPE),
                   ({"D": 0}, E_SHAPE), ({"D": 16385}, E_UNSUP), ({"dtype": 2}, E_UNSUP), ({"p": 1.0}, E_SHAPE),
                   ({"p": 0.999999}, E_SHAPE), ({"p": -0.1}, E_SHAPE), ({"p": float("nan")}, E_SHAPE), ({"x": NULL}, E_NULL),
                   ({"y": NULL}, E_NULL), ({"rng": NULL}, E_NULL), ({"x": ODD}, E_ALIGN), ({"res": ODD}, E_ALIGN),
                   ({"h": ODD}, E_ALIGN)):
        assert f(**kw) == st, kw
    assert f(T=0, x=NULL, y=NULL) == OK
    big = lib.layer_norm_pack_bwd_workspace_bytes(4, 1, 64)

    def b(dy=FAKE, h=FAKE, w=FAKE, dh=NULL, rng=FAKE, dx=FAKE, dr=NULL, dw=FAKE, db=FAKE, ws=FAKE, n=big, T=4, p=0.0):
        return lib.layer_norm_pack_bwd(dy, h, w, dh, rng, dx, dr, dw, db, ws, n, T, 1, 64, 1, p, 1e-5, NULL)
    for kw, st in (({"dy": NULL}, E_NULL), ({"h": NULL}, E_NULL), ({"dx": NULL}, E_NULL), ({"w": NULL}, E_NULL),
                   ({"ws": NULL}, E_WS), ({"n": big - 1}, E_WS), ({"ws": ODD}, E_ALIGN), ({"dh": ODD}, E_ALIGN),
                   ({"dr": ODD}, E_ALIGN), ({"p": 0.5, "rng": NULL}, E_NULL), ({"p": 2.0}, E_SHAPE)):
        assert b(**kw) == st, kw
    assert lib.layer_norm_pack_bwd_workspace_bytes(4, 1, 16385) == 0
    assert lib.layer_norm_pack_bwd_workspace_bytes(0, 1, 64) == 0


def test_dropout_refusals(lib):
    def f(x=FAKE, r=NULL, rng=FAKE, y=FAKE, n=100, dtype=1, p=0.1):
        return lib.dropout_pack_fwd(x, r, rng, y, n, dtype, p, NULL)
    for kw, st in (({"n": -1}, E_SHAPE), ({"n": 1 << 40}, E_SHAPE), ({"dtype": 2}, E_UNSUP), ({"p": 1.0}, E_SHAPE),
                   ({"p": -1e-9}, E_SHAPE), ({"p": float("nan")}, E_SHAPE), ({"x": NULL}, E_NULL), ({"y": NULL}, E_NULL),
                   ({"rng": NULL}, E_NULL), ({"x": ODD}, E_ALIGN), ({"r": ODD}, E_ALIGN), ({"y": ODD}, E_ALIGN)):
        assert f(**kw) == st, kw
    assert f(n=0, x=NULL) == OK
    assert lib.dropout_pack_bwd(NULL, FAKE, FAKE, 4, 1, 0.1, NULL) == E_NULL


HEADS = [  # Hk, Hv, Dk, Dv
    (4, 4, 128, 128), (1, 1, 8, 8), (1, 2, 64, 72), (2, 4, 40, 200), (1, 24, 128, 64), (8, 16, 128, 128), (1, 32, 64, 64),
    (16, 32, 128, 128), (1, 1, 128, 2048), (1, 100, 8, 8),
]


@pytest.mark.parametrize("heads", HEADS)
def test_sizes_never_fall(lib, heads):
    tokens = sorted(set(range(0, 40000, 61)) | {128 * i + j for i in range(1, 80) for j in (-1, 0, 1)}
                    | {2048 * i for i in range(1, 40)} | {1 << 17, 1 << 18, 1 << 19})
    for f in (lib.decay_attn_pack_fwd_scratch_bytes, lib.decay_attn_pack_bwd_scratch_bytes):
        for n in (1, 2, 3, 7, 8, 23, 24, 25, 32, 33, 100):
            sizes = [f(T, n, *heads) for T in tokens]
            assert sizes == sorted(sizes), n
        for T in (1, 63, 128, 129, 2047, 2048, 4096, 8192, 16385, 65536, 1 << 18):
            sizes = [f(T, n, *heads) for n in range(1, 130)]
            assert sizes == sorted(sizes), T


@pytest.mark.parametrize("row", [(1, 1), (1, 8), (1, 72), (6, 72), (1, 100), (3, 250), (1, 600), (1, 4096), (1, 4097), (1, 16384),
                                 (32, 128), (7, 9)])
def test_layer_norm_sizes_never_fall(lib, row):
    tokens = [T for T in list(range(0, 9000)) + [1 << i for i in range(14, 27)] if T * row[0] * row[1] < 1 << 40]
    sizes = [lib.layer_norm_pack_bwd_workspace_bytes(T, *row) for T in tokens]
    assert sizes == sorted(sizes)


def segment(T, nseq, work):
    """Tokens of a segment, by the rule beside the kernels."""
    if nseq * work >= 768:
        return 2048
    return min(max(T * work // 768 // 128 * 128, 128), 2048)


@pytest.mark.parametrize("heads", HEADS)
def test_states_between_segments_lie_inside_the_scratch(lib, heads):
    Hk, Hv, Dk, Dv = heads
    rng = random.Random(1)
    blocks = -(-Dv // 128)
    for T in [1, 127, 128, 129, 255, 256, 257, 500, 1000, 2047, 2048, 2049, 4097, 10000, 16384, 33000, 100000]:
        for nseq in (1, 2, 5, 9, 24, 100, 800):
            for work, scratch, ways in ((Hv * blocks, lib.decay_attn_pack_fwd_scratch_bytes(T, nseq, *heads), 1),
                                        (Hv, lib.decay_attn_pack_bwd_scratch_bytes(T, nseq, *heads), 2)):
                seg = segment(T, nseq, work)
                if T <= seg:
                    continue
                need = (T // seg + 1) * Hv * (Dk * Dv + 1) * 4 * ways
                assert scratch >= need, (T, nseq, seg)
                # no two sequences' states meet, whatever the division
                cuts = sorted(rng.randint(0, T) for _ in range(nseq - 1))
                cu = [0] + cuts + [T]
                seen = set()
                for a, b in zip(cu, cu[1:]):
                    for i in range(max(0, (b - a - 1) // seg)):
                        assert 0 <= a // seg + i <= T // seg and (a // seg + i) not in seen
                        seen.add(a // seg + i)
                # nor what dg's anchors keep behind every 256 tokens
                seen = set()
                for a, b in zip(cu, cu[1:]):
                    for i in range(max(0, (b - a - 1) // 256)):
                        assert 0 <= a // 256 + i < T // 256 and (a // 256 + i) not in seen
                        seen.add(a // 256 + i)


def test_segments_by_length():
    """The order in which a launch takes the segments of up to 64 sequences is one of all of them."""
    rng = random.Random(2)
    for _ in range(200):
        nseq, seg = rng.randint(1, 64), 128 * rng.randint(1, 16)
        lens = [rng.choice((0, 1, seg - 1, seg, seg + 1, rng.randint(0, 5 * seg))) for _ in range(nseq)]
        whole = [n // seg for n in lens]
        rest = [n % seg if n == 0 or n % seg else -1 for n in lens]
        before = [sum(whole[:i + 1]) for i in range(nseq)]
        got = []
        for r in range(sum(lens) // seg + nseq):
            if r < before[-1]:
                at = sum(b <= r for b in before)
                got.append((at, r - (before[at] - whole[at])))
            else:
                rank = [sum(v > rest[i] or (v == rest[i] and s < i) for s, v in enumerate(rest)) for i in range(nseq)]
                hit = [i for i in range(nseq) if rest[i] >= 0 and rank[i] == r - before[-1]]
                got += [(i, whole[i]) for i in hit[:1]]
        want = {(s, i) for s, n in enumerate(lens) for i in range(max(1, -(-n // seg)))}
        assert len(got) == len(set(got)) and set(got) == want
        sizes = [min(seg, lens[s] - i * seg) for s, i in got]
        assert sizes == sorted(sizes, reverse=True)


def test_binding_refusals():
    import selective_state_space_varlen_amd as m
    q, g = torch.zeros(4, 1, 64), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="device tensor"):
        m.decay_attn_pack_fwd(q, q, q, g, dc.cu_of([4]))
    with pytest.raises(ValueError, match="device tensor"):
        m.decay_attn_pack_bwd(q, q, q, g, dc.cu_of([4]), q)
    with pytest.raises(ValueError, match="heads"):
        m.decay_attn_pack_step(q[0], q, q, g, torch.zeros(1, 1, 64, 64))
    with pytest.raises(TypeError):
        m.decay_attn_pack_fwd(q.half(), q.half(), q.half(), g, dc.cu_of([4]))
    with pytest.raises(ValueError, match="tokens, size"):
        m.layer_norm_pack_fwd(torch.zeros(4))
    with pytest.raises(ValueError, match="device tensor"):
        m.layer_norm_pack_fwd(torch.zeros(4, 8))
    with pytest.raises(ValueError, match="device tensor"):
        m.dropout_pack_fwd(torch.zeros(4, 8), 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        m.dropout_pack_fwd(torch.zeros(4, 8).half(), 0.1, torch.zeros(2, dtype=torch.int64))


def test_block_refusals():
    import selective_state_space_varlen_amd as m
    t, cu = torch.zeros(4, 8), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="rotation"):
        m.decay_forward((t, t, t), t, cu, 1, 1, inv_freq=torch.ones(4))
    with pytest.raises(ValueError, match="without convs"):
        m.decay_forward((t, t, t), t, cu, 1, 1, initial_states={"conv": (t, t, t)})
    fwd_ = {"cu_seqlens": cu, "carry": False, "initial_states": {}, "convs": (None, None)}
    with pytest.raises(ValueError, match="final states"):
        m.decay_backward((t, t, t), t, fwd_, t, dfinal_states={"decay": t})
    with pytest.raises(ValueError, match="without convs"):
        m.decay_backward((t, t, t), t, dict(fwd_, carry=True), t, dfinal_states={"conv": (t, t, t)})


def test_reference_gradients_by_differences():
    lens, eps = [3, 0, 4], 1e-6
    for per_token in (True, False):
        d = ck.inputs(1, lens, 1, 2, 8, 8, torch.float32, True, per_token)
        ref = ck.reference(d, lens, 0.3)
        names = {"q": "dq", "k": "dk", "v": "dv", "g": "dg", "h0": "dh0"}

        def loss(x):
            out, hT = ck.attention(x["q"], x["k"], x["v"], x["g"], lens, 0.3, x["h0"])
            return float((out * d["dout"].double()).sum() + (hT * d["dhT"].double()).sum())
        x = {n: d[n].double() for n in names}
        gen = torch.Generator().manual_seed(3)
        for n, gname in names.items():
            way = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
            up, down = (loss(dict(x, **{n: x[n] + s * eps * way})) for s in (1, -1))
            assert abs((up - down) / (2 * eps) - float((ref[gname] * way).sum())) < 1e-6 * (1 + abs(up - down) / eps)


def test_generator_known_values():
    """Philox4x32-10's published results for a counter and key of zeros, and of ones."""
    assert [x.item() for x in ck.keep(8, 0.0, 0, 0)[0]] == [True] * 8
    from tests.test_layer_norm_gpu import philox_of
    halves = lambda *w: [h for x in w for h in (x & 0xffff, x >> 16)]  # noqa: E731
    assert philox_of([0, 0], 0, 0) == halves(0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)
    ones = 0xffffffff
    assert philox_of([ones, ones], (1 << 64) - 1, (1 << 64) - 1) == halves(0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)
