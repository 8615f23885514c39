"""GPU: layer norm (with the residual sum and dropout) and dropout against
their definitions in 64 bits. Buffers start as NaN."""
from __future__ import annotations

import pytest
import torch

from tests import decay_checks as ck

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def ssp():
    import selective_state_space_varlen_amd as m
    return m


def nan_like(t):
    return torch.full_like(t, float("nan"))


def rng(seed, stream):
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([wrap(seed), wrap(stream)], dtype=torch.int64, device="cuda")


def inputs(seed, T, row, dtype):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    one = [1] * len(row)
    return {"x": (rnd(T, *row) * (0.2 + torch.rand(T, *one, generator=gen)) + 2.0 * rnd(T, *one)).to(dtype),
            "res": rnd(T, *row).to(dtype), "dy": rnd(T, *row).to(dtype), "dh": rnd(T, *row).to(dtype),
            "w": 1.0 + 0.3 * rnd(*row), "b": 0.3 * rnd(*row)}


def forward(d, w, b, res, p, seeds, eps):
    x = {n: t.cuda() for n, t in d.items()}
    y, h = nan_like(x["x"]), nan_like(x["x"])
    ssp().layer_norm_pack_fwd(x["x"], x["w"] if w else None, x["b"] if b else None, eps=eps,
                              residual=x["res"] if res else None, p=p, rng=rng(*seeds), out=(y, h))
    return y, h


def sums(d, res, p, seeds):
    """h in 64 bits, the kept elements and their factor."""
    x = d["x"].to(F64)
    kept, by = ck.keep(x.numel(), p, *seeds)
    kept = kept.view(x.shape)
    h = torch.where(kept, x * by, 0.0)
    return (h + d["res"].to(F64) if res else h), kept, by


ROWS = [(1,), (2,), (3,), (7,), (8,), (24,), (64,), (65,), (72,), (128,), (250,), (256,), (264,), (512,), (520,), (1000,),
        (1025,), (1536,), (2048,), (2056,), (4096,), (4097,), (5000,), (8192,), (16384,), (16383,), (1, 8), (3, 5),
        (6, 72), (2, 128), (5, 33), (7, 520), (3, 2056)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("row", ROWS)
def test_forward_and_backward(row, dtype):
    T = 5 if row[-1] > 600 else 37
    D, eps = row[-1], 1e-3 if row[-1] < 4 else 1e-5
    d = inputs(len(row) * 1000 + D, T, row, dtype)
    for w, b, res, p in ((True, True, True, 0.25), (False, False, False, 0.0), (True, False, False, 0.0),
                         (False, True, True, 0.0)):
        seeds = (D, 17)
        h64, kept, by = sums(d, res, p, seeds)
        W, B = (d["w"].to(F64) if w else None), (d["b"].to(F64) if b else None)
        y, h = forward(d, w, b, res, p, seeds, eps)
        ck.near(h, h64, 2.0 ** -22 * (d["x"].to(F64).abs() * by + d["res"].abs().to(F64)), "h")  # two roundings of 32 bits
        ck.near(y, ck.layer_norm(h64, W, B, eps), ck.ln_tol(h64, W, eps), "y")
        # gradients, at h as it is stored
        hs = h if res or p else d["x"].cuda()
        leaf = hs.cpu().to(F64).requires_grad_()
        params = [t.clone().requires_grad_() for t in (W, B) if t is not None]
        it = iter(params)
        out = ck.layer_norm(leaf, next(it) if w else None, next(it) if b else None, eps)
        dy, dh = d["dy"].to(F64), d["dh"].to(F64)
        G = torch.autograd.grad((out * dy).sum() + ((leaf * dh).sum() if res else 0.0), [leaf] + params)
        got = ssp().layer_norm_pack_bwd(
            d["dy"].cuda(), hs, d["w"].cuda() if w else None, dh=d["dh"].cuda() if res else None, eps=eps, p=p,
            rng=rng(*seeds) if p else None, workspace=torch.full(
                (max(ssp().layer_norm_pack_bwd_workspace_bytes(T, row[0] if len(row) > 1 else 1, D), 1),), 255,
                dtype=torch.uint8, device="cuda"),
            out={"dx": nan_like(hs), "dresidual": nan_like(hs) if res else None,
                 "dw": nan_like(d["w"].cuda()) if w else None, "db": nan_like(d["b"].cuda()) if b else None})
        # dh' is r times a difference of terms of size |dy w|, as y is of h: r |dy w| in place of |w|
        dev = leaf.detach() - leaf.detach().mean(-1, keepdim=True)
        r = 1.0 / ((dev * dev).mean(-1, keepdim=True) + eps).sqrt()
        # n itself errs by ln_tol, and is multiplied by mean(c n) and summed with c (three terms)
        cw = (dy * (W if w else 1.0)).abs().amax(-1, keepdim=True)
        n_top = (dev * r).abs().amax(-1, keepdim=True).clamp(min=1.0)
        room = 3 * r * cw * n_top * ck.ln_tol(leaf.detach(), None, eps) + 2.0 ** -22 * dh.abs()
        if res:
            ck.near(got["dresidual"], G[0], room, "dresidual")
        ck.near(got["dx"], torch.where(kept, G[0] * by, 0.0), by * room, "dx")
        for name, on, gr in (("dw", w, G[1] if w else None), ("db", b, G[-1] if b else None)):
            if on:  # T terms: each errs by ln_tol of its size, and by the additions
                size = dy.abs().sum(0) * (float(ck.ln_tol(leaf.detach(), None, eps).max()) * float(n_top.max()) + T * 2.0 ** -24)
                ck.near(got[name], gr, size, name)
            else:
                assert got[name] is None


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_rows_for_each_group(dtype):
    """More rows than a lane adds up in 32 bits, in one and in several heads."""
    for row, T in (((8,), 200000), ((3, 16), 30000), ((2048,), 70000)):
        gen = torch.Generator("cuda").manual_seed(5)
        h = torch.randn(T, *row, generator=gen, device="cuda").to(dtype)
        dy = torch.randn(T, *row, generator=gen, device="cuda").to(dtype)
        w = 1.0 + torch.rand(*row, generator=gen, device="cuda")
        got = ssp().layer_norm_pack_bwd(dy, h, w, bias=True)
        x = h.double()
        dev = x - x.mean(-1, keepdim=True)
        n = dev / (dev.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        # 64 rows at a time in 32 bits: less than 64 2^-24 of a column's sum of |dy n| in the worst case; n errs by ln_tol
        tol = 64 * 2.0 ** -24 + float(ck.ln_tol(x, None, 1e-5).max())
        ck.near(got["dw"], (dy.double() * n).sum(0).cpu(), (tol * (dy.double() * n).abs().sum(0)).cpu(), "dw")
        ck.near(got["db"], dy.double().sum(0).cpu(), (64 * 2.0 ** -24 * dy.double().abs().sum(0)).cpu(), "db")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_in_place_and_repeated(dtype):
    d = inputs(3, 50, (520,), dtype)
    y, h = forward(d, True, True, True, 0.3, (5, 6), 1e-5)
    x, res = d["x"].cuda(), d["res"].cuda()
    ssp().layer_norm_pack_fwd(x, d["w"].cuda(), d["b"].cuda(), residual=res, p=0.3, rng=rng(5, 6), out=(x, res))
    assert torch.equal(x, y) and torch.equal(res, h)
    kw = dict(dh=d["dh"].cuda(), p=0.3, rng=rng(5, 6), bias=True, residual=True)
    a = ssp().layer_norm_pack_bwd(d["dy"].cuda(), h, d["w"].cuda(), **kw)
    dy = d["dy"].cuda()
    b = ssp().layer_norm_pack_bwd(dy, h.clone(), d["w"].cuda(), **dict(kw, dh=kw["dh"]),
                                  out={"dx": dy, "dresidual": kw["dh"], "dw": a["dw"].clone(), "db": a["db"].clone()})
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_a_row_that_cannot_be_normalised_stays_alone():
    d = inputs(4, 6, (136,), F32)
    d["x"][1] = float("nan")
    d["x"][2, 5] = float("inf")
    d["x"][3] = 2.5
    y, _ = forward(d, False, False, False, 0.0, (0, 0), 0.0)
    want = ck.layer_norm(d["x"].to(F64), None, None, 0.0)
    y = y.cpu()
    assert bool(y[1].isnan().all()) and bool(y[2].isnan().all()) and bool(y[3].isnan().all())
    ck.near(y[[0, 4, 5]], want[[0, 4, 5]], ck.ln_tol(d["x"].to(F64), None, 0.0)[[0, 4, 5]], "y")


def test_no_rows():
    m = ssp()
    x = torch.empty(0, 16, device="cuda")
    y, h = m.layer_norm_pack_fwd(x)
    assert y.shape == x.shape and h is None
    g = m.layer_norm_pack_bwd(x, x, nan_like(torch.empty(16, device="cuda")), bias=True)
    assert not bool(g["dw"].any()) and not bool(g["db"].any())


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 5000])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999])
def test_dropout(n, p, dtype):
    gen = torch.Generator().manual_seed(n)
    x, res, dy = (torch.randn(n, generator=gen).to(dtype) for _ in range(3))
    seeds = ((1 << 64) - 3, (1 << 40) + n)
    kept, by = ck.keep(n, p, *seeds)
    m = ssp()
    for r in (None, res):
        y = m.dropout_pack_fwd(x.cuda(), p, rng(*seeds), residual=None if r is None else r.cuda(), out=nan_like(x.cuda()))
        want = torch.where(kept, x.to(F64) * by, 0.0) + (0.0 if r is None else r.to(F64))
        ck.near(y, want, 2.0 ** -22 * (x.to(F64).abs() * by + res.to(F64).abs()) * (0.0 if r is None and not p else 1.0), "y")
    dx = m.dropout_pack_bwd(dy.cuda(), p, rng(*seeds), out=nan_like(x.cuda()))
    ck.near(dx, torch.where(kept, dy.to(F64) * by, 0.0), 2.0 ** -22 * by * dy.to(F64).abs(), "dx")
    assert torch.equal((dx.cpu() != 0) | (dy == 0), kept | (dy == 0))


def test_dropout_drops_what_is_not_finite():
    x = torch.full((4096,), float("nan"), device="cuda")
    y = ssp().dropout_pack_fwd(x, 0.5, rng(1, 2))
    kept, _ = ck.keep(4096, 0.5, 1, 2)
    assert torch.equal(y.isnan().cpu(), kept) and not bool(y[~kept.cuda()].any())


def test_dropout_share_streams_and_far_elements():
    """The share that is kept, streams that have nothing in common, and an index past 32 bits."""
    m, n = ssp(), 1 << 22
    x = torch.ones(n, device="cuda")
    a, b = m.dropout_pack_fwd(x, 0.1, rng(3, 1)) != 0, m.dropout_pack_fwd(x, 0.1, rng(3, 2)) != 0
    q = 1 - round(6553.6) / 65536
    sd = (q * (1 - q) / n) ** 0.5
    assert abs(float(a.double().mean()) - q) < 5 * sd and abs(float(b.double().mean()) - q) < 5 * sd
    assert abs(float((a & b).double().mean()) - q * q) < 5 * (q * q * (1 - q * q) / n) ** 0.5
    far = (1 << 32) + 24
    big = torch.ones(far, dtype=BF, device="cuda")
    y = m.dropout_pack_fwd(big, 0.5, rng(9, 4), out=big)
    for at in (0, (1 << 32) - 8, 1 << 32, (1 << 32) + 16):
        c = [at // 8 & 0xffffffff, at // 8 >> 32]
        k = philox_of(c, 9, 4)
        assert [bool(v) for v in (y[at:at + 8] != 0).cpu()] == [u >= 32768 for u in k]


@pytest.mark.parametrize("dtype,n", [(F32, (1 << 25) + 5), (BF, (1 << 26) + 5)])
def test_dropout_of_what_no_cache_holds(dtype, n):
    """Accesses of large tensors are others: the first elements as in a small
    call, the last ones, behind the last eight, by the definition."""
    m, few = ssp(), 4096
    x = torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dtype)
    r = x.flip(0)
    for res in (None, r):
        y = m.dropout_pack_fwd(x, 0.5, rng(9, 4), residual=res)
        assert torch.equal(y[:few], m.dropout_pack_fwd(x[:few], 0.5, rng(9, 4), residual=None if res is None else res[:few]))
        at = n // 8 * 8 - 8
        kept = torch.tensor([u >= 32768 for c in (at // 8, at // 8 + 1) for u in philox_of([c, 0], 9, 4)][:n - at])
        want = torch.where(kept, 2 * x[at:].cpu().float(), torch.zeros(()))  # p = 1/2: twice what is kept, exactly
        if res is not None:
            want = want + res[at:].cpu().float()
        assert torch.equal(y[at:].cpu(), want.to(dtype))


def test_rows_past_32_bits_of_elements():
    m, D = ssp(), 16384
    T, few = (1 << 18) + 3, 5
    o = dict(dtype=BF, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    x, dy, w = torch.randn(T, D, **o), torch.randn(T, D, **o), torch.rand(D, device="cuda")
    y, _ = m.layer_norm_pack_fwd(x, w)
    dx = m.layer_norm_pack_bwd(dy, x, w)["dx"]
    assert torch.equal(y[-few:], m.layer_norm_pack_fwd(x[-few:].clone(), w)[0])
    assert torch.equal(dx[-few:], m.layer_norm_pack_bwd(dy[-few:].clone(), x[-few:].clone(), w)["dx"])


def philox_of(c, seed, stream):
    low = 0xffffffff
    c, k = c + [stream & low, stream >> 32], [seed & low, seed >> 32]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return [u for w in c for u in (w & 0xffff, w >> 16)]
