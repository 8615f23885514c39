"""64-bit definitions on the CPU of linear attention with a decay, of the layer
norm and of dropout, seeded inputs, and what their tests allow.

Tolerances of the attention are those of the delta rule (tests/delta_checks.py),
whose state map is the same without the correction: it contracts (a <= 1), so
roundings of 2^-24 made at one token are not magnified later (`tol32`, with
max(Dk, Dv) in place of Dk, as the gradients exchange the two). Where a bf16
result is formed without dg, the decayed products and the state stand as two
cut bf16 parts each against an operand that is exact: an rms of 2^-14 / 3 of a
term each, sqrt 2 of that together, below 2^-15 of the largest value; four
times that, 2^-13, is allowed (`tol_parts`).

Layer norm: with D components of a row summed in 32 bits by pairs (a lane's at
most 64, then a tree), a mean errs by less than (64 + 10) 2^-24 of the mean size
of the row's components and the variance likewise; y is the quotient of two
such, so 4 * 74 * 2^-24 < 2^-15 of (1 + |mean| r) |w| bounds it in the worst case;
the errors of the additions are independent, so an eighth of that, 2^-18, is
four times their rms for any D here. The size of the mean counts, because h -
mean cancels: `ln_tol` takes max|h| r for it.
"""
from __future__ import annotations

import math

import torch

from tests import delta_checks as dc

F64 = torch.float64


def tol32(L: int, Dk: int, Dv: int) -> float:
    return dc.tol32(L, max(Dk, Dv))


def tol_parts(name: str, dtype, dg: bool = True) -> float:
    if dtype == torch.float32 or name not in ("out", "dq", "dk", "dv") or (dg and name in ("dq", "dk")):
        return 0.0
    return 2.0 ** -13


def attention(q, k, v, g, lens, scale, h0=None):
    """(out, final states) from the definition, token by token; differentiable."""
    Hv, Dk, Dv = v.shape[1], q.shape[2], v.shape[2]
    r = Hv // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    a = g.exp().expand(v.shape[0], Hv)
    outs, states, t = [], [], 0
    for s, n in enumerate(lens):
        S = torch.zeros(Hv, Dk, Dv, dtype=F64) if h0 is None else h0[s]
        for _ in range(n):
            S = S * a[t][:, None, None] + k[t][:, :, None] * v[t][:, None, :]
            outs.append(scale * (S * q[t][:, :, None]).sum(1))
            t += 1
        states.append(S)
    return torch.stack(outs) if outs else torch.zeros(0, Hv, Dv, dtype=F64), torch.stack(states)


def inputs(seed, lens, Hk, Hv, Dk, Dv, dtype, carry, per_token=True, tail=0):
    """Seeded inputs on the CPU: unit queries and keys, decays of 1e-3 to 1.6
    by token, or memories of 4 to 4096 tokens by head. `tail` more rows follow."""
    gen = torch.Generator().manual_seed(seed)
    T, n = sum(lens) + tail, len(lens)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()).to(dtype)  # noqa: E731
    g = -torch.exp(rnd(T, Hv) - 3.0) if per_token else torch.log1p(-torch.exp2(-2.0 - 10.0 * torch.rand(Hv, generator=gen)))
    return {"q": unit(rnd(T, Hk, Dk)), "k": unit(rnd(T, Hk, Dk) + 0.5 * rnd(Hk, Dk)), "v": rnd(T, Hv, Dv).to(dtype),
            "g": g, "dout": rnd(T, Hv, Dv).to(dtype), "h0": 0.3 * rnd(n, Hv, Dk, Dv) if carry else None,
            "dhT": 0.3 * rnd(n, Hv, Dk, Dv) if carry else None}


def reference(d, lens, scale):
    """Outputs and gradients in 64 bits: {"out", "hT", "dq", ..., "dh0"}."""
    T = sum(lens)
    x = {n: d[n][:T].to(F64).requires_grad_() for n in ("q", "k", "v")}
    g = (d["g"][:T] if d["g"].dim() == 2 else d["g"]).to(F64).requires_grad_()
    h0 = None if d["h0"] is None else d["h0"].to(F64).requires_grad_()
    out, hT = attention(x["q"], x["k"], x["v"], g, lens, scale, h0)
    loss = (out * d["dout"][:T].to(F64)).sum()
    if d["dhT"] is not None:
        loss = loss + (hT * d["dhT"].to(F64)).sum()
    leaves = list(x.values()) + [g] + ([] if h0 is None else [h0])
    grads = torch.autograd.grad(loss, leaves, allow_unused=True) if loss.requires_grad else [None] * len(leaves)
    grads = [torch.zeros_like(p) if gr is None else gr for gr, p in zip(grads, leaves)]
    res = {"out": out.detach(), "hT": hT.detach()}
    res.update(zip(("dq", "dk", "dv", "dg", "dh0"), grads))
    return res


def keep(n: int, p: float, seed: int, stream: int):
    """(kept, factor) of elements 0 .. n - 1, by Philox4x32-10 in Python's integers."""
    cut, low = round(65536 * p), 0xffffffff
    numbers = []
    for i in range(-(-n // 8)):
        c = [i & low, i >> 32, stream & low, (stream >> 32) & low]
        k = [seed & low, (seed >> 32) & low]
        for _ in range(10):
            a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
            k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
        for w in c:
            numbers += [w & 0xffff, w >> 16]
    return torch.tensor([x >= cut for x in numbers[:n]]), 65536 / (65536 - cut)


def layer_norm(h, w, b, eps):
    d = h - h.mean(-1, keepdim=True)
    y = d / ((d * d).mean(-1, keepdim=True) + eps).sqrt()
    y = y if w is None else y * w
    return y if b is None else y + b


def ln_tol(h, w, eps):
    """What y may be off by beside its own rounding, for each row: (..., 1)."""
    d = h - h.mean(-1, keepdim=True)
    r = 1.0 / ((d * d).mean(-1, keepdim=True) + eps).sqrt()
    top = 1.0 if w is None else float(w.abs().max())
    return 2.0 ** -18 * (1.0 + h.abs().amax(-1, keepdim=True) * r) * max(top, 1.0)


def near(got, ref, room, name):
    """|got - ref| <= half a step of got's type * |ref| + room, everywhere."""
    g, r = got.detach().cpu().to(F64), ref.detach().to(F64)
    assert g.shape == r.shape, f"{name}: {tuple(g.shape)} vs {tuple(r.shape)}"
    off, most = (g - r).abs(), torch.finfo(got.dtype).eps / 2 * r.abs() + room
    bad = ~(off <= most)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {r.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                                 f"{float(off[bad][0]):.3e} where {float(most.expand_as(off)[bad][0]):.3e} is allowed")


def meets(d, ref, lens):
    """The size of what dg adds up: the largest sum of |q.dq| and |k.dk| of a token."""
    T = sum(lens)
    return sum(float((ref[a].abs() * d[b][:T].to(F64).abs()).sum(-1).max()) if T else 0.0
               for a, b in (("dq", "q"), ("dk", "k")))


def rms_sum(L: int) -> float:
    """Errors of up to 256 tokens add up in dg, independent of one another."""
    return math.sqrt(min(max(L, 1), 256))
