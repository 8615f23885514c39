"""64-bit definitions of the delta rule and the head norm on the CPU, seeded
inputs for them, and the tolerances of their tests.

Tolerances. A result held in 32 bits is a sum of products, each rounded by at
most 2^-24 of its size. The rule's state map contracts (|k| <= 1, 0 <= beta
<= 1, a <= 1), so an error made at one token is not magnified at later ones:
after L tokens with about Dk + 64 roundings each that are independent of one
another, the rms is below sqrt(L (Dk + 64)) 2^-24 of the largest value, and
four times that is allowed (`tol32`). Gradients are the same recurrence
backwards. A result stored in bf16 is off by at most half a step more, 2^-8
of its value (finfo(bf16).eps / 2).

`out` and `dk` of bf16 inputs add products in which a 32-bit operand stands as
two bf16 parts. A part holds 8 significant bits. Cut, the first leaves less
than 2^-7 of the value and the second less than 2^-7 of that: 2^-14 of the
value at most, and an rms of 2^-14 / 3 < 2^-15.5 where the lower bits are
uniform (each remainder is r u with u uniform in (0, 1), whose rms is
1 / sqrt 3). Rounded to nearest, each is half of that, so both operands of a
product and the product of their second parts, which is left out, add
sqrt 3 2^-17.5 < 2^-16.5. Together the rms is below 2^-15 of a term, hence of
the root of the sum of the squared terms, which is below the largest value
as above; four times that, 2^-13, is allowed (`tol_parts`): 1 / 32 of the
type's own half step.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def tol32(L: int, Dk: int) -> float:
    return 4.0 * math.sqrt(max(L, 1) * (Dk + 64)) * 2.0 ** -24


def tol_parts(name: str, dtype) -> float:
    return 2.0 ** -13 if name in ("out", "dk") and dtype != torch.float32 else 0.0


def half_step(dtype) -> float:
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def check(got, ref, rel, name, scale=None):
    """|got - ref| <= half a step of got's type * |ref| + rel * scale, everywhere;
    scale: the largest |ref| unless given."""
    g, r = got.detach().cpu().to(F64), ref.detach().to(F64)
    assert g.shape == r.shape, f"{name}: {tuple(g.shape)} vs {tuple(r.shape)}"
    if not r.numel():
        return
    top = float(r.abs().max()) if scale is None else scale
    room = half_step(got.dtype) * r.abs() + rel * top
    off = (g - r).abs()
    bad = ~(off <= room)
    assert not bool(bad.any()), (
        f"{name}: {int(bad.sum())} of {r.numel()} off, worst {float(off[bad].max()):.3e} "
        f"(largest value {top:.3e}, allowed {rel:.2e} of it), first at {bad.nonzero()[0].tolist()}")


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)


def rule(q, k, v, g, beta, lens, scale, h0=None):
    """(out, final states) from the definition, token by token; differentiable."""
    Hv, Dk, Dv = v.shape[1], q.shape[2], v.shape[2]
    r = Hv // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    outs, states, t = [], [], 0
    for s, n in enumerate(lens):
        S = torch.zeros(Hv, Dk, Dv, dtype=F64) if h0 is None else h0[s]
        for t in range(t, t + n):
            S = S * g[t].exp()[:, None, None]
            e = v[t] - (S * k[t][:, :, None]).sum(1)
            S = S + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
            outs.append(scale * (S * q[t][:, :, None]).sum(1))
        t = sum(lens[:s + 1])
        states.append(S)
    return torch.stack(outs) if outs else torch.zeros(0, Hv, Dv, dtype=F64), torch.stack(states)


def rule_inputs(seed, lens, Hk, Hv, Dk, Dv, dtype, carry, tail=0):
    """Seeded inputs on the CPU: unit keys that share a direction, decays of
    1e-3 to 1.6, gates in (0, 1). `tail` more rows follow the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    T, n = sum(lens) + tail, len(lens)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()).to(dtype)  # noqa: E731
    d = {"q": unit(rnd(T, Hk, Dk)), "k": unit(rnd(T, Hk, Dk) + 0.5 * rnd(Hk, Dk)), "v": rnd(T, Hv, Dv).to(dtype),
         "g": -torch.exp(rnd(T, Hv) - 3.0), "beta": torch.sigmoid(rnd(T, Hv)), "dout": rnd(T, Hv, Dv).to(dtype),
         "h0": 0.3 * rnd(n, Hv, Dk, Dv) if carry else None, "dhT": 0.3 * rnd(n, Hv, Dk, Dv) if carry else None}
    return d


def rule_reference(d, lens, scale):
    """Outputs and gradients in 64 bits: {"out", "hT", "dq", ..., "dh0"}."""
    T = sum(lens)
    x = {n: d[n][:T].to(F64).requires_grad_() for n in ("q", "k", "v", "g", "beta")}
    h0 = None if d["h0"] is None else d["h0"].to(F64).requires_grad_()
    out, hT = rule(x["q"], x["k"], x["v"], x["g"], x["beta"], lens, scale, h0)
    loss = (out * d["dout"][:T].to(F64)).sum()
    if d["dhT"] is not None:
        loss = loss + (hT * d["dhT"].to(F64)).sum()
    leaves = list(x.values()) + ([] if h0 is None else [h0])
    if loss.requires_grad:
        grads = torch.autograd.grad(loss, leaves, allow_unused=True)
    else:
        grads = [None] * len(leaves)
    grads = [torch.zeros_like(p) if gr is None else gr for gr, p in zip(grads, leaves)]
    res = {"out": out.detach(), "hT": hT.detach()}
    res.update(zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), grads))
    return res


def turn(x, pos, inv_freq, interleaved, sign=1.0):
    """The rotation by its 2 x 2 matrices."""
    if inv_freq is None:
        return x
    rot = 2 * inv_freq.numel()
    a = pos.to(F64)[:, None, None] * inv_freq.to(F64)
    c, s = torch.cos(a), sign * torch.sin(a)
    if interleaved:
        u, w = x[..., :rot:2], x[..., 1:rot:2]
        y = torch.stack([u * c - w * s, u * s + w * c], -1).flatten(-2)
    else:
        u, w = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([u * c - w * s, u * s + w * c], -1)
    return torch.cat([y, x[..., rot:]], -1)


def norm(x, w, pos, inv_freq, l2, eps, interleaved):
    x = x.to(F64)
    m = x.square().sum(-1, keepdim=True) if l2 else x.square().mean(-1, keepdim=True)
    y = x / (m + eps).sqrt()
    return turn(y if w is None else y * w.to(F64), pos, inv_freq, interleaved)
