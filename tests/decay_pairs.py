"""64-bit values of linear attention with a decay by its closed form, a product of
pairs of tokens for each sequence, for packs that the recurrence token by token
(tests/decay_checks.py) takes too long for:
  out_i = scale (e^{G_i} q_i h0 + sum_{j <= i} e^{G_i - G_j} (q_i.k_j) v_j),
  hT = e^{G_L} h0 + sum_j e^{G_L - G_j} k_j v_j^T,   G the running sum of g.
"""
from __future__ import annotations

import torch

from tests import delta_checks as dc

F64 = torch.float64
HEADS = 8  # of them at a time


def reference(d, lens, scale, device="cpu"):
    """As decay_checks.reference, with the gradients of each value head's own
    queries and keys beside them ("dq_heads", "dk_heads": (T, Hv, Dk))."""
    T, Hv = sum(lens), d["v"].shape[1]
    r = Hv // d["q"].shape[1]
    put = lambda t: t.to(device, F64)  # noqa: E731
    x = {n: put(d[n][:T]) for n in ("q", "k", "v", "dout")}
    x["q"], x["k"] = (x[n].repeat_interleave(r, 1) for n in ("q", "k"))
    x["g"] = put(d["g"][:T] if d["g"].dim() == 2 else d["g"])
    Dk, Dv = x["q"].shape[2], x["v"].shape[2]
    n = len(lens)
    x["h0"] = put(d["h0"]) if d["h0"] is not None else torch.zeros(n, Hv, Dk, Dv, dtype=F64, device=device)
    out, hT = torch.zeros_like(x["v"]), torch.zeros_like(x["h0"])
    grads = {name: torch.zeros_like(x[name]) for name in ("q", "k", "v", "g", "h0")}
    t = 0
    for s, L in enumerate(lens):
        rows = slice(t, t + L)
        t += L
        for h in range(0, Hv, HEADS):
            hs = slice(h, min(h + HEADS, Hv))
            part = {name: x[name][rows, hs].transpose(0, 1).contiguous().requires_grad_() for name in ("q", "k", "v")}
            g = (x["g"][rows, hs].t().contiguous() if x["g"].dim() == 2 else x["g"][hs].clone()).requires_grad_()
            h0 = x["h0"][s, hs].clone().requires_grad_()
            G = (g if g.dim() == 2 else g[:, None].expand(-1, L)).cumsum(-1)
            end = G[:, -1:] if L else torch.zeros(g.shape[0], 1, dtype=F64, device=device)
            above = torch.ones(L, L, dtype=torch.bool, device=device).triu(1)
            D = torch.exp((G[:, :, None] - G[:, None, :]).masked_fill(above, float("-inf")))
            o = scale * (torch.exp(G)[..., None] * (part["q"] @ h0)
                         + ((part["q"] @ part["k"].transpose(1, 2).contiguous()) * D) @ part["v"])
            last = torch.exp(end)[..., None] * h0 + (torch.exp(end - G)[..., None] * part["k"]).transpose(1, 2).contiguous() @ part["v"]
            loss = (o * x["dout"][rows, hs].transpose(0, 1)).sum()
            if d["dhT"] is not None:
                loss = loss + (last * put(d["dhT"][s, hs])).sum()
            gq, gk, gv, gg, gh = torch.autograd.grad(loss, [part["q"], part["k"], part["v"], g, h0], allow_unused=True)
            with torch.no_grad():
                out[rows, hs], hT[s, hs] = o.transpose(0, 1), last
                for name, gr in zip(("q", "k", "v"), (gq, gk, gv)):
                    grads[name][rows, hs] = gr.transpose(0, 1)
                grads["h0"][s, hs] = 0.0 if gh is None else gh
                if gg is not None:
                    if g.dim() == 2:
                        grads["g"][rows, hs] = gg.t()
                    else:
                        grads["g"][hs] += gg
    add = lambda t: t.unflatten(1, (Hv // r, r)).sum(2)  # noqa: E731
    res = {"out": out, "hT": hT, "dq": add(grads["q"]), "dk": add(grads["k"]), "dv": grads["v"], "dg": grads["g"],
           "dh0": grads["h0"], "dq_heads": grads["q"], "dk_heads": grads["k"]}
    return {name: t.cpu() for name, t in res.items()}


def meets_of_heads(d, ref):
    """The size of what each head's dg adds up: the largest sum of |q.dq| and |k.dk| of a token, (Hv)."""
    r = d["v"].shape[1] // d["q"].shape[1]
    T = ref["dq_heads"].shape[0]
    return sum((ref[a].abs() * d[b][:T].to(F64).repeat_interleave(r, 1).abs()).sum(-1).amax(0)
               for a, b in (("dq_heads", "q"), ("dk_heads", "k")))


def check_dg(got, ref, meets, rel):
    """dg by token, each head by its own size: what its terms are, or dg itself."""
    for h in range(ref.shape[1]):
        top = max(float(meets[h]), float(ref[:, h].abs().max()) if ref.shape[0] else 0.0)
        dc.check(got[:ref.shape[0], h], ref[:, h], rel, f"dg of head {h}", scale=top)
