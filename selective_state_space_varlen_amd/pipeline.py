"""The sequence-wise part of one block on a packed batch, as a chain of library
calls (no arithmetic here). A Mamba-1 block:

  forward:  varlen_pack_indices -> conv1d_pack_fwd (SiLU) -> selective_scan_pack_fwd
  backward: selective_scan_pack_bwd -> conv1d_pack_bwd

A gated delta rule block (delta_forward, delta_backward), whose queries, keys
and values each pass a conv and whose query and key heads are normalised:

  forward:  varlen_pack_indices -> conv1d_pack_fwd (SiLU, three) -> qk_norm_pack_fwd -> gated_delta_pack_fwd
  backward: gated_delta_pack_bwd -> qk_norm_pack_bwd -> conv1d_pack_bwd (three)

A block of linear attention with a decay (decay_forward, decay_backward), of
which every part but the attention may be left out:

  forward:  conv1d_pack_fwd (SiLU, three) -> qk_norm_pack_fwd -> decay_attn_pack_fwd -> layer_norm_pack_fwd
            (of the heads) -> dropout_pack_fwd
  backward: the same back

Shanghai AI Lab article on packed variable-length Mamba-1 training
(gitcode.csdn.net/69d8cc1b54b52172bc6872cb.html), section "Mamba block中的步骤":
conv1d and the SSM are the block's two sequence-wise steps; the conv feeds
the scan through SiLU (Mamba-1's block order).
"""
from __future__ import annotations

import functools
from typing import Optional

import torch

from . import binding as _b


def forward(x: torch.Tensor, w: torch.Tensor, b: Optional[torch.Tensor], delta: torch.Tensor, A: torch.Tensor,
            B: torch.Tensor, C: torch.Tensor, Dskip: Optional[torch.Tensor], z: Optional[torch.Tensor],
            cu_seqlens: torch.Tensor, pos: Optional[torch.Tensor] = None, ws: Optional[dict] = None,
            initial_states: Optional[dict] = None, final_states: bool = False,
            delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
            gate_floor: float = 0.0) -> dict:
    """Returns {'pos', 'u', 'out', 'scan_ws', 'step_map'}; keep it for backward.

    delta_bias / delta_softplus / gate_floor: the scan's step is
    softplus(delta + bias) (or delta + bias) and its gate SiLU(z) + gate_floor;
    the backward takes them from the returned dict and adds 'ddelta_bias'.

    Sequences continued from an earlier pack (the article's section
    "结论与讨论": a sequence cut at a pack end keeps passing state) take
    initial_states = {'ssm': (nseq, D, N) fp32, 'conv': (nseq, W-1, D)} (either
    may be None: zeros); with final_states=True, or with initial states, the
    result also holds 'final_states' in the same form."""
    T = x.shape[0]
    if pos is None:
        pos, _, _ = _b.varlen_pack_indices(cu_seqlens, T, heads=False, dev_err=False)
    carry = initial_states is not None or final_states
    sm = {"delta_bias": delta_bias, "delta_softplus": delta_softplus, "gate_floor": gate_floor}
    res = {"pos": pos, "step_map": sm}
    if carry:
        st = initial_states or {}
        u, cf = _b.conv1d_pack_fwd(x, w, b, pos, silu=True, out=None if ws is None else ws.get("u"),
                                   cu_seqlens=cu_seqlens, conv_initial=st.get("conv"), conv_final=True)
        out, scan_ws, hT = _b.selective_scan_pack_fwd(u, delta, A, B, C, Dskip, z, pos,
                                                      workspace=None if ws is None else ws.get("scan"),
                                                      out=None if ws is None else ws.get("out"),
                                                      cu_seqlens=cu_seqlens, initial_state=st.get("ssm"),
                                                      final_state=True, **sm)
        res.update({"final_states": {"ssm": hT, "conv": cf}, "cu_seqlens": cu_seqlens, "initial_states": st})
    else:
        u = _b.conv1d_pack_fwd(x, w, b, pos, silu=True, out=None if ws is None else ws.get("u"))
        out, scan_ws = _b.selective_scan_pack_fwd(u, delta, A, B, C, Dskip, z, pos,
                                                  workspace=None if ws is None else ws.get("scan"),
                                                  out=None if ws is None else ws.get("out"), **sm)
    res.update({"u": u, "out": out, "scan_ws": scan_ws})
    return res


def backward(x: torch.Tensor, w: torch.Tensor, b: Optional[torch.Tensor], delta: torch.Tensor, A: torch.Tensor,
             B: torch.Tensor, C: torch.Tensor, Dskip: Optional[torch.Tensor], z: Optional[torch.Tensor],
             fwd: dict, dout: torch.Tensor, conv_ws: Optional[torch.Tensor] = None,
             dfinal_states: Optional[dict] = None) -> dict:
    """Gradients of sum(dout * out) (+ sum(dfinal * final) for carried states)
    for x, w, b, delta, A, B, C, Dskip, z. When the forward carried states, the
    result also holds 'dinitial_states' {'ssm', 'conv'}, the gradients to hand
    to the earlier pack's backward as its dfinal_states. With a step bias in
    the forward, the result also holds 'ddelta_bias'."""
    sm = fwd.get("step_map", {})
    if "cu_seqlens" not in fwd:
        g = _b.selective_scan_pack_bwd(fwd["u"], delta, A, B, C, Dskip, z, fwd["pos"], dout, fwd["scan_ws"], **sm)
        dx, dw, db = _b.conv1d_pack_bwd(x, w, b, fwd["pos"], g["du"], silu=True, workspace=conv_ws,
                                        want_db=b is not None)
        g.update({"dx": dx, "dw": dw, "db": db})
        return g
    cu, st, dfs = fwd["cu_seqlens"], fwd["initial_states"], dfinal_states or {}
    g = _b.selective_scan_pack_bwd(fwd["u"], delta, A, B, C, Dskip, z, fwd["pos"], dout, fwd["scan_ws"],
                                   cu_seqlens=cu, initial_state=st.get("ssm"), dfinal_state=dfs.get("ssm"),
                                   dinitial_state=True, **sm)
    dx, dw, db, dci = _b.conv1d_pack_bwd(x, w, b, fwd["pos"], g["du"], silu=True, workspace=conv_ws,
                                         want_db=b is not None, cu_seqlens=cu, conv_initial=st.get("conv"),
                                         dconv_final=dfs.get("conv"), dconv_initial=True)
    g.update({"dx": dx, "dw": dw, "db": db, "dinitial_states": {"ssm": g.pop("dinitial_state"), "conv": dci}})
    return g


def _on_its_device(f):
    """f with the device of its first argument's first tensor current, as the convs' launches need it to be."""
    @functools.wraps(f)
    def on_device(x, *args, **kw):
        with torch.cuda.device_of(x[0]):
            return f(x, *args, **kw)
    return on_device


@_on_its_device
def delta_forward(x: tuple, w: tuple, b: Optional[tuple], g: torch.Tensor, beta: torch.Tensor,
                  cu_seqlens: torch.Tensor, Hk: int, Hv: int, pos: Optional[torch.Tensor] = None,
                  scale: Optional[float] = None, norm: int = _b.SSMP_NORM_L2, eps: float = 1e-6,
                  norm_weights: tuple = (None, None), inv_freq: Optional[torch.Tensor] = None,
                  initial_states: Optional[dict] = None, final_states: bool = False, save: bool = True,
                  interleaved: bool = False) -> dict:
    """x = (xq (T, Hk * Dk), xk (T, Hk * Dk), xv (T, Hv * Dv)) with conv weights w
    and biases b (None, or a tuple) in the same order; g, beta fp32 (T, Hv).
    Returns {'out' (T, Hv, Dv), ...}; keep it for delta_backward (save=True).

    norm, eps, norm_weights (of the query and the key heads, either None),
    inv_freq and interleaved go to qk_norm_pack_fwd, with pos (default: the
    positions inside the pack's sequences) where inv_freq turns the heads.

    Sequences continued from an earlier pack take initial_states = {'delta':
    (nseq, Hv, Dk, Dv) fp32, 'conv': three contexts (nseq, W-1, .)} (either may
    be None: zeros); with final_states=True, or with initial states, the result
    also holds 'final_states' in the same form. pos then still counts inside
    the pack; a rotation (inv_freq) that goes on is given its own pos.

    cu_seqlens ends at T: the convs and norms go over every row, and sum their
    weights' gradients over every row."""
    T = x[0].shape[0]
    starts, _, _ = _b.varlen_pack_indices(cu_seqlens, T, heads=False, dev_err=False)
    carry = initial_states is not None or final_states
    st = initial_states or {}
    u, cf = [], []
    for i in range(3):
        bias = None if b is None else b[i]
        if carry:
            ctx = st.get("conv")
            y, f = _b.conv1d_pack_fwd(x[i], w[i], bias, starts, silu=True, cu_seqlens=cu_seqlens,
                                      conv_initial=None if ctx is None else ctx[i], conv_final=True)
            cf.append(f)
        else:
            y = _b.conv1d_pack_fwd(x[i], w[i], bias, starts, silu=True)
        u.append(y)
    q, k, v = (u[i].view(T, n, u[i].shape[1] // n) for i, n in enumerate((Hk, Hk, Hv)))
    nk = dict(wq=norm_weights[0], wk=norm_weights[1], pos=starts if pos is None else pos, inv_freq=inv_freq,
              norm=norm, eps=eps, interleaved=interleaved)
    qn, kn = _b.qk_norm_pack_fwd(q, k, **nk)
    out, saved, hT = _b.gated_delta_pack_fwd(qn, kn, v, g, beta, cu_seqlens, scale=scale,
                                             initial_state=st.get("delta"), final_state=carry, save=save)
    res = {"out": out, "starts": starts, "q": q, "k": k, "qn": qn, "kn": kn, "saved": saved, "norm": nk,
           "scale": scale, "cu_seqlens": cu_seqlens, "carry": carry, "initial_states": st}
    if carry:
        res["final_states"] = {"delta": hT, "conv": tuple(cf)}
    return res


@_on_its_device
def delta_backward(x: tuple, w: tuple, b: Optional[tuple], g: torch.Tensor, beta: torch.Tensor, fwd: dict,
                   dout: torch.Tensor, dfinal_states: Optional[dict] = None) -> dict:
    """Gradients of sum(dout * out) (+ sum(dfinal * final) for carried states):
    'dx', 'dw', 'db' (tuples in the order q, k, v; db None without biases),
    'dg', 'dbeta', 'dwq', 'dwk' (the norm weights'), and with carried states
    'dinitial_states', to hand to the earlier pack's backward. dfinal_states
    is refused where the forward gave no final states."""
    cu, carry, st, dfs = fwd["cu_seqlens"], fwd["carry"], fwd["initial_states"], dfinal_states or {}
    if not carry and any(t is not None for t in dfs.values()):
        raise ValueError("dfinal_states: the forward gave no final states (initial_states, or final_states=True)")
    G = _b.gated_delta_pack_bwd(fwd["qn"], fwd["kn"], g, beta, cu, dout, fwd["saved"], scale=fwd["scale"],
                                dfinal_state=dfs.get("delta"), dinitial_state=carry)
    N = _b.qk_norm_pack_bwd(fwd["q"], fwd["k"], G["dq"], G["dk"], **fwd["norm"])
    dx, dw, db, dci = [], [], [], []
    for i, du in enumerate((N["dq"], N["dk"], G["dv"])):
        bias = None if b is None else b[i]
        ctx, dctx = st.get("conv"), dfs.get("conv")
        kw = dict(cu_seqlens=cu, conv_initial=None if ctx is None else ctx[i],
                  dconv_final=None if dctx is None else dctx[i], dconv_initial=True) if carry else {}
        r = _b.conv1d_pack_bwd(x[i], w[i], bias, fwd["starts"], du.view(x[i].shape), silu=True,
                               want_db=bias is not None, **kw)
        for to, t in zip((dx, dw, db, dci), r):
            to.append(t)
    res = {"dx": tuple(dx), "dw": tuple(dw), "db": None if b is None else tuple(db), "dg": G["dg"],
           "dbeta": G["dbeta"], "dwq": N["dwq"], "dwk": N["dwk"]}
    if carry:
        res["dinitial_states"] = {"delta": G["dinitial_state"], "conv": tuple(dci)}
    return res


@_on_its_device
def decay_forward(x: tuple, g: torch.Tensor, cu_seqlens: torch.Tensor, Hk: int, Hv: int, w: Optional[tuple] = None,
                  b: Optional[tuple] = None, pos: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  norm: Optional[int] = None, eps: float = 1e-6, norm_weights: tuple = (None, None),
                  inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
                  out_norm: Optional[tuple] = None, out_eps: float = 1e-5, p: float = 0.0,
                  rng: Optional[torch.Tensor] = None, initial_states: Optional[dict] = None,
                  final_states: bool = False) -> dict:
    """x = (xq (T, Hk * Dk), xk (T, Hk * Dk), xv (T, Hv * Dv)); g fp32 (T, Hv), or
    (Hv) for one decay a head. Returns {'out' (T, Hv, Dv), ...}; keep it for
    decay_backward.

    w, b: conv weights and biases (b None, or a tuple) in the order of x; None:
    no convs. norm (SSMP_NORM_*; None: none), eps, norm_weights, inv_freq and
    interleaved go to qk_norm_pack_fwd, with pos (default: the positions inside
    the pack's sequences) where inv_freq turns the heads. out_norm = (weight,
    bias) fp32 (Hv, Dv), either None: the layer norm of each head of the result,
    with out_eps; None: none. p, rng: dropout of what is returned.

    Sequences continued from an earlier pack take initial_states = {'decay':
    (nseq, Hv, Dk, Dv) fp32, 'conv': three contexts (nseq, W-1, .)} (either may
    be None: zeros; without w there is no 'conv'); with final_states=True, or
    with initial states, the result also holds 'final_states' in the same form.
    pos then still counts inside the pack; a rotation that goes on is given its
    own pos.

    cu_seqlens ends at T: the convs and norms go over every row, and sum their
    weights' gradients over every row."""
    T = x[0].shape[0]
    if inv_freq is not None and norm is None:
        raise ValueError("the rotation (inv_freq) is done by the heads' norm")
    carry = initial_states is not None or final_states
    st = initial_states or {}
    if w is None and st.get("conv") is not None:
        raise ValueError("initial_states: conv contexts without convs (w)")
    starts, u, cf = None, list(x), []
    if w is not None or (inv_freq is not None and pos is None):
        starts, _, _ = _b.varlen_pack_indices(cu_seqlens, T, heads=False, dev_err=False)
    if w is not None:
        for i in range(3):
            bias, ctx = None if b is None else b[i], st.get("conv")
            kw = dict(cu_seqlens=cu_seqlens, conv_initial=None if ctx is None else ctx[i],
                      conv_final=True) if carry else {}
            u[i] = _b.conv1d_pack_fwd(x[i], w[i], bias, starts, silu=True, **kw)
            if carry:
                u[i], f = u[i]
                cf.append(f)
    q, k, v = (u[i].view(T, n, u[i].shape[1] // n) for i, n in enumerate((Hk, Hk, Hv)))
    qn, kn, nk = q, k, None
    if norm is not None:
        nk = dict(wq=norm_weights[0], wk=norm_weights[1], pos=starts if pos is None else pos, inv_freq=inv_freq,
                  norm=norm, eps=eps, interleaved=interleaved)
        qn, kn = _b.qk_norm_pack_fwd(q, k, **nk)
    o, hT = _b.decay_attn_pack_fwd(qn, kn, v, g, cu_seqlens, scale=scale, initial_state=st.get("decay"),
                                   final_state=carry)
    out = o
    if out_norm is not None:
        out, _ = _b.layer_norm_pack_fwd(out, *out_norm, eps=out_eps)
    if p:
        out = _b.dropout_pack_fwd(out, p, rng, out=out if out is not o else None)
    res = {"out": out, "starts": starts, "q": q, "k": k, "v": v, "qn": qn, "kn": kn, "attn": o, "norm": nk,
           "scale": scale, "out_norm": out_norm, "out_eps": out_eps, "dropout": (p, rng), "cu_seqlens": cu_seqlens,
           "carry": carry, "initial_states": st, "convs": (w, b)}
    if carry:
        res["final_states"] = {"decay": hT, "conv": tuple(cf) if cf else None}
    return res


@_on_its_device
def decay_backward(x: tuple, g: torch.Tensor, fwd: dict, dout: torch.Tensor, dfinal_states: Optional[dict] = None,
                   want_dg: bool = True) -> dict:
    """Gradients of sum(dout * out) (+ sum(dfinal * final) for carried states):
    'dx' and, with convs, 'dw', 'db' (tuples in the order q, k, v; None
    without), 'dg' (None with want_dg=False), 'dwq', 'dwk' (the norm weights'),
    'dout_norm' (those of out_norm's weight and bias, None where there is none),
    and with carried states 'dinitial_states', to hand to the earlier pack's
    backward. rng has to hold what it held in the forward. dfinal_states is
    refused where the forward gave no final states."""
    cu, carry, st, dfs = fwd["cu_seqlens"], fwd["carry"], fwd["initial_states"], dfinal_states or {}
    w, b = fwd["convs"]
    if not carry and any(t is not None for t in dfs.values()):
        raise ValueError("dfinal_states: the forward gave no final states (initial_states, or final_states=True)")
    if w is None and dfs.get("conv") is not None:
        raise ValueError("dfinal_states: conv contexts without convs")
    p, rng = fwd["dropout"]
    if p:
        dout = _b.dropout_pack_bwd(dout, p, rng)
    don = (None, None)
    if fwd["out_norm"] is not None:
        ow, ob = fwd["out_norm"]
        r = _b.layer_norm_pack_bwd(dout, fwd["attn"], ow, eps=fwd["out_eps"], bias=ob is not None)
        dout, don = r["dx"], (r["dw"], r["db"])
    G = _b.decay_attn_pack_bwd(fwd["qn"], fwd["kn"], fwd["v"], g, cu, dout, scale=fwd["scale"],
                               initial_state=st.get("decay"), dfinal_state=dfs.get("decay"), dinitial_state=carry,
                               want_dg=want_dg)
    dq, dk, dwq, dwk = G["dq"], G["dk"], None, None
    if fwd["norm"] is not None:
        N = _b.qk_norm_pack_bwd(fwd["q"], fwd["k"], dq, dk, **fwd["norm"])
        dq, dk, dwq, dwk = (N[n] for n in ("dq", "dk", "dwq", "dwk"))
    du = [t.view(y.shape) for t, y in zip((dq, dk, G["dv"]), x)]
    dw, db, dci = [], [], []
    if w is not None:
        for i in range(3):
            bias, ctx, dctx = None if b is None else b[i], st.get("conv"), dfs.get("conv")
            kw = dict(cu_seqlens=cu, conv_initial=None if ctx is None else ctx[i],
                      dconv_final=None if dctx is None else dctx[i], dconv_initial=True) if carry else {}
            r = _b.conv1d_pack_bwd(x[i], w[i], bias, fwd["starts"], du[i], silu=True, want_db=bias is not None, **kw)
            du[i] = r[0]
            for to, t in zip((dw, db, dci), r[1:]):
                to.append(t)
    res = {"dx": tuple(du), "dw": tuple(dw) if dw else None, "db": tuple(db) if w is not None and b is not None else None,
           "dg": G["dg"], "dwq": dwq, "dwk": dwk, "dout_norm": don}
    if carry:
        res["dinitial_states"] = {"decay": G["dinitial_state"], "conv": tuple(dci) if dci else None}
    return res
