"""What is measured of the delta-rule and head-norm operators: cases, inputs, a
plain form in elementary torch operations, and 64-bit values.

Operators (names of the package's entry points):
  gated_delta_pack_fwd / _bwd   gated delta rule over packed sequences
  gated_delta_pack_step         the same for one new token per sequence
  qk_norm_pack_fwd / _bwd       norms of query and key heads, with the position rotation

The rule, per value head with its key head (a_t = exp(g_t)):
  e_t = v_t - (a_t S_{t-1})^T k_t;  S_t = a_t S_{t-1} + beta_t k_t e_t^T;  o_t = scale S_t^T q_t
"""
import math
import random

import numpy as np
import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # serving, one user: a single token of one sequence; latency is all there is
        {"name": "step_1", "op": "step", "B": 1, "pool": 1, "Hk": 16, "Hv": 32, "Dk": 128, "Dv": 128, "dtype": "bf16"},
        # serving, a full batch in a larger pool of states
        {"name": "step_256", "op": "step", "B": 256, "pool": 320, "Hk": 16, "Hv": 32, "Dk": 128, "Dv": 128,
         "dtype": "bf16"},
        # odd head sizes in fp32
        {"name": "step_odd_fp32", "op": "step", "B": 37, "pool": 41, "Hk": 3, "Hv": 6, "Dk": 72, "Dv": 40,
         "dtype": "fp32"},
        # a prompt of one user, its state handed to the steps that follow
        {"name": "fwd_prompt", "op": "fwd", "T": 513, "lengths": "one", "mix": 0, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "dtype": "bf16", "carry": True},
        # 8 packs of 4096 tokens, lengths uniform in [64, 2048], width 4096: evaluation of a packed batch
        {"name": "fwd_8x4096", "op": "fwd", "T": 32768, "lengths": "uniform", "mix": 2, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "dtype": "bf16", "carry": True},
        # the same batch in training: the largest case
        {"name": "train_8x4096", "op": "train", "T": 32768, "lengths": "uniform", "mix": 4, "Hk": 16, "Hv": 32,
         "Dk": 128, "Dv": 128, "dtype": "bf16", "carry": False},
        # long documents at width 1536: few chains, many chunks each, states carried across packs
        {"name": "train_long", "op": "train", "T": 16384, "lengths": "buckets", "mix": 3, "Hk": 12, "Hv": 12,
         "Dk": 128, "Dv": 128, "dtype": "bf16", "carry": True},
        # fp32 training with odd head sizes and many short sequences
        {"name": "train_odd_fp32", "op": "train", "T": 1237, "lengths": "short", "mix": 5, "Hk": 2, "Hv": 6, "Dk": 40,
         "Dv": 72, "dtype": "fp32", "carry": True},
        # the norm of one new token's heads
        {"name": "norm_1", "op": "norm", "T": 1, "mix": 0, "Hq": 16, "Hk": 16, "D": 128, "rot": 0, "inter": False,
         "kind": "l2", "weights": False, "far": 0, "dtype": "bf16"},
        # a packed batch in training, feeding the rule (l2, no rotation)
        {"name": "norm_train_8x4096", "op": "norm_train", "T": 32768, "mix": 2, "Hq": 16, "Hk": 16, "D": 128, "rot": 0,
         "inter": False, "kind": "l2", "weights": False, "far": 0, "dtype": "bf16"},
        # shared key heads, half of each head rotated, positions of documents continued far in
        {"name": "norm_rope_far", "op": "norm", "T": 16384, "mix": 3, "Hq": 32, "Hk": 8, "D": 128, "rot": 64,
         "inter": False, "kind": "rms", "weights": True, "far": 1000000, "dtype": "bf16"},
        # fp32 training, odd sizes, adjacent pairs rotated
        {"name": "norm_train_odd_fp32", "op": "norm_train", "T": 1237, "mix": 5, "Hq": 6, "Hk": 2, "D": 72, "rot": 48,
         "inter": True, "kind": "rms", "weights": True, "far": 0, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head_dim(rng):
    return rng.choice([64, 128, 128, 8 * rng.randint(1, 16)])


def draw(rng):
    op = rng.choice(["step", "fwd", "train", "train", "norm", "norm_train"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op in ("norm", "norm_train"):
        heads = rng.choice([1, 2, 3, 4, 8, 12, 16])
        D = rng.choice([64, 128, 128, 256, 8 * rng.randint(2, 32)])
        c.update(T=_log(rng, 1, 32768), mix=rng.randrange(1 << 20), Hq=heads * rng.choice([1, 2, 4]), Hk=heads, D=D,
                 rot=rng.choice([0, D // 16 * 16, D // 32 * 16]), inter=rng.random() < 0.3,
                 kind=rng.choice(["l2", "rms"]), weights=rng.random() < 0.6, far=rng.choice([0, 0, 100000]))
        while c["T"] * (c["Hq"] + c["Hk"]) * D > 32768 * 32 * 128:
            c["T"] = c["T"] * 2 // 3
        return c
    Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
    c.update(Hk=Hk, Hv=Hk * rng.choice([1, 1, 2, 3]), Dk=_head_dim(rng), Dv=_head_dim(rng))
    if op == "step":
        c["B"] = _log(rng, 1, 256)
        c["pool"] = c["B"] + rng.randint(0, 40)
        return c
    c.update(T=_log(rng, 1, 32768), lengths=rng.choice(["one", "uniform", "buckets", "short"]),
             mix=rng.randrange(1 << 20), carry=rng.random() < 0.5)
    while c["T"] * c["Hv"] > 32768 * (32 if c["dtype"] == "bf16" else 8):
        c["T"] = c["T"] * 2 // 3
    if c["lengths"] == "one":
        c["T"] = min(c["T"], 16384)
    return c


def _lengths(case):
    """Sequence lengths of a packed batch of exactly case["T"] tokens, an empty one among the short."""
    rng, T, kind = random.Random(case["mix"]), case["T"], case["lengths"]
    if kind == "one":
        return [T]
    got, left = [], T
    while left:
        if kind == "uniform":
            n = rng.randint(64, 2048)
        elif kind == "buckets":
            b = rng.choice((512, 1024, 2048, 4096, 8192))
            n = rng.randint(b // 2 + 1, b)
        else:
            n = rng.choice((0, 1, 3, 63, 64, 65, 128, 200, rng.randint(1, 300)))
        n = min(n, left)
        got.append(n)
        left -= n
    return got


# ---------------------------------------------------------------------------
# inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    s = {"case": dict(case)}
    if case["op"] in ("norm", "norm_train"):
        T, Hq, Hk, D, rot = (case[k] for k in ("T", "Hq", "Hk", "D", "rot"))
        s["q"], s["k"] = randn(T, Hq, D).to(dt), randn(T, Hk, D).to(dt)
        s["wq"] = s["wk"] = s["pos"] = s["inv_freq"] = None
        if case["weights"]:
            s["wq"], s["wk"] = 1.0 + 0.2 * randn(D), 1.0 + 0.2 * randn(D)
        if rot:
            # positions inside sequences of the packed batch; a continued document starts far in
            lens = _lengths({"T": T, "mix": case["mix"], "lengths": "uniform"})
            s["pos"] = torch.from_numpy(np.concatenate([np.arange(n) + case["far"] * (i % 3) for i, n in
                                                        enumerate(lens)]).astype(np.int32)).to(dev)
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(dev)
        if case["op"] == "norm_train":
            s["dyq"], s["dyk"] = randn(T, Hq, D).to(dt), randn(T, Hk, D).to(dt)
        return s
    Hk, Hv, Dk, Dv = (case[k] for k in ("Hk", "Hv", "Dk", "Dv"))
    T = case["B"] if case["op"] == "step" else case["T"]

    def unit(x):
        return (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()).to(dt)

    # keys of a head share a direction, as trained ones do
    s["q"], s["k"] = unit(randn(T, Hk, Dk)), unit(randn(T, Hk, Dk) + 0.5 * randn(Hk, Dk))
    s["v"] = randn(T, Hv, Dv).to(dt)
    # log decay -A * step: A in [1, 16] and a step in [1e-3, 0.1] per head, varied by the token
    step = torch.exp(math.log(1e-3) + rand(Hv) * math.log(100.0))
    s["g"] = -(1.0 + 15.0 * rand(Hv)) * torch.nn.functional.softplus(randn(T, Hv) * 0.5 + torch.log(torch.expm1(step)))
    s["beta"] = torch.sigmoid(randn(T, Hv))
    if case["op"] == "step":
        s["state"] = randn(case["pool"], Hv, Dk, Dv) * 0.3
        s["slots"] = torch.randperm(case["pool"], generator=gen, device=dev)[:T].to(torch.int32)
        return s
    lens = _lengths(case)
    s["lengths"] = lens
    s["cu_seqlens"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(dev)
    s["h0"] = randn(len(lens), Hv, Dk, Dv) * 0.3 if case["carry"] else None
    if case["op"] == "train":
        s["dout"] = randn(T, Hv, Dv).to(dt)
        s["dhT"] = randn(len(lens), Hv, Dk, Dv) * 0.3 if case["carry"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own_pass(op, state)
    return {"step": _step, "fwd": _rule, "train": _rule, "norm": _norm, "norm_train": _norm}[op](state)


def _own_pass(op, s):
    import selective_state_space_varlen_amd as ssp
    c = s["case"]
    if op == "step":
        out = ssp.gated_delta_pack_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return {"out": out, "state": s["state"]}
    if op in ("norm", "norm_train"):
        kw = dict(wq=s["wq"], wk=s["wk"], pos=s["pos"], inv_freq=s["inv_freq"], eps=1e-6, interleaved=c["inter"],
                  norm=ssp.SSMP_NORM_L2 if c["kind"] == "l2" else ssp.SSMP_NORM_RMS)
        yq, yk = ssp.qk_norm_pack_fwd(s["q"], s["k"], **kw)
        res = {"yq": yq, "yk": yk}
        if op == "norm_train":
            res.update(ssp.qk_norm_pack_bwd(s["q"], s["k"], s["dyq"], s["dyk"], **kw))
        return {k: v for k, v in res.items() if v is not None}
    out, saved, hT = ssp.gated_delta_pack_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu_seqlens"],
                                              initial_state=s["h0"], final_state=c["carry"], save=op == "train")
    res = {"out": out, "hT": hT}
    if op == "train":
        res.update(ssp.gated_delta_pack_bwd(s["q"], s["k"], s["g"], s["beta"], s["cu_seqlens"], s["dout"], saved,
                                            dfinal_state=s["dhT"], dinitial_state=c["carry"]))
    return {k: v for k, v in res.items() if v is not None}


def work(case):
    elt = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        b = 2 * n * elt + (4 * case["T"] if case["rot"] else 0)
        if case["op"] == "norm":
            return {"bytes": b, "flops": 6 * n}
        return {"bytes": b + 2 * n * elt, "flops": 18 * n}
    Hk, Hv, Dk, Dv = (case[k] for k in ("Hk", "Hv", "Dk", "Dv"))
    T = case["B"] if case["op"] == "step" else case["T"]
    S = Hv * Dk * Dv
    b = T * (2 * Hk * Dk + 2 * Hv * Dv) * elt + T * Hv * 8  # q, k, v, out; g, beta
    if case["op"] == "step":
        return {"bytes": b + T * S * 8, "flops": 6 * T * S}
    n = len(_lengths(case)) if case["carry"] else 0
    b += n * S * 8
    if case["op"] == "fwd":
        return {"bytes": b, "flops": 6 * T * S}
    b += T * (2 * Hk * Dk + 2 * Hv * Dv) * elt + T * Hv * 8 + n * S * 8  # dout, dq, dk, dv; dg, dbeta; states' gradients
    return {"bytes": b, "flops": 20 * T * S}


# ---------------------------------------------------------------------------
# plain form
def _step(s):
    c, dt = s["case"], s["q"].dtype
    r = c["Hv"] // c["Hk"]
    q, k = (s[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    at = s["slots"].long()
    S = s["state"][at] * torch.exp(s["g"])[..., None, None]
    e = s["v"].float() - (S * k[..., None]).sum(-2)
    S = S + k[..., None] * (s["beta"][..., None] * e)[..., None, :]
    s["state"][at] = S
    return {"out": ((S * q[..., None]).sum(-2) * c["Dk"] ** -0.5).to(dt), "state": s["state"]}


def _layout(lens, dev):
    """Rows of the packed batch by chunks of 64 tokens that start anew in each
    sequence (row T stands for padding), and the chunks at each chunk position:
    (chunk numbers, sequence numbers)."""
    T, start, rows, seq, at = sum(lens), 0, [], [], []
    for i, n in enumerate(lens):
        m = -(-n // CHUNK)
        r = np.arange(m * CHUNK)
        rows.append(np.where(r < n, start + r, T))
        seq += [i] * m
        at += range(m)
        start += n
    seq, at = np.array(seq, np.int64), np.array(at, np.int64)
    order = [np.nonzero(at == p)[0] for p in range(int(at.max()) + 1 if len(at) else 0)]
    to = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    return to(np.concatenate(rows)), [(to(o), to(seq[o])) for o in order]


def _chunked(x, rows, heads):
    """(T, H, ...) -> (chunks, heads, 64, ...) in fp32, zeros in padding, heads repeated."""
    x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[rows].float()
    x = x.unflatten(0, (-1, CHUNK)).transpose(1, 2)
    return x.repeat_interleave(heads // x.shape[1], 1)


def _packed(x, rows, T, dt):
    """(chunks, heads, 64, ...) -> (T, heads, ...)."""
    x = x.transpose(1, 2).flatten(0, 1)
    out = x.new_zeros(T + 1, *x.shape[1:])
    out[rows] = x
    return out[:T].to(dt)


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A, row by row."""
    X = -A
    for i in range(1, CHUNK):
        X[..., i, :i] = X[..., i, :i] + (X[..., i, :i, None] * X[..., :i, :i]).sum(-2)
    return X + torch.eye(CHUNK, device=A.device)


def _rule(s):
    """The rule by chunks of 64 tokens: inside a chunk (I + L diag(beta)) E = V - e^G K S, with
    L_ij = exp(G_i - G_j) k_i.k_j below the diagonal and G the running sum of g."""
    c, dt, dev = s["case"], s["q"].dtype, s["q"].device
    T, Hk, Hv, Dk, Dv = (c[n] for n in ("T", "Hk", "Hv", "Dk", "Dv"))
    scale, n = Dk ** -0.5, len(s["lengths"])
    rows, order = _layout(s["lengths"], dev)
    q, k, v = (_chunked(s[x], rows, Hv) for x in ("q", "k", "v"))
    G = _chunked(s["g"], rows, Hv).double().cumsum(-1)
    beta = _chunked(s["beta"], rows, Hv)[..., None]
    i = torch.arange(CHUNK, device=dev)
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(i[:, None] < i, -math.inf)).float()
    eG, eL = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    eC = eG[..., -1:, :]
    L = (D * (k @ k.transpose(-1, -2))).tril(-1)
    P = D * (q @ k.transpose(-1, -2))
    M = _inverse(L * beta.transpose(-1, -2))
    S = torch.zeros(n, Hv, Dk, Dv, device=dev) if s["h0"] is None else s["h0"].clone()
    o, E = torch.empty_like(v), torch.empty_like(v)
    S0 = k.new_empty(k.shape[0], Hv, Dk, Dv) if c["op"] == "train" else None
    for at, seq in order:
        h = S[seq]
        e = M[at] @ (v[at] - eG[at] * (k[at] @ h))
        u = beta[at] * e
        o[at] = scale * (eG[at] * (q[at] @ h) + P[at] @ u)
        S[seq] = eC[at] * h + (eL[at] * k[at]).transpose(-1, -2) @ u
        if S0 is not None:
            S0[at], E[at] = h, e
    res = {"out": _packed(o, rows, T, dt)}
    if c["carry"]:
        res["hT"] = S
    if c["op"] == "fwd":
        return res
    # gradients: dU solves the transposed system, dS runs backwards over the chunks
    do = scale * _chunked(s["dout"], rows, Hv)
    U = beta * E
    M = _inverse(L * beta)
    dS = torch.zeros_like(S) if s["dhT"] is None else s["dhT"].clone()
    dU, dS1 = torch.empty_like(v), torch.empty_like(S0)
    for at, seq in reversed(order):
        h = dS[seq]
        y = P[at].transpose(-1, -2) @ do[at] + eL[at] * (k[at] @ h)
        w = M[at].transpose(-1, -2) @ y
        dS[seq] = eC[at] * h + (eG[at] * q[at]).transpose(-1, -2) @ do[at] - (
            (eG[at] * k[at]).transpose(-1, -2) @ (beta[at] * w))
        dU[at], dS1[at] = w, h
    dE = beta * dU
    a = D * (do @ U.transpose(-1, -2))
    b = (D * (dE @ U.transpose(-1, -2))).tril(-1)
    dq = eG * (do @ S0.transpose(-1, -2)) + a @ k
    dkr = -eG * (dE @ S0.transpose(-1, -2)) - b @ k
    inter = eL * (U @ dS1.transpose(-1, -2))
    dkw = inter + a.transpose(-1, -2) @ q - b.transpose(-1, -2) @ k
    dG = (q * dq + k * dkr - k * dkw).sum(-1).double()
    dG[..., -1] += eC[..., 0, 0] * (dS1 * S0).sum((-1, -2)) + (k * inter).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1).float()
    group = lambda x: x.unflatten(1, (Hk, Hv // Hk)).sum(2)  # noqa: E731
    res.update(dq=_packed(group(dq), rows, T, dt), dk=_packed(group(dkr + dkw), rows, T, dt),
               dv=_packed(dE, rows, T, dt), dg=_packed(dg, rows, T, torch.float32),
               dbeta=_packed((dU * E).sum(-1), rows, T, torch.float32))
    if c["carry"]:
        res["dinitial_state"] = dS
    return res


def _turn(x, cos, sin, rot, inter, back):
    """Rotates the first `rot` components of each head (pairs i, i + rot/2, or adjacent ones)."""
    if not rot:
        return x
    if back:
        sin = -sin
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _norm(s):
    c, dt = s["case"], s["q"].dtype
    cos = sin = None
    if c["rot"]:
        angle = s["pos"].double()[:, None, None] * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    res = {}
    mean = 1.0 / c["D"] if c["kind"] == "rms" else 1.0
    for n in ("q", "k"):
        x = s[n].float()
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) * mean + 1e-6)
        w = 1.0 if s["w" + n] is None else s["w" + n]
        res["y" + n] = _turn(x * r * w, cos, sin, c["rot"], c["inter"], False).to(dt)
        if c["op"] == "norm_train":
            h = _turn(s["dy" + n].float(), cos, sin, c["rot"], c["inter"], True)
            xr = x * r
            if s["w" + n] is not None:
                res["dw" + n] = (h * xr).double().sum((0, 1)).float()
            h = h * w
            res["d" + n] = (r * (h - xr * ((h * xr).sum(-1, keepdim=True) * mean))).to(dt)
    return res


# ---------------------------------------------------------------------------
# 64-bit values, token by token from the definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "fwd": _exact_rule, "train": _exact_rule, "norm": _exact_norm,
            "norm_train": _exact_norm}[case["op"]](s, case)


def _exact_step(s, c):
    heads = torch.arange(c["Hv"], device=s["q"].device) // (c["Hv"] // c["Hk"])
    state = s["state"].double()
    at = s["slots"].long()
    q, k, v = s["q"].double()[:, heads], s["k"].double()[:, heads], s["v"].double()
    S = state[at] * s["g"].double().exp()[:, :, None, None]
    e = v - torch.einsum("bhij,bhi->bhj", S, k)
    S = S + torch.einsum("bhi,bhj->bhij", k, e * s["beta"].double()[:, :, None])
    state[at] = S
    return {"out": torch.einsum("bhij,bhi->bhj", S, q) / math.sqrt(c["Dk"]), "state": state}


def _exact_rule(s, c):
    dev, lens = s["q"].device, s["lengths"]
    Hv, Dk, Dv, N, T = c["Hv"], c["Dk"], c["Dv"], len(lens), c["T"]
    heads = torch.arange(Hv, device=dev) // (Hv // c["Hk"])
    scale = 1.0 / math.sqrt(Dk)
    q, k, v = s["q"].double()[:, heads], s["k"].double()[:, heads], s["v"].double()
    a, beta = s["g"].double().exp(), s["beta"].double()
    # longest first: at token t the first active[t] sequences still run
    rank = sorted(range(N), key=lambda i: -lens[i])
    starts = np.concatenate([[0], np.cumsum(lens)])
    longest = max(lens) if lens else 0
    active = [sum(n > t for n in lens) for t in range(longest)]
    first = torch.tensor([int(starts[i]) for i in rank], device=dev)
    S = torch.zeros(N, Hv, Dk, Dv, dtype=torch.float64, device=dev)
    if s["h0"] is not None:
        S += s["h0"].double()[rank]
    o = torch.zeros(T, Hv, Dv, dtype=torch.float64, device=dev)
    mul = lambda x, M: (x[:, :, None, :] @ M)[:, :, 0]  # noqa: E731  x^T M
    vec = lambda M, x: (M @ x[..., None])[..., 0]  # noqa: E731

    def advance(S, t):
        m, at = active[t], first[:active[t]] + t
        aS = S[:m] * a[at][:, :, None, None]
        e = v[at] - mul(k[at], aS)
        return m, at, aS, e, aS + k[at][..., None] * (beta[at][..., None] * e)[:, :, None, :]

    B = 32
    marks = []
    for t in range(longest):
        if c["op"] == "train" and t % B == 0:
            marks.append(S[:active[t]].clone())
        m, at, _, _, new = advance(S, t)
        S[:m] = new
        o[at] = scale * mul(q[at], new)
    back = torch.empty(N, dtype=torch.long, device=dev)
    back[torch.tensor(rank, dtype=torch.long, device=dev)] = torch.arange(N, device=dev)
    res = {"out": o}
    if c["carry"]:
        res["hT"] = S[back]
    if c["op"] == "fwd":
        return res
    dS = torch.zeros_like(S)
    if s["dhT"] is not None:
        dS += s["dhT"].double()[rank]
    do = s["dout"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(a), torch.zeros_like(a)
    for b in reversed(range(len(marks))):
        S, kept = marks[b], []
        for t in range(b * B, min(longest, (b + 1) * B)):
            kept.append(advance(S, t))
            S = kept[-1][4]
        for t in reversed(range(b * B, min(longest, (b + 1) * B))):
            m, at, aS, e, new = kept.pop()
            d = dS[:m] + scale * q[at][..., None] * do[at][:, :, None, :]
            dq[at] = scale * vec(new, do[at])
            du = mul(k[at], d)
            dk[at] = vec(d, beta[at][..., None] * e)
            de = beta[at][..., None] * du
            dv[at], dbeta[at] = de, (du * e).sum(-1)
            dk[at] -= vec(aS, de)
            d = d - k[at][..., None] * de[:, :, None, :]
            dg[at] = (d * aS).sum((-1, -2))
            dS[:m] = d * a[at][:, :, None, None]
    total = lambda x: torch.stack([x[:, heads == h].sum(1) for h in range(c["Hk"])], 1)  # noqa: E731
    res.update(dq=total(dq), dk=total(dk), dv=dv, dg=dg, dbeta=dbeta)
    if c["carry"]:
        res["dinitial_state"] = dS[back]
    return res


def _exact_norm(s, c):
    """The rotation as a product of complex numbers; gradients by the chain rule written out."""
    D, rot = c["D"], c["rot"]
    res = {}
    pick = torch.arange(rot, device=s["q"].device)
    if rot:
        pick = pick.view(-1, 2).t().reshape(-1) if c["inter"] else pick  # first members of the pairs, then second ones
        unit = torch.polar(torch.ones((), dtype=torch.float64, device=pick.device),
                           s["pos"].double()[:, None] * s["inv_freq"].double())[:, None]

    def spin(x, by):
        y = x.clone()
        if rot:
            z = x[..., pick]
            z = torch.complex(z[..., :rot // 2], z[..., rot // 2:]) * by
            y[..., pick] = torch.cat([z.real, z.imag], -1)
        return y

    for n in ("q", "k"):
        x = s[n].double()
        size = x.square().mean(-1, keepdim=True) if c["kind"] == "rms" else x.square().sum(-1, keepdim=True)
        root = (size + 1e-6).sqrt()
        w = torch.ones(D, dtype=torch.float64, device=x.device) if s["w" + n] is None else s["w" + n].double()
        res["y" + n] = spin(x / root * w, unit if rot else None)
        if c["op"] == "norm_train":
            h = spin(s["dy" + n].double(), unit.conj() if rot else None)
            if s["w" + n] is not None:
                res["dw" + n] = torch.einsum("thd,thd->d", h, x / root)
            h = h * w
            inner = (h * x).sum(-1, keepdim=True) / (D if c["kind"] == "rms" else 1)
            res["d" + n] = h / root - x * inner / root ** 3
    return res
