"""What is measured of linear attention with a decay for each head, of the
layer norm and of dropout: cases, inputs, a plain form in elementary torch
operations, and 64-bit values.

Operators (names of the package's entry points):
  decay_attn_pack_fwd / _bwd   linear attention with a decay over packed sequences
  decay_attn_pack_step         the same for one new token per sequence
  layer_norm_pack_fwd / _bwd   layer norm of rows or heads, with the residual sum and dropout before it
  dropout_pack_fwd / _bwd      dropout from a counter, with the residual sum

Attention, per value head with its key head (a_t = exp(g_t), g by token or one for a head):
  S_t = a_t S_{t-1} + k_t v_t^T;  o_t = scale S_t^T q_t
Layer norm, over a row's D components:
  h = residual + drop(x);  y = (h - mean) (var + eps)^(-1/2) w + b
Dropout with rng = (seed, stream): element e is kept where the 16-bit number e % 8 of
Philox4x32-10 with key `seed` and counter (e / 8, stream) is at least c = round(65536 p);
what is kept is divided by 1 - c / 65536.
"""
import math
import random

import numpy as np
import torch

own = False

CHUNK = 64
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # serving, one user: a single token of one sequence; latency is all there is
        {"name": "step_1", "op": "step", "B": 1, "pool": 1, "Hk": 32, "Hv": 32, "Dk": 128, "Dv": 128, "per_token": True,
         "dtype": "bf16"},
        # serving, a full batch in a larger pool of states, a fixed decay for each head
        {"name": "step_256", "op": "step", "B": 256, "pool": 320, "Hk": 16, "Hv": 32, "Dk": 128, "Dv": 128,
         "per_token": False, "dtype": "bf16"},
        # a prompt of one user, its state handed to the steps that follow
        {"name": "fwd_prompt", "op": "fwd", "T": 513, "lengths": "one", "mix": 0, "Hk": 32, "Hv": 32, "Dk": 128,
         "Dv": 128, "per_token": True, "carry": True, "dtype": "bf16"},
        # 8 packs of 4096 tokens, lengths uniform in [64, 2048], width 4096: evaluation of a packed batch
        {"name": "fwd_8x4096", "op": "fwd", "T": 32768, "lengths": "uniform", "mix": 2, "Hk": 16, "Hv": 32, "Dk": 128,
         "Dv": 128, "per_token": True, "carry": True, "dtype": "bf16"},
        # such a batch in training, a key head for every value head: the largest case
        {"name": "train_8x4096", "op": "train", "T": 32768, "lengths": "uniform", "mix": 4, "Hk": 32, "Hv": 32,
         "Dk": 128, "Dv": 128, "per_token": True, "carry": False, "dtype": "bf16"},
        # long documents at width 1536, one key head for all value heads, states carried across packs
        {"name": "train_long", "op": "train", "T": 16384, "lengths": "buckets", "mix": 3, "Hk": 1, "Hv": 24, "Dk": 128,
         "Dv": 64, "per_token": True, "carry": True, "dtype": "bf16"},
        # fp32 training with odd head sizes, many short sequences and one decay for a head
        {"name": "train_odd_fp32", "op": "train", "T": 1237, "lengths": "short", "mix": 5, "Hk": 2, "Hv": 6, "Dk": 40,
         "Dv": 72, "per_token": False, "carry": True, "dtype": "fp32"},
        # the norm of one new token on its way through a block
        {"name": "ln_1", "op": "ln", "T": 1, "H": 0, "D": 4096, "residual": True, "p": 0.0, "affine": True,
         "dtype": "bf16"},
        # between two blocks in training: dropout of the block's result, the residual sum and its norm, both ways
        {"name": "ln_train_8x4096", "op": "ln_train", "T": 32768, "H": 0, "D": 4096, "residual": True, "p": 0.1,
         "affine": True, "dtype": "bf16"},
        # the heads of a short fp32 batch after the attention, each with weights of its own
        {"name": "ln_heads_fp32", "op": "ln_train", "T": 1237, "H": 6, "D": 72, "residual": False, "p": 0.0,
         "affine": True, "dtype": "fp32"},
        # dropout of a block's result with the residual sum, and its gradient
        {"name": "drop_8x4096", "op": "drop", "T": 32768, "D": 4096, "p": 0.1, "residual": True, "dtype": "bf16"},
        # a few rows of an odd size
        {"name": "drop_odd_fp32", "op": "drop", "T": 77, "D": 1537, "p": 0.35, "residual": False, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _head_dim(rng):
    return rng.choice([64, 128, 128, 8 * rng.randint(1, 16)])


def draw(rng):
    op = rng.choice(["step", "fwd", "train", "train", "ln", "ln_train", "drop"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op in ("ln", "ln_train", "drop"):
        c.update(T=_log(rng, 1, 32768), residual=rng.random() < 0.5,
                 p=rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.9), 3)]))
        if op == "drop":
            c.update(D=rng.choice([64, 1536, 4096, _log(rng, 1, 8192)]), p=c["p"] or 0.2)
        else:
            heads = rng.random() < 0.4
            c.update(H=rng.choice([1, 2, 3, 6, 12, 24, 32]) if heads else 0, affine=rng.random() < 0.8,
                     D=rng.choice([64, 128, 256, rng.randint(2, 256)]) if heads else
                     rng.choice([1536, 4096, _log(rng, 2, 8192)]))
        while c["T"] * max(c.get("H", 1), 1) * c["D"] > 32768 * 4096:
            c["T"] = c["T"] * 2 // 3
        return c
    Hk = rng.choice([1, 1, 2, 3, 4, 8, 12, 16])
    c.update(Hk=Hk, Hv=Hk * rng.choice([1, 1, 2, 3]) if Hk > 1 else rng.choice([1, 4, 12, 24]), Dk=_head_dim(rng),
             Dv=_head_dim(rng) if rng.random() < 0.8 else rng.choice([136, 192, 256]))
    c["per_token"] = c["Hv"] == 1 or rng.random() < 0.6  # fixed decays come as one for each of several heads
    if op == "step":
        c["B"] = _log(rng, 1, 256)
        c["pool"] = c["B"] + rng.randint(0, 40)
        return c
    c.update(T=_log(rng, 1, 32768), lengths=rng.choice(["one", "uniform", "buckets", "short"]),
             mix=rng.randrange(1 << 20), carry=rng.random() < 0.5)
    while c["T"] * c["Hv"] * max(c["Dv"], 64) > 32768 * 128 * (32 if c["dtype"] == "bf16" else 8):
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
    if case["op"] in ("ln", "ln_train", "drop"):
        T, D, H = case["T"], case["D"], case.get("H", 0)
        row = (H, D) if H else (D,)
        # rows whose mean and spread differ, as the residual stream's do
        s["x"] = (randn(T, *row) * (0.5 + rand(T, *[1] * len(row))) + 0.3 * randn(T, *[1] * len(row))).to(dt)
        s["residual"] = randn(T, *row).to(dt) if case["residual"] else None
        s["rng"] = torch.tensor([seed * 7919 + 13, seed + 1], dtype=torch.int64, device=dev) if case["p"] else None
        if case["op"] == "drop":
            s["dy"] = randn(T, D).to(dt)
            return s
        s["w"] = 1.0 + 0.2 * randn(*row) if case["affine"] else None
        s["b"] = 0.2 * randn(*row) if case["affine"] else None
        if case["op"] == "ln_train":
            s["dy"] = randn(T, *row).to(dt)
            # what the backward reads beside its gradient: the sum as the forward stored it, and the
            # gradient that reaches the sum past the norm
            if case["residual"] or case["p"]:
                s["h"], s["dh"] = (randn(T, *row) + 0.5 * randn(T, *[1] * len(row))).to(dt), randn(T, *row).to(dt)
            else:
                s["h"], s["dh"] = s["x"], None
        return s
    Hk, Hv, Dk, Dv = (case[k] for k in ("Hk", "Hv", "Dk", "Dv"))
    T = case["B"] if case["op"] == "step" else case["T"]

    def unit(x):
        return (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()).to(dt)

    # keys of a head share a direction, as trained ones do
    s["q"], s["k"] = unit(randn(T, Hk, Dk)), unit(randn(T, Hk, Dk) + 0.5 * randn(Hk, Dk))
    s["v"] = randn(T, Hv, Dv).to(dt)
    if case["per_token"]:
        # log decay -A * step: A in [1, 16] and a step in [1e-3, 0.1] per head, varied by the token
        step = torch.exp(math.log(1e-3) + rand(Hv) * math.log(100.0))
        s["g"] = -(1.0 + 15.0 * rand(Hv)) * torch.nn.functional.softplus(randn(T, Hv) * 0.5 + torch.log(torch.expm1(step)))
    else:
        # memories of 32 to 4096 tokens, spread over the heads
        s["g"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.arange(Hv, device=dev) / max(Hv - 1, 1)))
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
    if own:
        return _own_pass(state)
    op = state["case"]["op"]
    return {"step": _step, "fwd": _attention, "train": _attention, "ln": _norm, "ln_train": _norm,
            "drop": _dropout}[op](state)


def _own_pass(s):
    import selective_state_space_varlen_amd as ssp
    c, op = s["case"], s["case"]["op"]
    if op == "step":
        out = ssp.decay_attn_pack_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"])
        return {"out": out, "state": s["state"]}
    if op == "drop":
        y = ssp.dropout_pack_fwd(s["x"], c["p"], s["rng"], residual=s["residual"])
        return {"y": y, "dx": ssp.dropout_pack_bwd(s["dy"], c["p"], s["rng"])}
    if op in ("ln", "ln_train"):
        kw = dict(eps=EPS, p=c["p"], rng=s["rng"])
        y, h = ssp.layer_norm_pack_fwd(s["x"], s["w"], s["b"], residual=s["residual"], **kw)
        res = {"y": y, "h": h}
        if op == "ln_train":
            res.update(ssp.layer_norm_pack_bwd(s["dy"], s["h"], s["w"], dh=s["dh"], bias=c["affine"],
                                               residual=c["residual"], **kw))
        return {k: v for k, v in res.items() if v is not None}
    out, hT = ssp.decay_attn_pack_fwd(s["q"], s["k"], s["v"], s["g"], s["cu_seqlens"], initial_state=s["h0"],
                                      final_state=c["carry"])
    res = {"out": out, "hT": hT}
    if op == "train":
        res.update(ssp.decay_attn_pack_bwd(s["q"], s["k"], s["v"], s["g"], s["cu_seqlens"], s["dout"],
                                           initial_state=s["h0"], dfinal_state=s["dhT"], dinitial_state=c["carry"]))
    return {k: v for k, v in res.items() if v is not None}


def work(case):
    elt = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("ln", "ln_train", "drop"):
        n = case["T"] * max(case.get("H", 1), 1) * case["D"]
        streams = 2 + (1 if case["residual"] else 0)  # x, y, residual
        if case["op"] == "drop":
            return {"bytes": (streams + 2) * n * elt, "flops": 12 * n}
        summed = case["residual"] or case["p"] > 0
        streams += 1 if summed else 0  # h
        flops = 8 * n
        if case["op"] == "ln_train":
            # dy, h, dx; dh, and the residual's gradient where it is another
            streams += 3 + (1 if summed else 0) + (1 if case["residual"] and case["p"] else 0)
            flops += 14 * n
        return {"bytes": streams * n * elt, "flops": flops}
    Hk, Hv, Dk, Dv = (case[k] for k in ("Hk", "Hv", "Dk", "Dv"))
    T = case["B"] if case["op"] == "step" else case["T"]
    S = Hv * Dk * Dv
    g = 4 * Hv * (T if case["per_token"] else 1)
    b = T * (2 * Hk * Dk + 2 * Hv * Dv) * elt + g  # q, k, v, out; g
    if case["op"] == "step":
        return {"bytes": b + T * S * 8, "flops": 5 * T * S}
    n = len(_lengths(case)) if case["carry"] else 0
    b += n * S * 8
    if case["op"] == "fwd":
        return {"bytes": b, "flops": 5 * T * S}
    # the forward's inputs again, dout, dq, dk, dv; g, dg; the states' gradients
    b += T * (4 * Hk * Dk + 3 * Hv * Dv) * elt + 2 * g + n * S * 12
    return {"bytes": b, "flops": 17 * T * S}


# ---------------------------------------------------------------------------
# plain form
def _step(s):
    c, dt = s["case"], s["q"].dtype
    r = c["Hv"] // c["Hk"]
    q, k = (s[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    at = s["slots"].long()
    S = s["state"][at] * torch.exp(s["g"])[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    s["state"][at] = S
    return {"out": ((S * q[..., None]).sum(-2) * c["Dk"] ** -0.5).to(dt), "state": s["state"]}


def _layout(lens, dev):
    """Rows of the packed batch by chunks of 64 tokens that start anew in each
    sequence (row T stands for padding), and the chunks' sequences."""
    T = sum(lens)
    lens = np.array(lens, np.int64)
    start, m = np.cumsum(lens) - lens, -(-lens // CHUNK)
    seq = np.repeat(np.arange(len(lens)), m)
    first = (np.arange(len(seq)) - (np.cumsum(m) - m)[seq]) * CHUNK  # a chunk's first token in its sequence
    pos = first[:, None] + np.arange(CHUNK)
    rows = np.where(pos < lens[seq][:, None], start[seq][:, None] + pos, T)
    return torch.from_numpy(rows.reshape(-1)).to(dev), torch.from_numpy(seq).to(dev)


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


def _flow(W, X):
    """(heads, m, n) weights times n states a head: (n, heads, Dk, Dv) -> (m, heads, Dk, Dv)."""
    n, H, Dk, Dv = X.shape
    return (W @ X.transpose(0, 1).reshape(H, n, Dk * Dv)).view(H, -1, Dk, Dv).transpose(0, 1)


def _attention(s):
    """By chunks of 64 tokens: with G the running sum of g in a chunk and S the state that enters it,
    O = scale (e^G Q S + (D . Q K^T) V), D_ij = exp(G_i - G_j) on and below the diagonal; the states
    that enter the chunks are sums of what the sequence's earlier chunks add, decayed on the way."""
    c, dt, dev = s["case"], s["q"].dtype, s["q"].device
    T, Hk, Hv, Dk, Dv = (c[n] for n in ("T", "Hk", "Hv", "Dk", "Dv"))
    scale, n = Dk ** -0.5, len(s["lengths"])
    rows, seq = _layout(s["lengths"], dev)
    N = len(seq)
    q, k, v = (_chunked(s[x], rows, Hv) for x in ("q", "k", "v"))
    g = _chunked(s["g"] if c["per_token"] else s["g"].expand(T, Hv), rows, Hv).double()
    G = g.cumsum(-1)
    i = torch.arange(CHUNK, device=dev)
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(i[:, None] < i, -math.inf)).float()
    eG, eL = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    # decays between chunks: of what chunk b adds until chunk a begins, of the first state until then, of both until the end
    tot = G[..., -1].t()  # (heads, chunks)
    run_ = tot.cumsum(-1)
    a = torch.arange(N, device=dev)
    same = seq[:, None] == seq
    first = torch.searchsorted(seq, torch.arange(n, device=dev))  # a sequence's first chunk
    before = torch.cat([run_.new_zeros(Hv, 1), run_], 1)
    sums = lambda x, y, m: torch.exp((x - y).masked_fill(~m, -math.inf)).float()  # noqa: E731
    between = sums((run_ - tot)[:, :, None], run_[:, None], same & (a[:, None] > a))
    start = before[:, first]  # (heads, sequences): the sum before a sequence
    member = seq[:, None] == torch.arange(n, device=dev)
    enter = sums((run_ - tot)[:, :, None], start[:, None], member)
    last = before[:, torch.searchsorted(seq, torch.arange(n, device=dev), right=True)]
    leave = sums(last[:, :, None], run_[:, None], member.t())  # of what a chunk adds until its sequence ends
    whole = torch.exp(last - start).float().t()[..., None, None]
    U = (eL * k).transpose(-1, -2) @ v
    S = _flow(between, U)
    if s["h0"] is not None:
        S = S + _flow(enter, s["h0"])
    P = D * (q @ k.transpose(-1, -2))
    res = {"out": _packed(scale * (eG * (q @ S) + P @ v), rows, T, dt)}
    if c["carry"]:
        res["hT"] = _flow(leave, U) + whole * s["h0"]
    if c["op"] == "fwd":
        return res
    # gradients: dS is that of the state that leaves a chunk
    do = scale * _chunked(s["dout"], rows, Hv)
    dU = (eG * q).transpose(-1, -2) @ do
    dS = _flow(between.transpose(-1, -2), dU)
    if s["dhT"] is not None:
        dS = dS + _flow(leave.transpose(-1, -2), s["dhT"])
    dP = D * (do @ v.transpose(-1, -2))
    dq = eG * (do @ S.transpose(-1, -2)) + dP @ k
    inter = eL * (v @ dS.transpose(-1, -2))
    dk = inter + dP.transpose(-1, -2) @ q
    dv = eL * (k @ dS) + P.transpose(-1, -2) @ do
    dG = (q * dq - k * dk).sum(-1).double()
    dG[..., -1] += torch.exp(G[..., -1]).float() * (dS * S).sum((-1, -2)) + (k * inter).sum((-1, -2))
    dg = _packed(dG.flip(-1).cumsum(-1).flip(-1), rows, T, torch.float64)
    group = lambda x: x.unflatten(1, (Hk, Hv // Hk)).sum(2)  # noqa: E731
    res.update(dq=_packed(group(dq), rows, T, dt), dk=_packed(group(dk), rows, T, dt), dv=_packed(dv, rows, T, dt),
               dg=(dg if c["per_token"] else dg.sum(0)).float())
    if c["carry"]:
        res["dinitial_state"] = _flow(enter.transpose(-1, -2), dU) + whole * s["dhT"]
    return res


def _keep(shape, p, rng):
    """True where an element is kept, and what it is multiplied by."""
    n, mask = math.prod(shape), 0xffffffff
    cut = round(65536 * p)
    seed, stream = rng[0], rng[1]
    e = torch.arange(-(-n // 8), device=rng.device)
    x = [e & mask, (e >> 32) & mask, (stream & mask).expand_as(e), ((stream >> 32) & mask).expand_as(e)]
    key = [seed & mask, (seed >> 32) & mask]

    def mul(a, m):  # both halves of a 32 x 32 bit product
        lo, hi = (a & 0xffff) * m, (a >> 16) * m
        return ((lo >> 16) + hi) >> 16, (((hi & 0xffff) << 16) + lo) & mask

    for _ in range(10):
        h0, l0 = mul(x[0], 0xD2511F53)
        h1, l1 = mul(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & mask, (key[1] + 0xBB67AE85) & mask]
    u = torch.stack([y for w in x for y in (w & 0xffff, w >> 16)], -1)
    return (u.reshape(-1)[:n] >= cut).view(shape), 65536.0 / (65536 - cut)


def _dropout(s):
    p, x, dt = s["case"]["p"], s["x"].float(), s["x"].dtype
    keep, by = _keep(x.shape, p, s["rng"])
    y = torch.where(keep, x * by, 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(dt), "dx": torch.where(keep, s["dy"].float() * by, 0.0).to(dt)}


def _norm(s):
    c, dt = s["case"], s["x"].dtype
    h = s["x"].float()
    if c["p"]:
        keep, by = _keep(h.shape, c["p"], s["rng"])
        h = torch.where(keep, h * by, 0.0)
    if c["residual"]:
        h = h + s["residual"].float()
    res = {}
    if c["residual"] or c["p"]:
        res["h"] = h.to(dt)

    def standard(h):
        d = h - h.mean(-1, keepdim=True)
        r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
        return d * r, r

    n, _ = standard(h)
    res["y"] = (n * s["w"] + s["b"] if c["affine"] else n).to(dt)
    if c["op"] == "ln":
        return res
    n, r = standard(s["h"].float())
    dy = s["dy"].float()
    if c["affine"]:
        res["dw"], res["db"] = (dy * n).double().sum(0).float(), dy.double().sum(0).float()
        dy = dy * s["w"]
    dh = r * (dy - dy.mean(-1, keepdim=True) - n * (dy * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
    if c["residual"]:
        res["dresidual"] = dh.to(dt)
    res["dx"] = (torch.where(keep, dh * by, 0.0) if c["p"] else dh).to(dt)
    return res


# ---------------------------------------------------------------------------
# 64-bit values, token by token from the definition
def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "fwd": _exact_attention, "train": _exact_attention, "ln": _exact_norm,
            "ln_train": _exact_norm, "drop": _exact_dropout}[case["op"]](s, case)


def _exact_step(s, c):
    heads = torch.arange(c["Hv"], device=s["q"].device) // (c["Hv"] // c["Hk"])
    state = s["state"].double()
    at = s["slots"].long()
    q, k, v = s["q"].double()[:, heads], s["k"].double()[:, heads], s["v"].double()
    decay = s["g"].double().exp().expand(len(at), c["Hv"])
    S = torch.einsum("bhi,bhj->bhij", k, v) + state[at] * decay[:, :, None, None]
    state[at] = S
    return {"out": torch.einsum("bhij,bhi->bhj", S, q) / math.sqrt(c["Dk"]), "state": state}


def _exact_attention(s, c):
    dev, lens = s["q"].device, s["lengths"]
    Hv, Dk, Dv, N, T = c["Hv"], c["Dk"], c["Dv"], len(lens), c["T"]
    heads = torch.arange(Hv, device=dev) // (Hv // c["Hk"])
    scale = 1.0 / math.sqrt(Dk)
    q, k, v = s["q"].double()[:, heads], s["k"].double()[:, heads], s["v"].double()
    a = s["g"].double().exp().expand(T, Hv)
    # longest first: at token t the first active[t] sequences still run
    rank = sorted(range(N), key=lambda i: -lens[i])
    starts = np.concatenate([[0], np.cumsum(lens)])
    longest = max(lens) if lens else 0
    active = [sum(n > t for n in lens) for t in range(longest)]
    first = torch.tensor([int(starts[i]) for i in rank], device=dev)
    S = torch.zeros(N, Hv, Dk, Dv, dtype=torch.float64, device=dev)
    if s["h0"] is not None:
        S += s["h0"].double()[rank]
    train = c["op"] == "train"
    do = s["dout"].double() if train else None
    o = torch.zeros(T, Hv, Dv, dtype=torch.float64, device=dev)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    left = lambda x, M: (x[:, :, None, :] @ M)[:, :, 0]  # noqa: E731  x^T M
    right = lambda M, x: (M @ x[..., None])[..., 0]  # noqa: E731
    for t in range(longest):
        m, at = active[t], first[:active[t]] + t
        S[:m] = S[:m] * a[at][:, :, None, None] + k[at][..., None] * v[at][:, :, None, :]
        o[at] = scale * left(q[at], S[:m])
        if train:
            dq[at] = scale * right(S[:m], do[at])
    back = torch.empty(N, dtype=torch.long, device=dev)
    back[torch.tensor(rank, dtype=torch.long, device=dev)] = torch.arange(N, device=dev)
    res = {"out": o}
    if c["carry"]:
        res["hT"] = S[back]
    if not train:
        return res
    dS = torch.zeros_like(S)
    if s["dhT"] is not None:
        dS += s["dhT"].double()[rank]
    # d g_t = (dS_t . a_t S_{t-1}): what the state's gradient meets in the state before the token. With
    # x_t = (dS_t . S_t), x_t = d g_t + k_t.dk_t and x_t = d g_{t+1} + q_t.dq_t, so it runs back from the end.
    dg = torch.zeros(T, Hv, dtype=torch.float64, device=dev)
    meet = (dS * S).sum((-1, -2))
    for t in reversed(range(longest)):
        m, at = active[t], first[:active[t]] + t
        d = dS[:m] + scale * q[at][..., None] * do[at][:, :, None, :]
        dk[at], dv[at] = right(d, v[at]), left(k[at], d)
        meet[:m] += (q[at] * dq[at]).sum(-1) - (k[at] * dk[at]).sum(-1)
        dg[at] = meet[:m]
        dS[:m] = d * a[at][:, :, None, None]
    total = lambda x: torch.stack([x[:, heads == h].sum(1) for h in range(c["Hk"])], 1)  # noqa: E731
    res.update(dq=total(dq), dk=total(dk), dv=dv, dg=dg if c["per_token"] else dg.sum(0))
    if c["carry"]:
        res["dinitial_state"] = dS[back]
    return res


def _exact_factor(shape, p, rng):
    """0 or 1 / (1 - p) for each element, the generator in 64-bit words on the host."""
    n = int(np.prod(shape))
    seed, stream = (int(x) & (2 ** 64 - 1) for x in rng.cpu())
    low, half = np.uint64(0xffffffff), np.uint64(32)
    c = np.arange(-(-n // 8), dtype=np.uint64)
    a, b = c & low, c >> half
    d, e = np.full_like(c, stream & 0xffffffff), np.full_like(c, stream >> 32)
    for r in range(10):
        k0 = np.uint64((seed + r * 0x9E3779B9) & 0xffffffff)
        k1 = np.uint64(((seed >> 32) + r * 0xBB67AE85) & 0xffffffff)
        u, w = a * np.uint64(0xD2511F53), d * np.uint64(0xCD9E8D57)
        a, b, d, e = (w >> half) ^ b ^ k0, w & low, (u >> half) ^ e ^ k1, u & low
    numbers = np.stack([a, b, d, e], 1).astype("<u4").view("<u2").reshape(-1)[:n].reshape(shape)
    cut = round(65536 * p)
    return torch.from_numpy(numbers >= cut).to(rng.device).double() * (65536 / (65536 - cut))


def _exact_dropout(s, c):
    f = _exact_factor(tuple(s["x"].shape), c["p"], s["rng"])
    y = s["x"].double() * f
    return {"y": y if s["residual"] is None else y + s["residual"].double(), "dx": s["dy"].double() * f}


def _exact_norm(s, c):
    f = _exact_factor(tuple(s["x"].shape), c["p"], s["rng"]) if c["p"] else 1.0
    h = s["x"].double() * f
    if c["residual"]:
        h = h + s["residual"].double()
    res = {"h": h} if c["residual"] or c["p"] else {}
    w = s["w"].double() if c["affine"] else 1.0

    def parts(h):
        var, mean = torch.var_mean(h, -1, correction=0, keepdim=True)
        return mean, (var + EPS).sqrt()

    mean, sd = parts(h)
    res["y"] = (h - mean) / sd * w + (s["b"].double() if c["affine"] else 0.0)
    if c["op"] == "ln":
        return res
    h, dy, D = s["h"].double(), s["dy"].double(), c["D"]
    mean, sd = parts(h)
    if c["affine"]:
        res["dw"] = torch.einsum("t...,t...->...", dy, (h - mean) / sd)
        res["db"] = torch.einsum("t...->...", dy)
    gy = dy * w
    # through h - mean, then through the spread: d sd / d h = (h - mean) / (D sd)
    dsd = -(gy * (h - mean)).sum(-1, keepdim=True) / sd ** 2
    dh = gy / sd + dsd * (h - mean) / (D * sd)
    dh = dh - (gy / sd).sum(-1, keepdim=True) / D
    if s["dh"] is not None:
        dh = dh + s["dh"].double()
    if c["residual"]:
        res["dresidual"] = dh
    res["dx"] = dh * f
    return res
