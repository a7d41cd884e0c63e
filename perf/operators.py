"""The operators that are measured: cases, inputs, plain forms and values in 64 bits.

Linear attention with a decay for each head.  For every sequence and head h (group
g = h / (H/G)), with a P x N fp32 state S and a_t = exp(log_decay_t):

    S_t = a_t S_{t-1} + v_t k_t^T,      y_t = scale * S_t q_t

as a pass over whole prompts (``forward``), its gradients (``backward``) and one generation
step (``step``).  Beam search over a vocabulary (``select``): the best ``beams`` of beams x
vocabulary continuations by cumulative log-probability; and the reordering of the beams'
recurrent states that follows it (``reorder``).

``own`` false: the plain forms, elementary torch operations in 32 bits (angles, sums of
log-decays and scores in 64).  ``own`` true: the calls of ssd_sequence_mixing_b200.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # block length of the plain chunked form
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def _attention(name, op, dtype, batch, seqlen, H, G, N, P, decay="token", init=False, lengths=""):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "seqlen": seqlen, "H": H, "G": G, "N": N, "P": P,
            "decay": decay, "init": init, "lengths": lengths}


def listed():
    return [
        # one short sequence of a small model: the call's latency
        _attention("forward_tiny", "forward", "f32", 1, 256, 2, 1, 16, 16),
        # a prompt batch through a layer whose heads all share one query and key
        _attention("forward_layer", "forward", "bf16", 8, 2048, 80, 1, 128, 64),
        # a prompt batch through a layer with its own query and key in every head, constant
        # decays, continued from earlier states
        _attention("forward_heads", "forward", "bf16", 8, 2048, 32, 32, 128, 128, decay="head", init=True),
        # a server's packed prompts, from one token to thousands, each with its own state
        _attention("forward_packed", "forward", "bf16", 1, 0, 16, 4, 64, 128, init=True,
                   lengths="1,8192,37,700,2500,64,129,1023,5,3001,1,1999,350,4096,777,128"),
        # a training step's layer
        _attention("backward_heads", "backward", "bf16", 4, 2048, 16, 16, 128, 128),
        # shared queries and keys, odd sizes, gradients of and through the states
        _attention("backward_grouped", "backward", "f32", 2, 777, 8, 2, 96, 64, init=True),
        # one sequence's next token: latency
        _attention("step_small", "step", "bf16", 1, 1, 8, 1, 128, 64, init=True),
        # a server's batch of next tokens: the states' traffic
        _attention("step_serving", "step", "bf16", 64, 1, 32, 32, 128, 128, init=True),
        # one user's beam search step
        {"name": "select_small", "op": "select", "dtype": "bf16", "batch": 1, "beams": 4, "vocab": 50003, "finished": 0},
        # a batch of beam searches over a large vocabulary, some beams finished
        {"name": "select_large", "op": "select", "dtype": "f32", "batch": 64, "beams": 8, "vocab": 128000, "finished": 1},
        # the states of one user's beams, a small model of four layers
        {"name": "reorder_small", "op": "reorder", "batch": 1, "beams": 4, "layers": 4, "H": 8, "P": 64, "N": 64,
         "channels": 640},
        # the states of a batch of beam searches in eight layers of a large model
        {"name": "reorder_large", "op": "reorder", "batch": 16, "beams": 4, "layers": 8, "H": 80, "P": 64, "N": 128,
         "channels": 5376},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("forward", "forward", "backward", "backward", "step", "select", "reorder"))
    if op in ("forward", "backward", "step"):
        dtype = rng.choice(("bf16", "bf16", "f32"))
        G = rng.choice((1, 2, 4, 8, 16))
        H = G * rng.choice((1, 1, 2, 4, 5))
        N, P = rng.choice((16, 40, 64, 64, 96, 128, 128)), rng.choice((16, 24, 64, 64, 100, 128, 128))
        decay, init = rng.choice(("token", "token", "head")), rng.random() < 0.5
        if op == "step":
            batch = min(_log_int(rng, 1, 200), max(1, 64 * 32 * 128 * 128 // (H * N * P)))
            return {k: v for k, v in _attention("", op, dtype, batch, 1, H, G, N, P, decay, True).items() if k != "name"}
        # tokens of the whole call: at most the work of the largest listed case of the operator
        most = (16384 * 32 if op == "forward" else 8192 * 16) * 128 * 128 // (H * N * P)
        tokens = _log_int(rng, 1, min(most, 40000 if dtype == "bf16" else 8000))
        batch, lengths = 1, ""
        if rng.random() < 0.4:
            left, got = tokens, []
            while left > 0 and len(got) < 24:
                got.append(min(left, _log_int(rng, 1, 5000)))
                left -= got[-1]
            if rng.random() < 0.3:
                got.insert(rng.randrange(len(got) + 1), 0)
            lengths, seqlen = ",".join(map(str, got)), 0
            # the plain form pads every sequence to the longest
            while len(got) > 1 and len(got) * max(got) > 2 * most:
                got.remove(max(got))
                lengths = ",".join(map(str, got))
        else:
            batch = _log_int(rng, 1, min(8, tokens))
            seqlen = tokens // batch
        return {k: v for k, v in _attention("", op, dtype, batch, seqlen, H, G, N, P, decay, init, lengths).items()
                if k != "name"}
    if op == "select":
        beams = rng.choice((1, 2, 3, 4, 5, 8, 16))
        vocab = _log_int(rng, 500, 200000)
        batch = min(_log_int(rng, 1, 100), max(1, 64 * 8 * 128000 // (beams * vocab)))
        return {"op": op, "dtype": rng.choice(("bf16", "f32")), "batch": batch, "beams": beams, "vocab": vocab,
                "finished": rng.randrange(2)}
    beams, H, P, N = rng.choice((2, 3, 4, 5, 8)), rng.choice((1, 8, 24, 80)), rng.choice((16, 64, 128)), rng.choice((16, 40, 128))
    layers = rng.choice((1, 2, 5, 8))
    batch = min(_log_int(rng, 1, 64), max(1, 16 * 4 * 8 * 80 * 64 * 128 // (beams * layers * H * P * N)))
    return {"op": op, "batch": batch, "beams": beams, "layers": layers, "H": H, "P": P, "N": N,
            "channels": 8 * rng.randrange(1, 700)}


# ------------------------------------------------------------------------------ inputs
def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")] if case["lengths"] else []


def _log_decay(case, shape, gen):
    """Log-decays of a selective layer: -softplus(noise + b_h) * A_h, with e^b from 1e-3 to
    1e-1 and A from 1 to 16; or one constant for each head, memories of 32 to 4096 tokens."""
    H, dev = case["H"], "cuda"
    if case["decay"] == "head":
        return torch.log1p(-torch.exp2(-torch.linspace(5, 12, H, device=dev, dtype=torch.float64))).float()
    dt0 = torch.exp(math.log(1e-3) + (math.log(1e-1) - math.log(1e-3)) * torch.rand(H, generator=gen, device=dev))
    b = torch.log(torch.expm1(dt0))
    A = torch.exp(math.log(16.0) * torch.rand(H, generator=gen, device=dev))
    raw = 0.5 * torch.randn(shape + (H,), generator=gen, device=dev) + b
    return -torch.log1p(torch.exp(raw)) * A


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    s = {"case": case}
    if case["op"] in ("forward", "backward", "step"):
        dtype, H, G, N, P = DTYPE[case["dtype"]], case["H"], case["G"], case["N"], case["P"]
        lengths = _lengths(case)
        batch, T = (1, sum(lengths)) if lengths else (case["batch"], case["seqlen"])
        rows = len(lengths) if lengths else batch
        lead = (batch,) if case["op"] == "step" else (batch, T)
        s["scale"] = N ** -0.5
        s["q"], s["k"] = (normal(*lead, G, N).to(dtype) for _ in range(2))
        s["v"] = normal(*lead, H, P).to(dtype)
        s["log_decay"] = _log_decay(case, lead, gen)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda") if lengths else None
        s["init"] = normal(rows, H, P, N) if case["init"] else None
        if case["op"] == "backward":
            s["dy"] = normal(*lead, H, P).to(dtype)
            s["dfinal"] = normal(rows, H, P, N) if case["init"] else None
        if lengths:
            s["lengths"] = lengths
            # row r, column t of the padded batch is token offset_r + t (past the end: token 0)
            off = s["cu"][:-1, None].long()
            t = torch.arange(max(lengths), device="cuda")[None]
            s["inside"] = t < torch.tensor(lengths, device="cuda")[:, None]
            s["token"] = torch.where(s["inside"], off + t, torch.zeros_like(t))
    elif case["op"] == "select":
        b, k, V = case["batch"], case["beams"], case["vocab"]
        s["logits"] = (3 * normal(b, k, V)).to(DTYPE[case["dtype"]])
        s["logits"][:, :, torch.randint(V, (max(1, V // 100),), generator=gen, device="cuda")] = -math.inf  # banned words
        s["scores"] = torch.sort(-20 * torch.rand(b, k, generator=gen, device="cuda"), dim=1, descending=True).values
        s["finished"] = (torch.rand(b, k, generator=gen, device="cuda") < 0.2) if case["finished"] else None
        s["eos"] = 2
    else:
        rows = case["batch"] * case["beams"]
        s["parents"] = torch.randint(case["beams"], (case["batch"], case["beams"]), generator=gen, device="cuda", dtype=torch.int32)
        s["states"] = [normal(rows, case["H"], case["P"], case["N"]) for _ in range(case["layers"])]
        s["states"] += [normal(rows, 3, case["channels"]).bfloat16() for _ in range(case["layers"])]
    return s


# ---------------------------------------------------------------------- the plain forms
def _rows(s, x):
    """Packed tokens (1, T, ...) as a batch padded with zeros; a dense batch as it is."""
    if s["cu"] is None:
        return x
    keep = s["inside"].reshape(s["inside"].shape + (1,) * (x.dim() - 2))
    return torch.where(keep, x[0][s["token"]], torch.zeros((), dtype=x.dtype, device=x.device))


def _tokens(s, x):
    """The way back: (rows, longest, ...) to (1, T, ...)."""
    return x if s["cu"] is None else x[s["inside"]][None]


def _chunked(query, key, value, g, start):
    """out_i = sum_{j <= i} exp(g_{j+1} + ... + g_i) (query_i . key_j) value_j, and from `start`.

    query, key (B, T, H, N), value (B, T, H, P) in 32 bits, g (B, T, H) in 64, start
    (B, H, P, N) or None -> out (B, T, H, P), the state after the last token (B, H, P, N)."""
    B, T, H, N = query.shape
    P = value.shape[-1]
    C = min(CHUNK, max(T, 1))
    K = -(-T // C)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, K * C - T))
    cut = lambda x: pad(x).reshape((B, K, C) + x.shape[2:]).movedim(3, 1)  # (B, H, K, C, ...)
    q, k, v = cut(query), cut(key), cut(value)
    c = torch.cumsum(cut(g), dim=-1)  # (B, H, K, C), from the chunk's start
    i = torch.arange(C, device=g.device)
    L = torch.where(i[:, None] >= i[None], c[..., :, None] - c[..., None, :], -math.inf).exp().float()
    out = ((q @ k.transpose(-1, -2)) * L) @ v
    states = (v * (c[..., -1:] - c).exp().float()[..., None]).transpose(-1, -2) @ k  # (B, H, K, P, N)
    # the state before chunk m (m = K: after the last) from chunks n < m and from the start
    E = torch.cumsum(torch.nn.functional.pad(c[..., -1], (1, 0)), dim=-1)  # (B, H, K + 1)
    m = torch.arange(K + 1, device=g.device)
    carry = torch.where(m[:, None] > m[None, :-1], E[..., :, None] - E[..., None, 1:], -math.inf).exp().float()
    before = (carry @ states.reshape(B, H, K, P * N)).reshape(B, H, K + 1, P, N)
    if start is not None:
        before = before + E.exp().float()[..., None, None] * start[:, :, None]
    out = out + (q * c.exp().float()[..., None]) @ before[:, :, :-1].transpose(-1, -2)
    return out.movedim(1, 3).reshape(B, K * C, H, P)[:, :T], before[:, :, -1]


def _plain_parts(s):
    rep = s["v"].shape[-2] // s["q"].shape[-2]
    q, k = (_rows(s, s[n]).float().repeat_interleave(rep, dim=-2) for n in ("q", "k"))
    v = _rows(s, s["v"]).float()
    g = s["log_decay"].double()
    g = _rows(s, g) if g.dim() > 1 else g.expand(v.shape[:-1])
    if s["cu"] is not None:
        g = torch.where(s["inside"][..., None], g, torch.zeros_like(g))
    return q * s["scale"], k, v, g


def _plain_forward(s):
    q, k, v, g = _plain_parts(s)
    y, final = _chunked(q, k, v, g, s["init"])
    return {"y": _tokens(s, y).to(s["v"].dtype), "final_state": final}


def _plain_backward(s):
    q, k, v, g = _plain_parts(s)
    dy = _rows(s, s["dy"]).float()
    back = lambda x: x.flip(1)
    swap = lambda x: None if x is None else x.transpose(-1, -2)
    # the gradient of the state runs backwards: before token t it has decayed by a_{t+1}, ...
    r = torch.nn.functional.pad(back(g)[:, :-1], (0, 0, 1, 0)) if g.shape[1] else g
    dq, final = _chunked(dy, v, k, g, swap(s["init"]))
    dk, _ = _chunked(back(v), back(dy), back(q), r, swap(s["dfinal"]))
    dv, dstart = _chunked(back(k), back(q), back(dy), r, s["dfinal"])
    dk, dv = back(dk), back(dv)
    # d log_decay_t: everything from tokens before t to tokens from t on
    d = (q * dq).double().sum(-1) - (k * dk).double().sum(-1)
    dg = torch.cumsum(d.flip(1), dim=1).flip(1)
    if s["dfinal"] is not None:
        dg = dg + (s["dfinal"].double() * swap(final).double()).sum((-1, -2))[:, None]
    dq = dq * s["scale"]
    G, N = s["q"].shape[-2:]
    group = lambda x: _tokens(s, x.reshape(x.shape[:2] + (G, -1, N)).sum(3)).to(s["q"].dtype)
    out = {"dq": group(dq), "dk": group(dk), "dv": _tokens(s, dv).to(s["v"].dtype)}
    dg = _tokens(s, dg)
    out["dlog_decay"] = (dg if s["log_decay"].dim() > 1 else dg.sum((0, 1))).float()
    if s["init"] is not None:
        out["dinit_state"] = dstart * g[:, 0].exp().float()[..., None, None]
    return out


def _plain_step(s):
    rep = s["v"].shape[-2] // s["q"].shape[-2]
    q, k = (s[n].float().repeat_interleave(rep, dim=1) for n in ("q", "k"))
    S = s["init"]
    S.mul_(s["log_decay"].exp()[..., None, None]).add_(s["v"].float()[..., None] * k[..., None, :])
    y = (S * q[..., None, :]).sum(-1) * s["scale"]
    return {"y": y.to(s["v"].dtype), "state": S}


def _plain_select(s):
    b, beams, V = s["logits"].shape
    x = s["logits"].float()
    top = x.max(dim=-1, keepdim=True).values.double()
    lse = top + (x.double() - top).exp().sum(-1, keepdim=True).log()
    best, token = torch.sort(x, dim=-1, descending=True, stable=True)  # ties: the lowest token first
    best, token = best[..., :beams], token[..., :beams]
    score = s["scores"].double()[..., None] + (best.double() - lse)
    if s["finished"] is not None:
        # a finished beam goes on as it is, by its end token alone
        f = s["finished"][..., None]
        first = torch.arange(beams, device=x.device) == 0
        score = torch.where(f, torch.where(first, s["scores"].double()[..., None], -math.inf), score)
        token = torch.where(f, s["eos"], token)
    # compared as they are returned; equal ones: the lower beam, then the larger logit
    score, at = torch.sort(score.float().reshape(b, -1), dim=1, descending=True, stable=True)
    score, at = score[:, :beams], at[:, :beams]
    return {"scores": score, "tokens": token.reshape(b, -1).gather(1, at).int(), "parents": (at // beams).int()}


def _plain_reorder(s):
    b, beams = s["parents"].shape
    source = (torch.arange(b, device="cuda")[:, None] * beams + s["parents"]).reshape(-1).long()
    for x in s["states"]:
        x.copy_(x[source])
    return {"states": s["states"]}


PLAIN = {"forward": _plain_forward, "backward": _plain_backward, "step": _plain_step, "select": _plain_select,
         "reorder": _plain_reorder}


def _own(s):
    import ssd_sequence_mixing_b200 as ssd

    op = s["case"]["op"]
    if op == "forward":
        y, final = ssd.linear_attention_forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                                init_state=s["init"], cu_seqlens=s["cu"])
        return {"y": y, "final_state": final}
    if op == "backward":
        dq, dk, dv, dg, dinit = ssd.linear_attention_backward(s["dy"], s["q"], s["k"], s["v"], s["log_decay"],
                                                              scale=s["scale"], init_state=s["init"],
                                                              dfinal_state=s["dfinal"], cu_seqlens=s["cu"])
        out = {"dq": dq, "dk": dk, "dv": dv, "dlog_decay": dg}
        if s["init"] is not None:
            out["dinit_state"] = dinit
        return out
    if op == "step":
        y = ssd.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["init"], scale=s["scale"])
        return {"y": y, "state": s["init"]}
    if op == "select":
        scores, tokens, parents = ssd.beam_select(s["logits"], s["scores"], finished=s["finished"], eos=s["eos"])
        return {"scores": scores, "tokens": tokens, "parents": parents}
    ssd.state_reorder(s["states"], s["parents"])
    return {"states": s["states"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------- work
def work(case):
    """Every input read once, every output written once, and the recurrence's own products."""
    if case["op"] in ("forward", "backward", "step"):
        e = 2 if case["dtype"] == "bf16" else 4
        H, G, N, P = case["H"], case["G"], case["N"], case["P"]
        lengths = _lengths(case)
        tokens = sum(lengths) if lengths else case["batch"] * case["seqlen"]
        rows = len(lengths) if lengths else case["batch"]
        state, decay = rows * H * P * N * 4, 4 * (tokens * H if case["decay"] == "token" else H)
        qk, v = tokens * G * N * e, tokens * H * P * e
        if case["op"] == "forward":
            return {"bytes": 2 * qk + 2 * v + decay + state * (2 if case["init"] else 1), "flops": 4 * tokens * H * P * N}
        if case["op"] == "backward":
            # q, k, v, dy and the decays in; dq, dk, dv and the decays' gradients out
            return {"bytes": 4 * qk + 3 * v + 2 * decay + state * (3 if case["init"] else 0), "flops": 10 * tokens * H * P * N}
        return {"bytes": 2 * qk + 2 * v + decay + 2 * state, "flops": 4 * tokens * H * P * N}
    if case["op"] == "select":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 16 * case["batch"] * case["beams"], "flops": 3 * n}
    # random parents: the rows that move are written, and each of their sources is read once
    b = case["beams"]
    row = case["layers"] * (4 * case["H"] * case["P"] * case["N"] + 2 * 3 * case["channels"])
    written, read = 1 - 1 / b, 1 - (1 - 1 / b) ** (b - 1)
    return {"bytes": case["batch"] * b * (row * (written + read) + 4), "flops": 0}


# ------------------------------------------------------------------- values in 64 bits
def _sequences(case, s):
    """(tokens' slice, rows' slice) of what runs as one recurrence: the whole dense batch, or
    each packed sequence."""
    lengths = _lengths(case)
    if not lengths:
        return [(slice(0, case["seqlen"]), slice(0, case["batch"]))]
    ends = np.cumsum(lengths).tolist()
    return [(slice(e - n, e), slice(r, r + 1)) for r, (n, e) in enumerate(zip(lengths, ends))]


def _exact_attention(case, s):
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    head = torch.arange(H, device="cuda") // (H // G)
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    a = s["log_decay"].double().exp()
    a = a if a.dim() > 1 else a.expand(v.shape[:-1])
    outer = lambda x, y: x[..., :, None] * y[..., None, :]
    if case["op"] == "step":
        S = s["init"].double() * a[..., None, None] + outer(v, k[:, head])
        return {"y": s["scale"] * (S @ q[:, head][..., None])[..., 0], "state": S}
    dy = s["dy"].double() if case["op"] == "backward" else None
    out = {}
    keep = lambda name, like: out.setdefault(name, torch.zeros(like, dtype=torch.float64, device="cuda"))
    rows = len(_lengths(case)) or case["batch"]
    for t_range, r_range in _sequences(case, s):
        b_range = slice(0, case["batch"]) if not _lengths(case) else slice(0, 1)
        part = lambda x: x[b_range, t_range]
        Q, Kk, V, A = part(q)[:, :, head], part(k)[:, :, head], part(v), part(a)
        n, T = r_range.stop - r_range.start, t_range.stop - t_range.start
        S = s["init"][r_range].double().clone() if s["init"] is not None else torch.zeros((n, H, P, N), dtype=torch.float64, device="cuda")
        if case["op"] == "forward":
            y = keep("y", v.shape)
            for t in range(T):
                S.mul_(A[:, t, :, None, None]).add_(outer(V[:, t], Kk[:, t]))
                y[b_range, t_range.start + t] = s["scale"] * (S @ Q[:, t][..., None])[..., 0]
            keep("final_state", (rows, H, P, N))[r_range] = S
            continue
        DY = part(dy)
        dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (Q, Q, V))
        dg = torch.zeros(V.shape[:-1], dtype=torch.float64, device="cuda")
        for t in range(T):
            S.mul_(A[:, t, :, None, None]).add_(outer(V[:, t], Kk[:, t]))
            dq[:, t] = s["scale"] * (DY[:, t][..., None, :] @ S)[..., 0, :]
        D = s["dfinal"][r_range].double().clone() if s["dfinal"] is not None else torch.zeros_like(S)
        through = (D * S).sum((-1, -2))
        for t in range(T - 1, -1, -1):
            D.add_(s["scale"] * outer(DY[:, t], Q[:, t]))
            dv[:, t] = (D @ Kk[:, t][..., None])[..., 0]
            dk[:, t] = (V[:, t][..., None, :] @ D)[..., 0, :]
            through = through + (Q[:, t] * dq[:, t]).sum(-1) - (Kk[:, t] * dk[:, t]).sum(-1)
            dg[:, t] = through
            D.mul_(A[:, t, :, None, None])
        shared = lambda x: x.reshape(x.shape[:2] + (G, H // G, N)).sum(3)
        keep("dq", q.shape)[b_range, t_range] = shared(dq)
        keep("dk", k.shape)[b_range, t_range] = shared(dk)
        keep("dv", v.shape)[b_range, t_range] = dv
        keep("dg", v.shape[:-1])[b_range, t_range] = dg
        if s["init"] is not None:
            keep("dinit_state", (rows, H, P, N))[r_range] = D
    if case["op"] == "backward":
        dg = out.pop("dg")
        out["dlog_decay"] = dg if s["log_decay"].dim() > 1 else dg.sum((0, 1))
    return out


def _exact_select(case, s):
    beams = case["beams"]
    scores, tokens, parents = [], [], []
    for b in range(case["batch"]):
        total = (torch.log_softmax(s["logits"][b].double(), dim=-1) + s["scores"][b].double()[:, None]).cpu().numpy()
        for i in range(beams):
            if s["finished"] is not None and bool(s["finished"][b, i]):
                total[i] = -math.inf
                total[i, s["eos"]] = float(s["scores"][b, i])
        flat, rounded = total.reshape(-1), total.reshape(-1).astype(np.float32)
        at = np.flatnonzero(rounded >= np.partition(rounded, flat.size - beams)[flat.size - beams])
        # equal as they are returned: the lower beam, then the larger logit, then the lower token
        logit = s["logits"][b].reshape(-1)[torch.from_numpy(at).cuda()].double().cpu().numpy()
        at = at[np.lexsort((at, -logit, at // case["vocab"], -rounded[at]))][:beams]
        scores.append(flat[at])
        tokens.append(at % case["vocab"])
        parents.append(at // case["vocab"])
    return {"scores": torch.from_numpy(np.stack(scores)), "tokens": torch.from_numpy(np.stack(tokens)).int(),
            "parents": torch.from_numpy(np.stack(parents)).int()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(case, s)
    if case["op"] == "reorder":
        moved = []
        for x in s["states"]:
            rows = x.reshape((case["batch"], case["beams"]) + x.shape[1:])
            moved.append(torch.stack([torch.stack([rows[b, p] for p in order]) for b, order in enumerate(s["parents"].tolist())]).reshape(x.shape).double())
        return {"states": moved}
    steps = 2 * (sum(_lengths(case)) or case["seqlen"])
    return _exact_attention(case, s) if steps <= 90000 else None
