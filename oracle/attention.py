"""Linear attention with a decay for each head, its gradients, and beam search's selection, in
plain numpy fp64 -- TEST INFRASTRUCTURE, not the product.

The recurrence is taken literally, token by token, and its gradients by the adjoint recurrence
with every state kept: dlog_decay_t = a_t <D_t, S_{t-1}>, no difference of sums.

All sequences are packed: q, k (T, G, N), v, dy (T, H, P), log_decay (T, H) or (H,),
init, dfinal (nseq, H, P, N) or None, offsets (nseq + 1).
"""
from __future__ import annotations

import numpy as np


def _expand(q, k, v, log_decay):
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    rep = v.shape[1] // q.shape[1]
    a = np.exp(np.broadcast_to(np.asarray(log_decay, dtype=np.float64), v.shape[:2]))
    return np.repeat(q, rep, axis=1), np.repeat(k, rep, axis=1), v, a


def forward(q, k, v, log_decay, scale, init=None, offsets=None):
    """Returns y (T, H, P) and the states after each sequence (nseq, H, P, N)."""
    q, k, v, a = _expand(q, k, v, log_decay)
    T, H, P = v.shape
    offs = [0, T] if offsets is None else [int(o) for o in offsets]
    y, final = np.zeros_like(v), np.zeros((len(offs) - 1, H, P, q.shape[2]))
    for s in range(len(offs) - 1):
        S = np.zeros(final.shape[1:]) if init is None else np.array(init[s], dtype=np.float64)
        for t in range(offs[s], offs[s + 1]):
            S = a[t][:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            y[t] = scale * np.einsum("hpn,hn->hp", S, q[t])
        final[s] = S
    return y, final


def backward(dy, q, k, v, log_decay, scale, init=None, dfinal=None, offsets=None):
    """Returns dq, dk (T, G, N), dv (T, H, P), dlog_decay in log_decay's layout and dinit
    (nseq, H, P, N)."""
    G = np.asarray(q).shape[1]
    constant = np.asarray(log_decay).ndim == 1
    q, k, v, a = _expand(q, k, v, log_decay)
    dy = np.asarray(dy, dtype=np.float64)
    T, H, P = v.shape
    N = q.shape[2]
    offs = [0, T] if offsets is None else [int(o) for o in offsets]
    dq, dk, dv, dl = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((T, H))
    dinit = np.zeros((len(offs) - 1, H, P, N))
    for s in range(len(offs) - 1):
        lo, hi = offs[s], offs[s + 1]
        states = [np.zeros((H, P, N)) if init is None else np.array(init[s], dtype=np.float64)]
        for t in range(lo, hi):
            states.append(a[t][:, None, None] * states[-1] + v[t][:, :, None] * k[t][:, None, :])
        D = np.zeros((H, P, N)) if dfinal is None else np.array(dfinal[s], dtype=np.float64)
        for t in range(hi - 1, lo - 1, -1):
            D = D + scale * dy[t][:, :, None] * q[t][:, None, :]
            dq[t] = scale * np.einsum("hpn,hp->hn", states[t - lo + 1], dy[t])
            dv[t] = np.einsum("hpn,hn->hp", D, k[t])
            dk[t] = np.einsum("hpn,hp->hn", D, v[t])
            dl[t] = a[t] * np.einsum("hpn,hpn->h", D, states[t - lo])
            D = a[t][:, None, None] * D
        dinit[s] = D
    share = lambda x: x.reshape(T, G, H // G, N).sum(axis=2)
    return share(dq), share(dk), dv, (dl.sum(axis=0) if constant else dl), dinit


def beam_select(logits, scores, finished=None, eos=-1, count=None):
    """One batch item: logits (beams, vocab), scores (beams,).  Returns (scores, tokens, parents)
    of the best ``count`` continuations; what is missing as the library documents it.  Scores are
    compared in fp32, as they are returned; equal ones: the lower beam, the larger logit, the
    lower token."""
    x = np.asarray(logits, dtype=np.float64)
    beams, vocab = x.shape
    count = beams if count is None else count
    found = []
    for i in range(beams):
        if finished is not None and finished[i]:
            found.append((float(scores[i]), i, 0.0, eos))
            continue
        with np.errstate(all="ignore"):
            m = np.max(x[i])
            lse = m + np.log(np.sum(np.exp(x[i] - m)))
            total = float(scores[i]) + (x[i] - lse)
        found += [(s, i, x[i, w], w) for w, s in enumerate(total) if s > -np.inf]
    found = sorted((e for e in found if e[0] > -np.inf), key=lambda e: (-np.float32(e[0]), e[1], -e[2], e[3]))[:count]
    out = [(s, w, i) for s, i, _, w in found]
    out += [(-np.inf, max(eos, 0), i % beams) for i in range(len(out), count)]
    return (np.array([o[0] for o in out]), np.array([o[1] for o in out], dtype=np.int64),
            np.array([o[2] for o in out], dtype=np.int64))


def state_reorder(state, parents):
    """state (batch * beams, ...), parents (batch, beams): row (b, i) of row (b, parents[b, i])."""
    batch, beams = np.asarray(parents).shape
    out = np.array(state)
    for b in range(batch):
        for i in range(beams):
            out[b * beams + i] = state[b * beams + int(parents[b][i])]
    return out
