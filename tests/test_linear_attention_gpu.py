"""GPU parity of linear attention with a decay for each head (prompt pass, gradients, single
step) against the fp64 recurrence.

Tolerances.  The oracle takes the rounded inputs, so only the library's arithmetic counts.
fp32 results (states, decay gradients, and everything with fp32 inputs): every product takes
its operands to 24 bits and sums at most 8 x 6 tensor-core steps, each cut off at 2^-23 of
the running sum, 48 * 2^-23 = 5.8e-6 if all fell the same way: relative L2 1e-5.  The decay's
gradient is a difference of two such sums, twice that: 2e-5.  bf16 results: three roundings
at most meet in a value (the masked product, the state's copy, the result), each at most half a
step, 2^-8, and spread evenly over that, so 2^-8 / sqrt(3) in the mean: sqrt(3) * 2^-8 / sqrt(3)
= 3.9e-3 in relative L2, held to 5e-3; any single value within 3e-2 of the largest.  That mean
needs many values: with fewer than 256 each is held to the roundings' sum instead, 2^-8 of the
result and 2^-8 of the sizes of the terms that make it up (each term passes one of the other
two roundings), from the same formula on absolute values; (1 + 2^-7) covers their products.
"""
import numpy as np
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from oracle import attention

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(batch, T, H, G, N, P, dtype, decay="token", init=True, lengths=None, seed=0, strength=1.0):
    r = np.random.default_rng(seed)
    if lengths is not None:
        batch, T = 1, int(sum(lengths))
    rows = len(lengths) if lengths is not None else batch
    t = lambda a, d=torch.float32: torch.from_numpy(np.asarray(a)).to(d)
    x = {n: t(r.standard_normal((batch, T, G, N)), DT[dtype]) for n in ("q", "k")}
    x["v"], x["dy"] = (t(r.standard_normal((batch, T, H, P)), DT[dtype]) for _ in range(2))
    shape = (H,) if decay == "head" else (batch, T, H)
    x["log_decay"] = t(-strength * np.exp(r.uniform(np.log(1e-3), np.log(1.5), shape)))
    x["init"] = t(r.standard_normal((rows, H, P, N))) if init else None
    x["dfinal"] = t(r.standard_normal((rows, H, P, N))) if init else None
    x["cu"] = None if lengths is None else t(np.concatenate([[0], np.cumsum(lengths)]), torch.int32)
    x["scale"] = N ** -0.5
    x["offsets"] = x["cu"].numpy() if lengths is not None else np.arange(batch + 1) * T
    return x


def gpu(x):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in x.items()}


def flat(x, n):
    v = x[n]
    v = v.double().numpy()
    return v.reshape((-1,) + v.shape[2:]) if n != "log_decay" or v.ndim > 1 else v


def reference(x):
    f = {n: flat(x, n) for n in ("q", "k", "v", "dy", "log_decay")}
    init, dfin = (None if x[n] is None else x[n].double().numpy() for n in ("init", "dfinal"))
    y, fin = attention.forward(f["q"], f["k"], f["v"], f["log_decay"], x["scale"], init, x["offsets"])
    return f, init, dfin, y, fin


def sizes(x):
    """The operands' absolute values: what the terms of every sum add up to without their signs."""
    return {n: abs(v) if n in ("q", "k", "v", "dy", "init", "dfinal") and v is not None else v for n, v in x.items()}


def close(name, got, ref, dtype, tol32=1e-5, size=None):
    got = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(got).all(), name
    if not ref.size:
        return
    if dtype == "bf16" and ref.size < 256 and size is not None:
        assert (np.abs(got - ref) <= 2.0 ** -8 * (1 + 2.0 ** -7) * (np.abs(ref) + size)).all(), name
        return
    norm, off = np.linalg.norm(ref), np.linalg.norm(got - ref)
    tol = 5e-3 if dtype == "bf16" else tol32
    assert off <= tol * norm + 1e-30, f"{name}: relative L2 {off / norm:.3e} > {tol:.0e}"
    if dtype == "bf16":
        assert np.abs(got - ref).max() <= 3e-2 * np.abs(ref).max(), name


FORWARD = [
    # batch, T, H, G, N, P, dtype, decay, init, lengths
    (1, 1, 1, 1, 1, 1, "bf16", "token", True, None),
    (2, 1, 4, 2, 128, 64, "f32", "token", True, None),
    (1, 63, 2, 2, 64, 64, "bf16", "token", False, None),
    (2, 64, 2, 1, 128, 128, "bf16", "token", True, None),
    (1, 65, 3, 3, 40, 24, "f32", "head", True, None),
    (1, 127, 2, 2, 128, 128, "bf16", "head", True, None),
    (3, 128, 4, 4, 128, 64, "bf16", "token", True, None),
    (1, 129, 5, 1, 100, 72, "bf16", "token", False, None),
    (2, 257, 2, 2, 127, 33, "bf16", "token", True, None),
    (2, 200, 2, 1, 3, 5, "f32", "token", True, None),
    (1, 130, 2, 2, 17, 128, "f32", "token", True, None),
    (1, 3000, 1, 1, 128, 64, "bf16", "token", True, None),
    (1, 1500, 2, 1, 64, 128, "f32", "head", True, None),
    (8, 300, 80, 1, 128, 64, "bf16", "token", True, None),
    (4, 520, 40, 40, 64, 128, "bf16", "head", False, None),
    (1, 0, 4, 2, 64, 64, "bf16", "token", True, [0, 1, 5, 0, 64, 65, 300, 128, 0]),
    (1, 0, 2, 2, 128, 128, "bf16", "token", False, [1, 700, 3, 129, 1000]),
    (1, 0, 3, 1, 72, 40, "f32", "head", True, [33, 0, 600, 1]),
    (1, 0, 16, 4, 64, 128, "bf16", "token", True, [1] * 40 + [200, 17]),
    (1, 0, 2, 1, 32, 32, "bf16", "token", True, [0, 0]),
    (3, 0, 2, 1, 32, 32, "f32", "token", True, None),
]
ids = lambda c: "x".join(str(v) for v in c[:6]) + "_" + "_".join(
    str(v) if not isinstance(v, list) else f"packed{len(v)}" for v in c[6:])


@pytest.mark.parametrize("case", FORWARD, ids=ids)
def test_forward(case):
    b, T, H, G, N, P, dtype, decay, init, lengths = case
    x = make(b, T, H, G, N, P, dtype, decay, init, lengths)
    _, _, _, y_ref, fin_ref = reference(x)
    d = gpu(x)
    y, fin = ssd.linear_attention_forward(d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"], cu_seqlens=d["cu"])
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    close("y", y, y_ref, dtype, size=reference(sizes(x))[3])
    close("final_state", fin, fin_ref, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "strong", "resets", "mixed"])
def test_forward_decays(kind, dtype):
    """No decay at all; decays to nothing within a token or two; decays of zero (-inf), which
    forget; and long memories right after a reset, whose sums must not lose their digits."""
    x = make(2, 300, 4, 2, 64, 64, dtype, seed=3)
    ld = x["log_decay"]
    if kind == "none":
        ld.zero_()
    elif kind == "strong":
        ld.mul_(1e4)
    elif kind == "resets":
        ld[:, ::7] = -float("inf")
    else:
        ld.mul_(1e-3)
        ld[:, 50::97] = -1e30
        ld[:, 51::97] = -float("inf")
    _, _, _, y_ref, fin_ref = reference(x)
    d = gpu(x)
    y, fin = ssd.linear_attention_forward(d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"])
    close("y", y, y_ref, dtype)
    close("final_state", fin, fin_ref, "f32")


BACKWARD = [
    (1, 1, 1, 1, 1, 1, "bf16", "token", True, None),
    (2, 1, 2, 1, 64, 64, "f32", "head", True, None),
    (1, 64, 2, 2, 128, 128, "bf16", "token", True, None),
    (2, 65, 4, 2, 128, 64, "bf16", "token", True, None),
    (1, 129, 3, 3, 40, 24, "f32", "token", True, None),
    (2, 257, 2, 1, 33, 127, "bf16", "head", True, None),
    (1, 200, 6, 2, 3, 5, "f32", "token", False, None),
    (1, 2100, 1, 1, 64, 128, "bf16", "token", True, None),
    (1, 1300, 2, 1, 64, 64, "f32", "head", True, None),
    (8, 700, 24, 24, 64, 64, "bf16", "token", True, None),
    (4, 192, 40, 1, 128, 64, "bf16", "token", False, None),
    (1, 0, 4, 2, 64, 64, "bf16", "token", True, [0, 1, 5, 0, 64, 65, 300, 128, 0]),
    (1, 0, 2, 2, 128, 128, "bf16", "token", False, [1, 700, 3, 129, 600]),
    (1, 0, 3, 1, 72, 40, "f32", "head", True, [33, 0, 600, 1]),
    (1, 0, 2, 1, 32, 32, "bf16", "head", True, [0, 0]),
    (3, 0, 2, 1, 32, 32, "f32", "token", True, None),
]


@pytest.mark.parametrize("case", BACKWARD, ids=ids)
def test_backward(case):
    b, T, H, G, N, P, dtype, decay, init, lengths = case
    x = make(b, T, H, G, N, P, dtype, decay, init, lengths, seed=1)
    f, i, dfin, _, _ = reference(x)
    ref = attention.backward(f["dy"], f["q"], f["k"], f["v"], f["log_decay"], x["scale"], i, dfin, x["offsets"])
    d = gpu(x)
    got = ssd.linear_attention_backward(d["dy"], d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"],
                                        dfinal_state=d["dfinal"], cu_seqlens=d["cu"])
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    z = sizes(x)
    fz, iz, dz, _, _ = reference(z)
    size = attention.backward(fz["dy"], fz["q"], fz["k"], fz["v"], fz["log_decay"], x["scale"], iz, dz, x["offsets"])
    for name, g, r, m in zip(("dq", "dk", "dv"), got, ref, size):
        close(name, g, r, dtype, size=m)
    close("dlog_decay", got[3], ref[3], "f32", 2e-5)
    if init:
        close("dinit_state", got[4], ref[4], "f32")
    else:
        assert got[4] is None
    # without the decay's gradient: the others stay within their tolerances
    less = ssd.linear_attention_backward(d["dy"], d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"],
                                         dfinal_state=d["dfinal"], cu_seqlens=d["cu"], need_dlog_decay=False)
    assert less[3] is None
    for name, g, r, m in zip(("dq", "dk", "dv"), less, ref, size):
        close(name, g, r, dtype, size=m)


@pytest.mark.parametrize("kind", ["none", "strong", "resets"])
def test_backward_decays(kind):
    x = make(1, 300, 4, 2, 64, 64, "f32", seed=3)
    ld = x["log_decay"]
    if kind == "none":
        ld.zero_()
    elif kind == "strong":
        ld.mul_(30)
    else:
        ld[:, ::7] = -float("inf")
    f, i, dfin, _, _ = reference(x)
    ref = attention.backward(f["dy"], f["q"], f["k"], f["v"], f["log_decay"], x["scale"], i, dfin, x["offsets"])
    d = gpu(x)
    got = ssd.linear_attention_backward(d["dy"], d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"],
                                        dfinal_state=d["dfinal"])
    for name, g, r in zip(("dq", "dk", "dv", "dlog_decay", "dinit_state"), got, ref):
        if name == "dlog_decay" and kind == "strong":
            # gradients far below the sums whose difference they are: held to those sums
            size = np.linalg.norm((f["q"] * ref[0]).sum(-1))
            assert np.linalg.norm(g.double().cpu().numpy().reshape(r.shape) - r) <= 2e-5 * (size + np.linalg.norm(r))
            continue
        close(name, g, r, "f32", 2e-5)
    if kind == "resets":
        assert (got[3][:, ::7] == 0).all()


def test_gradients_against_differences():
    """Through the library alone: the forward pass's differences along random directions."""
    x = gpu(make(1, 70, 2, 1, 24, 40, "f32", seed=9))
    names = {"q": "q", "k": "k", "v": "v", "log_decay": "log_decay", "init": "init_state"}
    got = dict(zip(names, ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"],
                                                        init_state=x["init"], dfinal_state=x["dfinal"])))

    def loss(z):
        y, fin = ssd.linear_attention_forward(z["q"], z["k"], z["v"], z["log_decay"], init_state=z["init"])
        return float((y.double() * x["dy"].double()).sum() + (fin.double() * x["dfinal"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for n in names:
        way = torch.randn(x[n].shape, generator=gen, device="cuda")
        if n == "log_decay":
            way = way * x[n].abs()  # stays below zero
        e = 2.0 ** -6
        slope = (loss({**x, n: x[n] + e * way}) - loss({**x, n: x[n] - e * way})) / (2 * e)
        want = float((got[n].double() * way.double()).sum())
        # the loss is linear in q, k, v and init alone (differences are exact but for fp32 rounding
        # of some 1e-6 of its terms' size, over e); in the decays the third derivative adds e^2 / 6
        # of terms like the slope's own
        size = float((got[n].double() * way.double()).square().sum().sqrt())
        assert abs(slope - want) <= 2e-3 * size + 1e-3 * abs(want), (n, slope, want, size)


@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1, "bf16", "token"), (3, 4, 2, 128, 128, "bf16", "token"),
                                  (2, 6, 3, 36, 17, "f32", "head"), (5, 8, 8, 64, 64, "bf16", "head"),
                                  (2, 3, 1, 127, 100, "f32", "token"), (64, 4, 1, 16, 33, "bf16", "token")],
                         ids=lambda c: "x".join(map(str, c[:5])) + f"_{c[5]}_{c[6]}")
def test_steps_match_the_recurrence(case):
    rows, H, G, N, P, dtype, decay = case
    x = make(rows, 5, H, G, N, P, dtype, decay, True, seed=6)
    _, _, _, y_ref, fin_ref = reference(x)
    d = gpu(x)
    state = d["init"].clone()
    ptr, ys = state.data_ptr(), []
    for t in range(5):
        ld = d["log_decay"] if decay == "head" else d["log_decay"][:, t].clone(memory_format=torch.contiguous_format)
        q, k, v = (d[n][:, t].clone(memory_format=torch.contiguous_format) for n in ("q", "k", "v"))
        ys.append(ssd.linear_attention_step(q, k, v, ld, state))
    assert state.data_ptr() == ptr
    close("y", torch.stack(ys, dim=1), y_ref, dtype, size=reference(sizes(x))[3])
    close("state", state, fin_ref, "f32")


def test_prompt_then_steps_continue_one_sequence():
    x = make(2, 150, 4, 2, 64, 64, "bf16", seed=8)
    _, _, _, y_ref, fin_ref = reference(x)
    d = gpu(x)
    cut = lambda n, a, b: d[n][:, a:b].contiguous()
    y, state = ssd.linear_attention_forward(cut("q", 0, 141), cut("k", 0, 141), cut("v", 0, 141),
                                            cut("log_decay", 0, 141), init_state=d["init"])
    ys = [y]
    for t in range(141, 150):
        ys.append(ssd.linear_attention_step(*(d[n][:, t].contiguous() for n in ("q", "k", "v", "log_decay")), state)[:, None])
    close("y", torch.cat(ys, dim=1), y_ref, "bf16")
    close("state", state, fin_ref, "f32")


def test_same_bits_again_and_inputs_untouched():
    x = gpu(make(2, 333, 8, 2, 64, 128, "bf16", seed=10))
    before = {n: v.clone() for n, v in x.items() if isinstance(v, torch.Tensor)}
    f = lambda: ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"])
    b = lambda: ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"],
                                              dfinal_state=x["dfinal"])
    for one, two in zip(f() + b(), f() + b()):
        assert torch.equal(one, two)
    for n, v in before.items():
        assert torch.equal(v, x[n]), n


def test_a_spoiled_sequence_leaves_the_others():
    """NaN and infinities in one packed sequence and head do not reach its neighbours."""
    lengths = [100, 70, 130]
    x = make(1, 0, 2, 2, 64, 64, "bf16", lengths=lengths, seed=11)
    d = gpu(x)
    y0, f0 = ssd.linear_attention_forward(d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"], cu_seqlens=d["cu"])
    d["v"][0, 100:170, 1] = float("nan")
    d["k"][0, 120, 1, 3] = float("inf")
    y1, f1 = ssd.linear_attention_forward(d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"], cu_seqlens=d["cu"])
    assert torch.equal(y0[:, :, 0], y1[:, :, 0]) and torch.equal(f0[:, 0], f1[:, 0])
    for a, b in ((0, 100), (170, 300)):
        assert torch.equal(y0[:, a:b], y1[:, a:b])
    assert torch.equal(f0[[0, 2]], f1[[0, 2]]) and torch.isnan(f1[1, 1]).any()


def test_bad_device_offsets_are_reported_and_nothing_is_written():
    x = gpu(make(1, 0, 2, 1, 64, 64, "bf16", lengths=[40, 60], seed=12))
    for bad in ([0, 70, 60], [1, 40, 100], [0, 40, 99]):
        cu = torch.tensor(bad if bad[-1] != 60 else [0, 120, 100], dtype=torch.int32, device="cuda")
        y = torch.full_like(x["v"], 7.0)
        fin = torch.full_like(x["init"], 7.0)
        ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"], cu_seqlens=cu, y=y,
                                     final_state=fin)
        assert ssd.query_status() == 6
        assert (y == 7).all() and (fin == 7).all()
        ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"],
                                      dfinal_state=x["dfinal"], cu_seqlens=cu)
        assert ssd.query_status() == 6
    assert ssd.query_status() == 0


def test_other_streams_and_two_captured_graphs():
    """On a side stream; and two captured graphs replayed in turn (and at once, on two
    streams) give what eager calls give: no workspace of one is another's."""
    xs = [gpu(make(1, 700, 2, 1, 64, 64, "bf16", seed=s)) for s in (20, 21)]
    call = lambda x: ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"]) + \
        ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"],
                                      dfinal_state=x["dfinal"])
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(xs[0])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
