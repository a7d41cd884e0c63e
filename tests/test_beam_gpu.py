"""GPU parity of beam search's selection and of the reordering of states, and a generation
loop of both with the recurrent step, against the oracle."""
import numpy as np
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from oracle import attention

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check_select(logits, scores, finished=None, eos=-1, count=None):
    got = ssd.beam_select(logits.cuda(), scores.cuda(), None if finished is None else finished.cuda(), eos, count)
    torch.cuda.synchronize()
    for b in range(logits.shape[0]):
        s, w, p = attention.beam_select(logits[b].double().numpy(), scores[b].double().numpy(),
                                        None if finished is None else finished[b].numpy(), eos, count)
        assert got[1][b].tolist() == w.tolist() and got[2][b].tolist() == p.tolist(), b
        g = got[0][b].double().cpu().numpy()
        assert (np.isneginf(g) == np.isneginf(s)).all()
        fin = np.isfinite(s)
        # one rounding to fp32 (2^-24) and the log of a sum of terms exact to some 2^-21
        np.testing.assert_allclose(g[fin], s[fin], rtol=2.0 ** -24, atol=2.0 ** -20)
    return got


SELECT = [
    # batch, beams, vocab, dtype, count
    (1, 1, 1, "f32", 1), (1, 1, 2, "bf16", 4), (2, 3, 7, "f32", 5), (1, 4, 50003, "bf16", None),
    (3, 5, 1001, "bf16", None), (2, 8, 4096, "f32", 16), (1, 64, 333, "bf16", 64), (1, 2, 200001, "f32", 3),
    (5, 4, 2049, "bf16", 8), (2, 16, 30000, "bf16", 32), (1, 1, 1 << 20, "bf16", 64),
]


@pytest.mark.parametrize("case", SELECT, ids=lambda c: "x".join(map(str, c)))
def test_select(case):
    b, k, V, dtype, count = case
    r = np.random.default_rng(V)
    logits = torch.from_numpy(3 * r.standard_normal((b, k, V))).to(DT[dtype])
    scores = torch.from_numpy(-np.sort(r.uniform(0, 20, (b, k)))).float()
    check_select(logits, scores, count=count)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_ties_go_to_the_lowest(dtype):
    V = 5000
    flat = torch.zeros((2, 3, V), dtype=DT[dtype])
    check_select(flat, torch.tensor([[0.0, -1.0, -2.0], [-3.0, -3.0, -3.0]]), count=9)
    few = torch.randint(0, 3, (2, 3, V), generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    few[:, 1] = few[:, 0]
    few[:, 2] = few[:, 0]  # equal rows: equal sums, equal scores
    check_select(few, torch.zeros((2, 3)), count=12)
    zeros = torch.zeros((1, 1, 64), dtype=DT[dtype])
    zeros[0, 0, ::2] = -0.0
    check_select(zeros, torch.zeros((1, 1)), count=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_sorted_rows(dtype):
    """The best continuations all lie side by side: one block's few threads hold them all."""
    x = (torch.arange(6000).float() / 6000 * 40).to(DT[dtype])
    check_select(torch.stack([x, x.flip(0)])[None], torch.tensor([[-0.5, -0.25]]), count=64)


def test_select_masks_and_finished_beams():
    r = np.random.default_rng(3)
    ninf = -float("inf")
    x = torch.from_numpy(3 * r.standard_normal((6, 4, 3000))).float()
    scores = torch.from_numpy(-np.sort(r.uniform(0, 9, (6, 4)))).float()
    x[0, 1] = ninf                       # a row that its mask leaves nothing
    x[1, :, 7:] = ninf                   # few are left
    x[2] = ninf                          # none at all
    x[3, 0, 11] = float("nan")           # a spoiled row
    x[3, 1, 12] = float("inf")
    x[4, :, 2:] = torch.finfo(torch.float32).min  # masks of the type's lowest value
    scores[5, 2:] = ninf                 # unused beams
    fin = torch.zeros((6, 4), dtype=torch.bool)
    fin[0, 0] = fin[5, 1] = True
    check_select(x, scores, fin, 2, 8)
    check_select(x, scores, torch.ones_like(fin), 0, 6)
    check_select(x.bfloat16(), scores, fin, 2999, None)
    check_select(x, scores, None, -1, 3)


def test_select_peaked_and_spread_rows():
    x = torch.full((1, 3, 9000), -80.0)
    x[0, 0, 4321] = 90.0
    x[0, 1] = torch.linspace(-1e4, 1e4, 9000)
    x[0, 2] = 1e30
    check_select(x, torch.zeros((1, 3)), count=6)


REORDER = [
    # batch, beams, row shapes and types
    (1, 1, [((3,), torch.float32)]),
    (2, 4, [((8, 64, 64), torch.float32), ((3, 640), torch.bfloat16)]),
    (3, 5, [((7,), torch.uint8), ((5, 3), torch.bfloat16), ((64,), torch.float64), ((2, 2), torch.float32)]),
    (2, 16, [((1000,), torch.float32), ((0,), torch.float32)]),
    (1, 64, [((260,), torch.float32), ((3,), torch.int16)]),
    (2, 17, [((64,), torch.float32)]),
    (4, 8, [((16, 4), torch.bfloat16)] * 300),
]


@pytest.mark.parametrize("case", REORDER, ids=lambda c: f"{c[0]}x{c[1]}_{len(c[2])}")
@pytest.mark.parametrize("kind", ["random", "same", "one", "turned"])
def test_reorder(case, kind):
    batch, beams, rows = case
    gen = torch.Generator().manual_seed(batch * 100 + beams)
    parents = torch.arange(beams).expand(batch, beams).clone()
    if kind == "random":
        parents = torch.randint(beams, (batch, beams), generator=gen)
    elif kind == "one":
        parents[:] = beams // 2
    elif kind == "turned":
        parents = parents.roll(1, dims=1)
    states = [(100 * torch.rand((batch * beams,) + shape, generator=gen)).to(t) for shape, t in rows]
    d = [s.cuda() for s in states]
    ssd.state_reorder(d, parents.int().cuda())
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    for got, was in zip(d, states):
        want = attention.state_reorder(was.float().numpy() if was.dtype == torch.bfloat16 else was.numpy(), parents.numpy())
        assert torch.equal(got.cpu().to(torch.float64), torch.from_numpy(want).to(torch.float64))


def test_reorder_bad_parents_keep_their_rows():
    x = torch.arange(24.0).reshape(6, 4).cuda()
    ssd.state_reorder(x, torch.tensor([[1, -1, 0], [3, 2, 1]], dtype=torch.int32, device="cuda"))
    assert ssd.query_status() == 8
    assert ssd.query_status() == 0
    assert x[:, 0].tolist() == [4.0, 4.0, 0.0, 12.0, 20.0, 16.0]


def test_select_in_a_graph_and_on_a_side_stream():
    r = np.random.default_rng(5)
    xs = [torch.from_numpy(3 * r.standard_normal((2, 4, 7001))).to(torch.bfloat16).cuda() for _ in range(2)]
    scores = torch.zeros((2, 4), device="cuda")
    want = [ssd.beam_select(x, scores) for x in xs]
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ssd.beam_select(x, scores))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_generation_with_beams():
    """A packed prompt, then beam steps: every step's selection, reordering and recurrent update,
    for a linear attention layer and a convolution window, against the oracle's own loop."""
    batch, beams, H, G, N, P, V, eos = 2, 3, 2, 1, 32, 16, 211, 0
    r = np.random.default_rng(12)
    emb = {n: r.standard_normal((V, d)) for n, d in (("q", G * N), ("k", G * N), ("v", H * P))}
    head = r.standard_normal((H * P, V)) / 4
    decay = -np.array([0.05, 0.4])
    prompts = [r.integers(0, V, n) for n in (37, 5)]
    f32 = lambda a: torch.from_numpy(np.asarray(a)).float().cuda()
    look = lambda n, w, heads: emb[n][w].reshape(len(w), heads, -1)

    words = np.concatenate(prompts)
    cu = np.concatenate([[0], np.cumsum([len(p) for p in prompts])])
    y, state = ssd.linear_attention_forward(f32(look("q", words, G))[None], f32(look("k", words, G))[None],
                                            f32(look("v", words, H))[None], f32(decay), cu_seqlens=f32(cu).int())
    y_ref, state_ref = attention.forward(look("q", words, G), look("k", words, G), look("v", words, H), decay,
                                         N ** -0.5, None, cu)
    last = y[0, torch.from_numpy(cu[1:] - 1).cuda()].double().cpu().numpy()
    np.testing.assert_allclose(last, y_ref[cu[1:] - 1], atol=1e-4)
    # every beam starts from its prompt; at first only one of them is in use
    state = state.repeat_interleave(beams, dim=0)
    state_ref = np.repeat(state_ref, beams, axis=0)
    window, window_ref = torch.zeros((batch * beams, 3), device="cuda"), np.zeros((batch * beams, 3))
    scores = torch.full((batch, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    scores_ref = scores.double().cpu().numpy()
    finished = torch.zeros((batch, beams), dtype=torch.bool, device="cuda")
    out_ref = np.repeat(y_ref[cu[1:] - 1], beams, axis=0)
    out = f32(out_ref)
    W = f32(head)
    for step in range(6):
        logits = (out.reshape(batch, beams, -1) @ W).contiguous()
        logits_ref = logits.double().cpu().numpy()  # the matrix product is not what is tested
        scores, tokens, parents = ssd.beam_select(logits, scores, finished=finished, eos=eos)
        for b in range(batch):
            s, w, p = attention.beam_select(logits_ref[b], scores_ref[b], finished[b].cpu().numpy(), eos)
            assert tokens[b].tolist() == w.tolist() and parents[b].tolist() == p.tolist()
            scores_ref[b] = s
        np.testing.assert_allclose(scores.double().cpu().numpy(), scores_ref, atol=1e-4)
        scores_ref = scores.double().cpu().numpy()
        finished = finished.gather(1, parents.long()) | (tokens == eos)
        ssd.state_reorder([state, window], parents)
        state_ref = attention.state_reorder(state_ref, parents.cpu().numpy())
        window_ref = attention.state_reorder(window_ref, parents.cpu().numpy())
        w = tokens.reshape(-1).cpu().numpy()
        window = torch.cat([window[:, 1:], tokens.reshape(-1, 1).float()], dim=1).contiguous()
        window_ref = np.concatenate([window_ref[:, 1:], w[:, None]], axis=1)
        out = ssd.linear_attention_step(f32(look("q", w, G)), f32(look("k", w, G)), f32(look("v", w, H)), f32(decay), state)
        for row in range(batch * beams):
            o, s = attention.forward(look("q", w[row:row + 1], G), look("k", w[row:row + 1], G),
                                     look("v", w[row:row + 1], H), decay, N ** -0.5, state_ref[row:row + 1])
            out_ref[row], state_ref[row] = o[0], s[0]
        np.testing.assert_allclose(out.double().cpu().numpy(), out_ref, atol=1e-4)
        np.testing.assert_allclose(state.double().cpu().numpy(), state_ref, atol=1e-4)
        assert torch.equal(window.cpu(), torch.from_numpy(window_ref).float())
