"""Values that are not finite in one sequence of a batch leave the others' results as they are, bit
for bit: prompt pass and gradients, packed and dense batches whose sequences end inside a block of
64 tokens (so that a block's tiles also hold the next sequence's first tokens), both kernels."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from test_linear_attention_gpu import gpu, make

pytestmark = pytest.mark.gpu

BATCHES = {  # batch, T, lengths; the middle sequence is the spoiled one
    "packed": (1, 0, [100, 70, 130]),
    "packed_long": (1, 0, [1111, 700, 1300]),
    "dense": (3, 70, None),
    "dense_long": (3, 1100, None),
}
HEADS = {"own": (2, 2, 64, 64), "shared": (4, 1, 128, 64), "wide": (2, 2, 128, 128)}
VALUES = {"nan": float("nan"), "inf": float("inf"), "huge": 3e38}


def forward(x):
    return ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"], cu_seqlens=x["cu"])


def backward(x, decays):
    return ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"],
                                         dfinal_state=x["dfinal"], cu_seqlens=x["cu"], need_dlog_decay=decays)


def calls(x):
    out = dict(zip(("y", "final_state"), forward(x)))
    for decays in (True, False):
        for n, g in zip(("dq", "dk", "dv", "dlog_decay", "dinit_state"), backward(x, decays)):
            if g is not None:
                out[f"{n}{'' if decays else ' without the decays'}"] = g
    return out


@pytest.mark.parametrize("path", [ssd.PATH_AUTO, ssd.PATH_SIMT], ids=["tensor_core", "general"])
@pytest.mark.parametrize("heads", list(HEADS))
@pytest.mark.parametrize("batch", list(BATCHES))
def test_a_spoiled_sequence_leaves_the_others_gradients(batch, heads, path):
    b, T, lengths = BATCHES[batch]
    H, G, N, P = HEADS[heads]
    clean = gpu(make(b, T, H, G, N, P, "bf16", lengths=lengths, seed=70))
    at = clean["offsets"]
    tokens = lambda t: t.reshape((-1,) + t.shape[2:])
    inside = torch.zeros(int(at[-1]), dtype=torch.bool, device="cuda")
    inside[int(at[1]):int(at[2])] = True

    def others(name, t):
        if "state" in name:  # (rows, H, P, N)
            return t[[0, 2]]
        return tokens(t)[~inside]

    ssd.set_path(path)
    try:
        want = {n: others(n, t) for n, t in calls(clean).items()}
        assert all(torch.isfinite(t).all() for t in want.values())
        for operand in ("q", "k", "v", "dy", "log_decay", "init", "dfinal"):
            for value in VALUES:
                x = dict(clean)
                x[operand] = clean[operand].clone()
                if operand in ("init", "dfinal"):
                    x[operand][1] = VALUES[value]
                else:
                    tokens(x[operand])[inside] = VALUES[value]
                for n, t in calls(x).items():
                    assert torch.equal(others(n, t), want[n]), f"{value} in {operand}: {n}"
        torch.cuda.synchronize()
        assert ssd.query_status() == 0
    finally:
        ssd.set_path(ssd.PATH_AUTO)


@pytest.mark.parametrize("path", [ssd.PATH_AUTO, ssd.PATH_SIMT], ids=["tensor_core", "general"])
@pytest.mark.parametrize("heads", ["own", "shared", "wide"])
def test_a_spoiled_head_leaves_the_others_gradients(heads, path):
    """The same for one head of every sequence; what heads share (dq and dk of a group) is spoiled."""
    H, G, N, P = HEADS[heads]
    clean = gpu(make(2, 700, H, G, N, P, "bf16", seed=71))
    own = G == H
    ssd.set_path(path)
    try:
        want = calls(clean)
        for operand in ("q", "k", "v", "dy", "log_decay", "init", "dfinal"):
            if operand in ("q", "k") and not own:
                continue
            x = dict(clean)
            x[operand] = clean[operand].clone()
            if operand in ("init", "dfinal"):
                x[operand][:, 1] = float("nan")
            else:
                x[operand][:, 300:400, 1] = float("nan")
            for n, t in calls(x).items():
                if n.startswith(("dq", "dk")) and not own:
                    continue
                dim = 1 if "state" in n else 2
                keep = torch.tensor([h for h in range(H) if h != 1], device="cuda")
                assert torch.equal(t.index_select(dim, keep), want[n].index_select(dim, keep)), f"{operand}: {n}"
        torch.cuda.synchronize()
        assert ssd.query_status() == 0
    finally:
        ssd.set_path(ssd.PATH_AUTO)
