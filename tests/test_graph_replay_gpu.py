"""Captured ssd_forward calls replayed on changing inputs: every replay gives what an eager call on the
same inputs gives, so no hand-on of a state and no split of the work comes from the replay before."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd

pytestmark = pytest.mark.gpu

CASES = {  # batch, T, H, G, N, dtype, init, lengths
    "ranges": (4, 2048, 16, 1, 128, torch.bfloat16, True, None),       # ranges cross the units
    "long": (1, 8192, 4, 1, 64, torch.bfloat16, False, None),          # segments
    "wide": (2, 2048, 8, 2, 256, torch.bfloat16, True, None),          # two launches
    "packed": (1, 5000, 8, 1, 128, torch.bfloat16, True, [0, 1, 2900, 3100, 5000]),
    "many_tiles": (300, 300, 4, 1, 64, torch.bfloat16, False, None),   # weights by a kernel of their own
    "general": (2, 700, 3, 1, 40, torch.float32, True, None),
}


@pytest.mark.parametrize("which", list(CASES))
def test_replays_on_changing_inputs(which):
    b, T, H, G, N, dtype, init, lengths = CASES[which]
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    rows = b if lengths is None else len(lengths) - 1
    cu = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    A, D = -torch.exp(r(H)), r(H)

    def inputs(i):
        step = torch.nn.functional.softplus(r(b, T, H) - 3)
        step[:, : T * (i % 3) // 3] *= 1e-4  # where the decays are weak differs
        return [r(b, T, H, 64).to(dtype), step, (r(b, T, G, N) * N ** -0.5).to(dtype), (r(b, T, G, N) * N ** -0.5).to(dtype),
                r(rows, H, 64, N) if init else None]

    def call(z):
        return ssd.ssd_forward(z[0], z[1], A, z[2], z[3], D, z[4], cu, 128)

    held = inputs(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, fin = call(held)
    for i in range(6):
        new = inputs(i)
        for h, n in zip(held, new):
            if h is not None:
                h.copy_(n)
        graph.replay()
        got = y.clone(), fin.clone()
        want = call(new)
        torch.cuda.synchronize()
        assert ssd.query_status() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
