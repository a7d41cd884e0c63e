"""A process's first call of an entry point may be a captured one: what the library sets up once (its
scratch pool, its kernels) does not end the capture, and the graph replays to what a later eager call
gives.  Each call has a process of its own."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
import torch
import ssd_sequence_mixing_b200 as ssd

gen = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(s, generator=gen, device="cuda")
T = 700
q, k = r(1, T, 2, 64).bfloat16(), r(1, T, 2, 64).bfloat16()
v, dy = r(1, T, 4, 64).bfloat16(), r(1, T, 4, 64).bfloat16()
decay, state = -r(1, T, 4).abs(), r(1, 4, 64, 64)
logits, scores = r(2, 4, 5000), r(2, 4)
parents = torch.randint(4, (2, 4), generator=gen, device="cuda", dtype=torch.int32)
rows = r(8, 100)
x, dt, A = r(2, 320, 4, 64).bfloat16(), 0.1 * r(2, 320, 4).abs(), -r(4).abs()
B, C, D = r(2, 320, 1, 128).bfloat16(), r(2, 320, 1, 128).bfloat16(), r(4)
cu = torch.tensor([0, 5, 300, 700], dtype=torch.int32, device="cuda")
start, taps = r(3, 4, 64, 64), r(256, 4)


def reorder():
    z = rows.clone()
    ssd.state_reorder(z, parents)
    return (z,)


calls = {
    "forward": lambda: ssd.linear_attention_forward(q, k, v, decay, init_state=state),
    "packed": lambda: ssd.linear_attention_forward(q, k, v, decay, init_state=start, cu_seqlens=cu),
    "fp32": lambda: ssd.linear_attention_forward(q.float(), k.float(), v.float(), decay, init_state=state),
    "backward": lambda: ssd.linear_attention_backward(dy, q, k, v, decay, init_state=state, dfinal_state=state),
    "step": lambda: (ssd.linear_attention_step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                                               decay[:, 0].contiguous(), state.clone()),),
    "select": lambda: ssd.beam_select(logits, scores),
    "reorder": reorder,
    "ssd": lambda: ssd.ssd_forward(x, dt, A, B, C, D),
    "ssd_fp32": lambda: ssd.ssd_forward(x.float(), dt, A, B.float(), C.float(), D),
    "conv": lambda: (ssd.causal_conv1d_silu(x.reshape(2, 320, 256), taps),),
}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls[sys.argv[1]]()
graph.replay()
torch.cuda.synchronize()
want = calls[sys.argv[1]]()
torch.cuda.synchronize()
assert ssd.query_status() == 0
assert all(torch.equal(a, b) for a, b in zip(got, want))
"""


@pytest.mark.parametrize("which", ["forward", "packed", "fp32", "backward", "step", "select", "reorder", "ssd",
                                   "ssd_fp32", "conv"])
def test_first_call_captured(which):
    done = subprocess.run([sys.executable, "-c", PROGRAM, which], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr[-2000:]
