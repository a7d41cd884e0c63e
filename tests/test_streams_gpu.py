"""The sequence-mixing entry points on a stream that is not torch's current one: their results are
not memory that the current stream has freed but not finished writing."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd

pytestmark = pytest.mark.gpu


def calls():
    gen = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    b, T, H, P, G, N = 2, 320, 4, 64, 1, 128
    x, dt, A = r(b, T, H, P).bfloat16(), r(b, T, H).abs() * 0.1, -r(H).abs()
    B, C, D = r(b, T, G, N).bfloat16(), r(b, T, G, N).bfloat16(), r(H)
    z, w = r(b, T, H, P).bfloat16(), r(P)
    xbc, cw = r(b, T, 256).bfloat16(), r(256, 4)
    states, decays = r(2, H, P, N), -r(2, H).abs()
    state = r(b, H, P, N)
    one = [t[:, 0].contiguous() for t in (x, dt)], [t[:, 0].contiguous() for t in (B, C)]
    return {
        "forward": lambda s: ssd.ssd_forward(x, dt, A, B, C, D, stream=s),
        "final_state": lambda s: (ssd.ssd_final_state(x, dt, A, B, stream=s),),
        "noalloc": lambda s: ssd.ssd_forward_noalloc(x, dt, A, B, C, D, stream=s),
        "dt": lambda s: ssd.ssd_forward_dt(x, dt, A, B, C, D, stream=s),
        "conv": lambda s: (ssd.causal_conv1d_silu(xbc, cw, stream=s),),
        "norm": lambda s: (ssd.gated_rmsnorm(x, z, w, stream=s),),
        "logdecay": lambda s: (ssd.segment_logdecay(dt[:1], A, stream=s),),
        "prefix": lambda s: (ssd.state_prefix(2, states, decays, stream=s),),
        "decode": lambda s: (ssd.ssd_decode_step(one[0][0], one[0][1], A, one[1][0], one[1][1], D, copies.pop(), stream=s),),
    }, state


copies = []


@pytest.mark.parametrize("which", ["forward", "final_state", "noalloc", "dt", "conv", "norm", "logdecay", "prefix",
                                   "decode"])
def test_results_are_not_memory_in_use_by_the_current_stream(which):
    f, state = calls()
    copies[:] = [state.clone() for _ in range(4)]
    want = [t.clone() for t in f[which](None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        junk = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(20_000_000)  # about 10 ms on the current stream, then its writes
        for t in junk:
            t.fill_(7)
        del junk, t
        got = f[which](handle)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert ssd.query_status() == 0
