"""A call whose scratch does not fit the GPU fails by itself: the next calls, the library's and torch's,
are not told of it."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from test_linear_attention_gpu import gpu, make

pytestmark = pytest.mark.gpu


def test_the_next_call_is_not_told():
    x = gpu(make(1, 200, 4, 2, 128, 128, "bf16", init=False, seed=7))
    want = ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"])
    # a million empty sequences: a state for each is more than any GPU holds
    cu = torch.full(((1 << 20) + 1,), 200, dtype=torch.int32, device="cuda")
    cu[0] = 0
    for _ in range(2):
        with pytest.raises(ssd.SsdError) as e:
            ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], cu_seqlens=cu)
        assert e.value.code == 4  # SSD_ERR_CUDA
        got = ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with pytest.raises(ssd.SsdError):
            ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], cu_seqlens=cu)
        assert int((torch.ones(1000, device="cuda") + 1).sum()) == 2000
        torch.cuda.synchronize()
    assert ssd.query_status() == 0


def test_no_entry_point_is_told():
    x = gpu(make(1, 200, 4, 2, 128, 128, "bf16", init=True, seed=7))
    cu = torch.full(((1 << 20) + 1,), 200, dtype=torch.int32, device="cuda")
    cu[0] = 0
    gen = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    z, dt, A = r(4, 2048, 16, 64).bfloat16(), 0.1 * r(4, 2048, 16).abs(), -r(16).abs()
    B, C, D = r(4, 2048, 1, 128).bfloat16(), r(4, 2048, 1, 128).bfloat16(), r(16)
    part = lambda t, n: t[:, :n].contiguous()
    small = [part(t, 130) for t in (z, dt, B, C)]
    state, state2, taps, one = r(4, 16, 64, 128), r(1, 4, 128, 128), r(1024, 4), [t[:, 0].contiguous() for t in (z, dt, B, C)]
    logits, scores, parents = r(2, 3, 5000), r(2, 3), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    tok = [x[n][:, 0].contiguous() for n in ("q", "k", "v", "log_decay")]
    calls = [
        lambda: ssd.ssd_forward(z, dt, A, B, C, D, None, None, 128),
        lambda: ssd.ssd_forward(small[0], small[1], A, small[2], small[3], D, None, None, 64),
        lambda: ssd.ssd_forward(small[0].float(), small[1], A, small[2].float(), small[3].float(), D, None, None, 64),
        lambda: ssd.ssd_final_state(z, dt, A, B),
        lambda: ssd.ssd_forward_dt(z, dt, A, B, C, D),
        lambda: ssd.ssd_forward_noalloc(part(small[0], 40), part(small[1], 40), A, part(small[2], 40), part(small[3], 40), D),
        lambda: ssd.ssd_decode_step(one[0], one[1], A, one[2], one[3], D, state),
        lambda: ssd.causal_conv1d_silu(z.reshape(4, 2048, 1024), taps),
        lambda: ssd.gated_rmsnorm(z.reshape(4, 2048, 1024), z.reshape(4, 2048, 1024), r(1024)),
        lambda: ssd.segment_logdecay(dt[:1], A),
        lambda: ssd.state_prefix(2, state, -dt[0, :4].contiguous()),
        lambda: ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"]),
        lambda: ssd.linear_attention_forward(x["q"].float(), x["k"].float(), x["v"].float(), x["log_decay"]),
        lambda: ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"]),
        lambda: ssd.linear_attention_step(*tok, state2),
        lambda: ssd.beam_select(logits, scores),
        lambda: ssd.state_reorder(r(4, 8), parents),
    ]
    for f in calls:
        f()
        with pytest.raises(ssd.SsdError):
            ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], cu_seqlens=cu)
        f()
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
