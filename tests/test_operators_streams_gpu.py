"""Calls on a stream that is not torch's current one: what they allocate is theirs.  Memory that the
current stream has freed but not finished writing must not come back as a result written by
another stream, nor a result that the current stream still reads as the next call's."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from test_linear_attention_gpu import gpu, make

pytestmark = pytest.mark.gpu


def attention_calls():
    x = gpu(make(2, 300, 4, 2, 64, 64, "bf16", seed=90))
    step = [x[n][:, 0].contiguous() for n in ("q", "k", "v", "log_decay")]
    gen = torch.Generator(device="cuda").manual_seed(9)
    logits = torch.randn(3, 4, 5003, generator=gen, device="cuda")
    scores = torch.randn(3, 4, generator=gen, device="cuda")
    return {
        "forward": lambda s: ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"],
                                                          stream=s),
        "backward": lambda s: ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"],
                                                            init_state=x["init"], dfinal_state=x["dfinal"], stream=s),
        "step": lambda s: (ssd.linear_attention_step(*step, x["init"].clone(), stream=s),) if s is None else
                          (ssd.linear_attention_step(*step, states.pop(), stream=s),),
        "select": lambda s: ssd.beam_select(logits, scores, stream=s),
    }, x


states = []


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("which", ["forward", "backward", "step", "select"])
def test_results_are_not_memory_in_use_by_the_current_stream(which, raw):
    calls, x = attention_calls()
    want = [t.clone() for t in calls[which](None)]
    states[:] = [x["init"].clone() for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        junk = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(20_000_000)  # about 10 ms on the current stream, then its writes
        for t in junk:
            t.fill_(7)
        del junk, t
        got = calls[which](side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("which", ["forward", "backward", "step", "select"])
def test_results_that_the_current_stream_reads_are_not_reused(which):
    calls, x = attention_calls()
    want = [t.clone() for t in calls[which](None)]
    states[:] = [x["init"].clone() for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = calls[which](side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    kept = [t.clone() for t in got]  # reads the results once the sleep is over
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):  # (writes what side's own pool gives)
        junk = [torch.empty(s, dtype=d, device="cuda").fill_(3) for s, d in shapes]
    torch.cuda.synchronize()
    assert len(junk) == len(want)
    for a, b in zip(kept, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("which", ["forward", "backward", "select"])
def test_a_capture_that_forks_to_another_stream(which):
    calls, x = attention_calls()
    want = [t.clone() for t in calls[which](None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = calls[which](side)
        torch.cuda.current_stream().wait_stream(side)
        sums = [t.float().sum() for t in got]
        del got
        side.wait_stream(torch.cuda.current_stream())
        got = calls[which](side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b.float().sum()) for a, b in zip(sums, want))
    assert ssd.query_status() == 0
