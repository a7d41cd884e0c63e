"""Selections of different sizes from several host threads at once: each call gets the shared memory it
asks for, whatever another thread's call asked for meanwhile."""
import threading

import pytest
import torch

import ssd_sequence_mixing_b200 as ssd

pytestmark = pytest.mark.gpu


# batch, beams, count, vocab, calls of a thread
SMALL = [(1, 2, c, 500, 4000) for c in (64, 53, 58, 64)]  # 66, 46 and 54 KB in the merge
LARGE = [(20, c, c, 32000, 300) for c in (64, 45, 52)]    # 70, 49 and 57 KB of candidates a block


@pytest.mark.parametrize("sizes", [SMALL, LARGE], ids=["small", "large"])
def test_threads_with_different_counts(sizes):
    gen = torch.Generator(device="cuda").manual_seed(5)
    work = []
    for batch, beams, count, vocab, calls in sizes:
        logits = torch.randn(batch, beams, vocab, generator=gen, device="cuda").bfloat16()
        scores = torch.randn(batch, beams, generator=gen, device="cuda")
        work.append((logits, scores, count, calls, ssd.beam_select(logits, scores, count=count)))
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(work))

    def run(logits, scores, count, calls, want):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(calls):
                    got = ssd.beam_select(logits, scores, count=count)
            stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        except BaseException as e:  # noqa: B036  (reported by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
