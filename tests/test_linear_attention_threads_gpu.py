"""Linear attention from several host threads at once, each on its own stream: the same bits as one
call alone."""
import threading

import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from test_linear_attention_gpu import gpu, make
from test_linear_attention_paths_gpu import backward, forward

pytestmark = pytest.mark.gpu


def test_threads():
    xs = [gpu(make(*s, seed=60 + i)) for i, s in enumerate([
        (2, 300, 4, 2, 64, 64, "bf16"), (1, 1000, 2, 2, 128, 128, "bf16"), (2, 150, 3, 1, 40, 24, "f32"),
        (1, 500, 4, 1, 128, 64, "bf16")])] + [gpu(make(1, 0, 4, 2, 64, 128, "bf16", lengths=[1, 700, 0, 300], seed=64))]
    want = [forward(x) + backward(x) for x in xs]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(xs))

    def run(x, w):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(60):
                    got = forward(x) + backward(x)
                    stream.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, w))
        except BaseException as e:  # noqa: B036  (reported by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=a) for a in zip(xs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert ssd.query_status() == 0
