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
