"""Without an initial state the first token's decay of every sequence acts on nothing: its gradient is
zero, not the rounding of the two sums whose difference it is."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from test_linear_attention_gpu import gpu, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch", [(2, 1, None), (3, 200, None), (1, 3000, None), (1, 0, [1, 0, 70, 700, 1])],
                         ids=["one", "short", "long", "packed"])
def test_first_decay(batch, dtype):
    b, T, lengths = batch
    x = make(b, T, 4, 2, 64, 64, dtype, init=False, lengths=lengths, seed=21)
    d = gpu(x)
    dfinal = torch.randn(x["offsets"].size - 1, 4, 64, 64, device="cuda")
    got = ssd.linear_attention_backward(d["dy"], d["q"], d["k"], d["v"], d["log_decay"], dfinal_state=dfinal,
                                        cu_seqlens=d["cu"])[3].reshape(-1, 4)
    off = x["offsets"]
    first = sorted({int(a) for a, e in zip(off[:-1], off[1:]) if e > a})
    assert (got[first] == 0).all()
    others = [t for t in range(got.shape[0]) if t not in first]
    assert (got[others] != 0).all()
    # constant decays: a batch of single tokens has no gradient at all
    if T == 1:
        const = d["log_decay"][0, 0].contiguous()
        assert not ssd.linear_attention_backward(d["dy"], d["q"], d["k"], d["v"], const, dfinal_state=dfinal)[3].any()
