"""A kernel wait that runs out where the loads of a whole list of units have already been issued (a
few blocks, one unit to a CTA), so that the load warp itself has nothing left to wait for: the call
reports it and the next ones are right."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from test_linear_attention_gpu import gpu, make
from test_linear_attention_paths_gpu import backward, check_all, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["forward", "backward"])
@pytest.mark.parametrize("T", [1, 64, 128, 190])
def test_a_short_list_that_times_out(T, which):
    x = make(2, T, 2, 2, 64, 64, "bf16", seed=80)
    d = gpu(x)
    assert ssd.query_status() == 0
    for limit in (20_000_000, 200_000):  # about 10 ms and 0.1 ms per wait
        ssd.set_test_hooks(wait_limit_cycles=limit, withhold_product=True)
        try:
            forward(d) if which == "forward" else backward(d)
            torch.cuda.synchronize()
        finally:
            ssd.set_test_hooks()
        assert ssd.query_status() == 5  # SSD_ERR_DEVICE_TIMEOUT
        y, fin = forward(d)
        check_all(x, y, fin, backward(d))
        assert ssd.query_status() == 0
