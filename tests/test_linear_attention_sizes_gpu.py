"""Head dimensions that are whole 16-byte rows but fill neither a 64-column tile nor a warp's 32 rows, on the
tensor-core kernel: prompt pass and gradients, one head and two heads to a product.  Tolerances as
in test_linear_attention_gpu.py."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from test_linear_attention_gpu import gpu, make
from test_linear_attention_paths_gpu import backward, check_all, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(2, 2), (4, 1), (3, 1)], ids=["own", "pairs", "odd"])
@pytest.mark.parametrize("N,P", [(8, 8), (24, 40), (40, 24), (72, 104), (104, 72), (120, 8), (8, 120), (128, 56), (56, 128),
                                 (64, 16), (96, 64)])
def test_sizes(N, P, heads):
    H, G = heads
    x = make(2, 135, H, G, N, P, "bf16", seed=N + P)
    d = gpu(x)
    ssd.set_path(ssd.PATH_TC)
    try:
        y, fin = forward(d)
        grads = backward(d)
        torch.cuda.synchronize()
    finally:
        ssd.set_path(ssd.PATH_AUTO)
    assert ssd.query_status() == 0
    check_all(x, y, fin, grads)
