"""Linear attention beyond the ordinary call: a kernel wait that runs out, the general kernel on
bf16 operands, batches of which only some sequences are cut into windows, arrays past 2^31
elements, and calls that run at the same time.  Tolerances as in test_linear_attention_gpu.py."""
import numpy as np
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from oracle import attention
from test_linear_attention_gpu import close, gpu, make, reference, sizes

pytestmark = pytest.mark.gpu


def forward(x):
    return ssd.linear_attention_forward(x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"], cu_seqlens=x["cu"])


def backward(x):
    return ssd.linear_attention_backward(x["dy"], x["q"], x["k"], x["v"], x["log_decay"], init_state=x["init"],
                                         dfinal_state=x["dfinal"], cu_seqlens=x["cu"])


def check_all(x, y, fin, grads, dtype="bf16"):
    f, i, dfin, y_ref, fin_ref = reference(x)
    ref = attention.backward(f["dy"], f["q"], f["k"], f["v"], f["log_decay"], x["scale"], i, dfin, x["offsets"])
    z = sizes(x)
    fz, iz, dz, y_size, _ = reference(z)
    size = attention.backward(fz["dy"], fz["q"], fz["k"], fz["v"], fz["log_decay"], x["scale"], iz, dz, x["offsets"])
    close("y", y, y_ref, dtype, size=y_size)
    close("final_state", fin, fin_ref, "f32")
    for name, g, r, m in zip(("dq", "dk", "dv"), grads, ref, size):
        close(name, g, r, dtype, size=m)
    close("dlog_decay", grads[3], ref[3], "f32", 2e-5)
    if x["init"] is not None:
        close("dinit_state", grads[4], ref[4], "f32")


@pytest.mark.parametrize("which", ["forward", "backward"])
def test_a_withheld_product_times_out_and_the_next_call_is_correct(which):
    x = make(2, 130, 2, 2, 64, 64, "bf16", seed=30)
    d = gpu(x)
    assert ssd.query_status() == 0
    ssd.set_test_hooks(wait_limit_cycles=20_000_000, withhold_product=True)  # about 10 ms per wait
    try:
        forward(d) if which == "forward" else backward(d)
        torch.cuda.synchronize()
    finally:
        ssd.set_test_hooks()
    assert ssd.query_status() == 5  # SSD_ERR_DEVICE_TIMEOUT
    assert ssd.query_status() == 0  # read and cleared
    y, fin = forward(d)
    check_all(x, y, fin, backward(d))
    assert ssd.query_status() == 0


@pytest.mark.parametrize("case", [(1, 1, 1, 1, 8, 8, None), (2, 65, 4, 2, 128, 64, None), (1, 1100, 2, 1, 64, 128, None),
                                  (1, 0, 4, 1, 64, 64, [0, 1, 129, 0, 300])], ids=lambda c: "x".join(map(str, c[:6])))
def test_bf16_on_the_general_kernel(case):
    b, T, H, G, N, P, lengths = case
    x = make(b, T, H, G, N, P, "bf16", lengths=lengths, seed=31)
    d = gpu(x)
    ssd.set_path(ssd.PATH_SIMT)
    try:
        y, fin = forward(d)
        grads = backward(d)
        torch.cuda.synchronize()
    finally:
        ssd.set_path(ssd.PATH_AUTO)
    assert ssd.query_status() == 0
    check_all(x, y, fin, grads)


def test_the_tensor_core_path_refuses_what_it_cannot_take():
    ssd.set_path(ssd.PATH_TC)
    try:
        for shape in ((1, 4, 2, 1, 64, 64, "f32"), (1, 4, 2, 1, 60, 64, "bf16"), (1, 4, 2, 1, 64, 36, "bf16")):
            x = gpu(make(*shape, seed=32))
            for call in (forward, backward):
                with pytest.raises(ssd.SsdError) as e:
                    call(x)
                assert e.value.code == 2  # SSD_ERR_UNSUPPORTED
    finally:
        ssd.set_path(ssd.PATH_AUTO)


def test_some_sequences_of_a_batch_are_cut():
    """One sequence more than the GPU has SMs: all but the last ones run whole, those as windows.
    The reference is formed for the first two and the last four sequences."""
    rows = torch.cuda.get_device_properties(0).multi_processor_count + 1
    x = make(rows, 1500, 1, 1, 64, 128, "bf16", seed=33)
    y, fin = forward(gpu(x))
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    for part in (slice(0, 2), slice(rows - 4, rows)):
        z = {n: v[part] if isinstance(v, torch.Tensor) else v for n, v in x.items()}
        z["offsets"] = np.arange(z["q"].shape[0] + 1) * 1500
        _, _, _, y_ref, fin_ref = reference(z)
        close("y", y[part], y_ref, "bf16")
        close("final_state", fin[part], fin_ref, "f32")


def test_some_sequences_of_a_training_batch_are_cut():
    """The same for the gradients, whose three passes share the SMs: a third as many sequences."""
    rows = torch.cuda.get_device_properties(0).multi_processor_count // 3 + 1
    x = make(rows, 1500, 1, 1, 64, 64, "bf16", seed=34)
    got = backward(gpu(x))
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    for part in (slice(0, 1), slice(rows - 3, rows)):
        z = {n: v[part] if isinstance(v, torch.Tensor) else v for n, v in x.items()}
        z["offsets"] = np.arange(z["q"].shape[0] + 1) * 1500
        f, i, dfin, _, _ = reference(z)
        ref = attention.backward(f["dy"], f["q"], f["k"], f["v"], f["log_decay"], x["scale"], i, dfin, z["offsets"])
        for name, g, r in zip(("dq", "dk", "dv"), got, ref):
            close(name, g[part], r, "bf16")
        close("dlog_decay", got[3][part], ref[3], "f32", 2e-5)
        close("dinit_state", got[4][part], ref[4], "f32")


def test_two_heads_share_query_and_key_where_one_is_spoiled():
    """Two heads of 64 rows or fewer run side by side in one product: NaN in one stays there."""
    x = gpu(make(1, 200, 4, 1, 128, 40, "bf16", seed=35))
    y0, f0 = forward(x)
    x["v"][0, 100:150, 1] = float("nan")
    y1, f1 = forward(x)
    keep = [0, 2, 3]
    assert torch.equal(y0[:, :, keep], y1[:, :, keep]) and torch.equal(f0[:, keep], f1[:, keep])
    # a block is 64 tokens: what comes before the one that holds token 100 stays
    assert torch.equal(y0[:, :64, 1], y1[:, :64, 1]) and torch.isnan(f1[:, 1]).any()


def test_arrays_past_two_to_the_31_elements():
    """A packed batch of two sequences, the first so long that the second begins past 2^31
    elements of v; zeros but for the second, which is checked in full, and the first's state."""
    H, P, N, tail = 64, 128, 64, 150
    head = (1 << 31) // (H * P) + 77
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    z = make(1, tail, H, 1, N, P, "bf16", seed=36)
    T = head + tail
    x = {"q": torch.zeros(1, T, 1, N, dtype=torch.bfloat16, device="cuda")}
    x["k"] = torch.zeros_like(x["q"])
    x["v"] = torch.zeros(1, T, H, P, dtype=torch.bfloat16, device="cuda")
    x["dy"] = torch.zeros_like(x["v"])
    x["log_decay"] = torch.full((1, T, H), -1e-3, device="cuda")
    for n in ("q", "k", "v", "dy", "log_decay"):
        x[n][:, head:] = z[n].cuda()
    first = torch.ones(1, H, P, N)
    x["init"] = torch.cat([first, z["init"]]).cuda()
    x["dfinal"] = torch.cat([torch.zeros_like(first), z["dfinal"]]).cuda()
    x["cu"] = torch.tensor([0, head, T], dtype=torch.int32, device="cuda")
    y, fin = forward(x)
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    f, i, dfin, y_ref, fin_ref = reference(z)
    close("y", y[:, head:], y_ref, "bf16")
    close("final_state", fin[1:], fin_ref, "f32")
    assert not y[:, :head].any()
    assert fin[0].abs().max() < 1e-30  # exp(-262): a state that only decays
    del y, fin
    got = backward(x)
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    ref = attention.backward(f["dy"], f["q"], f["k"], f["v"], f["log_decay"], z["scale"], i, dfin, z["offsets"])
    for name, g, r in zip(("dq", "dk", "dv"), got, ref):
        close(name, g[:, head:], r, "bf16")
        assert not g[:, :head].any(), name
    close("dlog_decay", got[3][:, head:], ref[3], "f32", 2e-5)
    close("dinit_state", got[4][1:], ref[4], "f32")


def test_calls_that_run_at_the_same_time():
    """Prompt passes, gradients and steps of different shapes on four streams at once."""
    shapes = [(2, 900, 8, 2, 64, 128, "bf16"), (1, 1300, 4, 4, 128, 128, "bf16"), (3, 200, 6, 1, 40, 24, "f32"),
              (4, 500, 16, 1, 128, 64, "bf16")]
    xs = [gpu(make(*s, seed=40 + n)) for n, s in enumerate(shapes)]
    want = [forward(x) + backward(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(forward(x) + backward(x))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert ssd.query_status() == 0


def test_packed_batches_at_the_same_time_and_replayed():
    """Packed batches, whose windows go to whichever CTA is free, on three streams at once and as
    replayed graphs: the same bits as one call alone."""
    lens = [[1, 2500, 0, 700, 64, 1200], [3000, 3, 129], [40] * 50]
    xs = [gpu(make(1, 0, 4, 2, 64, 128, "bf16", lengths=n, seed=50 + i)) for i, n in enumerate(lens)]
    want = [forward(x) + backward(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(forward(x) + backward(x))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(forward(x) + backward(x))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    assert ssd.query_status() == 0


def test_overlapping_outputs_are_refused_and_two_buffers_taken_in_turn():
    x = make(1, 700, 2, 1, 64, 64, "bf16", seed=60)
    d = gpu(x)
    with pytest.raises(ssd.SsdError):
        ssd.linear_attention_forward(d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"], final_state=d["init"])
    with pytest.raises(ssd.SsdError):
        ssd.linear_attention_forward(d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"], y=d["v"])
    # one sequence in two calls, each in a buffer of its own
    part = lambda a, b, s: ssd.linear_attention_forward(
        *(d[n][:, a:b].clone(memory_format=torch.contiguous_format) for n in ("q", "k", "v", "log_decay")), init_state=s)
    y0, mid = part(0, 384, d["init"])
    y1, fin = part(384, 700, mid)
    _, _, _, y_ref, fin_ref = reference(x)
    close("y", torch.cat([y0, y1], dim=1), y_ref, "bf16")
    close("final_state", fin, fin_ref, "f32")
