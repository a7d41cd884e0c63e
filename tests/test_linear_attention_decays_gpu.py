"""Decays of all kinds in the gradients of bf16 operands, and long runs of resets followed by weak decays
in both directions, on both kernels.  Tolerances as in test_linear_attention_gpu.py; where log-decays
of a block sum to thousands the prompt pass's factors 2^(c_i - c_j) come from sums of up to 9600
held to 2^-11 each, 2^-10 ln 2 = 7e-4 of a factor: a sixth of the half step, 2^-8, that the same
product's rounding is held to, and within the margin of the three roundings' 3.9e-3 to 5e-3."""
import numpy as np
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd
from oracle import attention
from test_linear_attention_gpu import close, gpu, make, reference

pytestmark = pytest.mark.gpu

SHAPES = {"pairs": (2, 300, 4, 2, 64, 64), "wide": (1, 200, 2, 2, 128, 128), "shared": (2, 190, 6, 1, 128, 64)}
PATHS = {"tensor_core": ssd.PATH_AUTO, "general": ssd.PATH_SIMT}


def with_decays(shape, kind, dtype="bf16"):
    x = make(*shape, dtype, seed=3)
    ld = x["log_decay"]
    if kind == "none":
        ld.zero_()
    elif kind == "strong":
        ld.mul_(30)
    elif kind == "resets":
        ld[:, ::7] = -float("inf")
    elif kind == "mixed":
        ld.mul_(1e-3)
        ld[:, 50::97] = -1e30
        ld[:, 51::97] = -float("inf")
    else:  # 40 tokens of each block of 64 forget everything, the others hardly anything
        ld.mul_(1e-3)
        at = torch.arange(ld.shape[1]) % 64
        ld[:, (at < 40) if kind == "run_first" else (at >= 24)] = -float("inf")
    return x


@pytest.fixture(params=list(PATHS))
def path(request):
    ssd.set_path(PATHS[request.param])
    yield request.param
    ssd.set_path(ssd.PATH_AUTO)


@pytest.mark.parametrize("kind", ["run_first", "run_last"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_forward_of_many_resets(shape, kind, path):
    x = with_decays(SHAPES[shape], kind)
    _, _, _, y_ref, fin_ref = reference(x)
    d = gpu(x)
    y, fin = ssd.linear_attention_forward(d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"])
    close("y", y, y_ref, "bf16")
    close("final_state", fin, fin_ref, "f32")


@pytest.mark.parametrize("decays", [True, False], ids=["all", "without_dlog"])
@pytest.mark.parametrize("kind", ["none", "strong", "resets", "mixed", "run_first", "run_last"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_backward(shape, kind, decays, path):
    x = with_decays(SHAPES[shape], kind)
    f, i, dfin, _, _ = reference(x)
    ref = attention.backward(f["dy"], f["q"], f["k"], f["v"], f["log_decay"], x["scale"], i, dfin, x["offsets"])
    d = gpu(x)
    got = ssd.linear_attention_backward(d["dy"], d["q"], d["k"], d["v"], d["log_decay"], init_state=d["init"],
                                        dfinal_state=d["dfinal"], need_dlog_decay=decays)
    for name, g, r in zip(("dq", "dk", "dv"), got, ref):
        close(name, g, r, "bf16")
    close("dinit_state", got[4], ref[4], "f32")
    if not decays:
        return
    # a difference of sums, each to fp32's accuracy: held to their size
    T, H = ref[3].shape
    dots = np.repeat((f["q"] * ref[0]).sum(-1), H // x["q"].shape[2], axis=-1)
    size = np.linalg.norm(dots) + np.linalg.norm(np.einsum("rhpn,rhpn->rh", np.abs(dfin), np.abs(i)))
    off = np.linalg.norm(got[3].double().cpu().numpy().reshape(T, H) - ref[3])
    assert off <= 2e-5 * (size + np.linalg.norm(ref[3])), off / (size + np.linalg.norm(ref[3]))
    zero = torch.isneginf(d["log_decay"])
    assert (got[3][zero] == 0).all()
