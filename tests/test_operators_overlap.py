"""Linear attention and beam selection refuse outputs that share bytes with an input or another
output, and reordering buffers that hold its parents, before anything is launched (no GPU needed)."""
import ctypes

import pytest

import ssd_sequence_mixing_b200 as ssd
from test_operators_boundary import backward, forward, select, shape, step

# 2 sequences of 300 tokens, 4 heads of 64, 2 groups of 128, bf16
QK, VY, DECAY, STATE = 2 * 300 * 2 * 128 * 2, 2 * 300 * 4 * 64 * 2, 2 * 300 * 4 * 4, 2 * 4 * 64 * 128 * 4
SIZE = dict(q=QK, k=QK, v=VY, dy=VY, y=VY, log_decay=DECAY, init=STATE, final=STATE, dfinal=STATE, dq=QK, dk=QK, dv=VY,
            dlog=DECAY, dinit=STATE, state=STATE)
INPUTS = {"forward": ("q", "k", "v", "log_decay", "init"), "step": ("q", "k", "v", "log_decay"),
          "backward": ("dy", "q", "k", "v", "log_decay", "init", "dfinal")}
OUTPUTS = {"forward": ("y", "final"), "step": ("y", "state"), "backward": ("dq", "dk", "dv", "dlog", "dinit")}
CALL = {"forward": forward, "backward": backward, "step": step}


def places(which):
    at, out = 1 << 20, {}
    for n in INPUTS[which] + OUTPUTS[which]:
        out[n] = at
        at += SIZE[n] + 15 & ~15  # side by side
    return out


@pytest.mark.parametrize("which", list(CALL))
def test_overlaps_are_refused(which):
    s = shape(batch=2, seqlen=1) if which == "step" else shape(batch=2)
    size = dict(SIZE)
    if which == "step":
        size.update(q=QK // 300, k=QK // 300, v=VY // 300, y=VY // 300, log_decay=DECAY // 300)
    for out in OUTPUTS[which]:
        for other in INPUTS[which] + OUTPUTS[which]:
            if other == out:
                continue
            # the same place; the last 16 bytes of one on the first of the other, and the reverse
            for shift in (0, size[other] - 16, 16 - size[out]):
                at = places(which)
                at[out] = at[other] + shift
                assert CALL[which](s, **{n: ctypes.c_void_p(a) for n, a in at.items()}) == 1, (out, other, shift)


def test_selection_and_reordering():
    # 2 x 4 rows of 100 fp32 logits, count 4
    size = dict(logits=3200, scores=32, finished=8, s=32, t=32, p=32)
    places, at = {}, 1 << 20
    for n in size:
        places[n] = at
        at += size[n] + 15 & ~15
    for out in ("s", "t", "p"):
        for other in size:
            if other == out:
                continue
            for shift in (0, size[other] - 16 & ~15, 16 - size[out]):
                a = {n: ctypes.c_void_p(v) for n, v in {**places, out: places[other] + shift}.items()}
                assert select(eos=1, **a) == 1, (out, other, shift)
    ptrs, rows = (ctypes.c_void_p * 1)(1 << 20), (ctypes.c_int64 * 1)(64)  # 8 rows of 64 bytes
    for parents in ((1 << 20), (1 << 20) + 508, (1 << 20) - 28):
        rc = ssd.library().ssd_state_reorder(2, 4, ctypes.c_void_p(parents), 1, ptrs, rows, None)
        assert rc == 1, parents
