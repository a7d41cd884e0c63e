"""Linear attention refuses outputs that share bytes with an input or another output, before
anything is launched (no GPU needed)."""
import ctypes

import pytest

import ssd_sequence_mixing_b200 as ssd
from test_operators_boundary import backward, forward, shape, step

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
