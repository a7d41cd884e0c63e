"""Reordering of more small rows than one launch has blocks: all buffers are moved, whatever the
sizes of the others in the call."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd

pytestmark = pytest.mark.gpu


def test_more_blocks_than_a_launch_has():
    batch, beams, small = 1 << 24, 2, 128  # 128 buffers of a block per batch item: 2^31 blocks
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    gen = torch.Generator(device="cuda").manual_seed(3)
    parents = torch.randint(beams, (batch, beams), generator=gen, device="cuda", dtype=torch.int32)
    wide = torch.randint(1 << 30, (batch * beams, 4), generator=gen, device="cuda", dtype=torch.int32)
    bytes_ = torch.randint(256, (small, batch * beams), generator=gen, device="cuda", dtype=torch.uint8)
    wide_was, bytes_was = wide.clone(), bytes_.clone()
    ssd.state_reorder([wide] + list(bytes_), parents)
    torch.cuda.synchronize()
    assert ssd.query_status() == 0
    source = (torch.arange(batch, device="cuda")[:, None] * beams + parents).reshape(-1)
    assert torch.equal(wide, wide_was[source])
    for now, was in zip(bytes_, bytes_was):
        assert torch.equal(now, was[source])
