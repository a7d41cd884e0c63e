"""An end token that does not fit 32 bits is refused, not taken modulo 2^32 (no GPU needed)."""
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd


@pytest.mark.parametrize("eos", [2 ** 31, 2 ** 32 + 2, -2 ** 31 - 1, 2 ** 63])
def test_end_tokens_beyond_32_bits(eos):
    with pytest.raises(ValueError, match="eos"):
        ssd.beam_select(torch.zeros(1, 2, 5), torch.zeros(1, 2), eos=eos)
