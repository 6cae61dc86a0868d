"""Sizes beyond 32 bits of tensors that hold nothing."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV

pytestmark = pytest.mark.gpu


def test_no_elements_and_a_size_beyond_32_bits():
    """2^32 + 1 rows of no token are not the one row that 32 bits make of them, whose state
    alone would be written."""
    many = (1 << 32) + 1
    p, taps = torch.zeros(8, device=DEV), torch.zeros(8, 4, device=DEV)
    x = torch.zeros(many, 0, 8, device=DEV)
    for call in (lambda: kda.gated_scan_fwd(x, x, x, p, p, output_final_state=False),
                 lambda: kda.short_conv_fwd(x, taps, output_final_state=False)):
        with pytest.raises(kda.LibKdaError):
            call()
    assert kda.layer_norm_fwd(x, p)[0].shape == (many, 0, 8)  # (no rows at all)
