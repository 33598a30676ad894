"""Refusals of the decode gate's and mask's lengths, on the CPU: nothing here
launches a kernel."""
import pytest
import torch

import long_context_prefill_attngate_b200 as seer


@pytest.mark.parametrize("lens", [torch.zeros(2, dtype=torch.int64), torch.zeros(3, dtype=torch.int32),
                                  torch.zeros((2, 1), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)[::2],
                                  torch.zeros(2, dtype=torch.int32, device="meta")])
def test_lens_is_checked(lens):
    q, wq = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((4, 64, 32), dtype=torch.bfloat16)
    kt, s = torch.zeros((2, 2, 4, 32)), torch.zeros((2, 4, 4))
    with pytest.raises(ValueError, match="lens"):
        seer.seer_decode_gate_scores_cached(q, kt, wq, 200, 2, lens=lens)
    with pytest.raises(ValueError, match="lens"):
        seer.seer_decode_block_mask(s, density=0.5, lens=lens)
