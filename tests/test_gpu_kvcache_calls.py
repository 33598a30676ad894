"""Calls on the quantised cache that a program may make in other ways than the
plain one: workspaces, two calls at once."""
import pytest
import torch

import long_context_prefill_attngate_b200 as seer
from test_gpu_kvcache import attend, gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def test_workspace_of_another_device_is_refused():
    """On the host, before any launch."""
    cache, q, mask, o, lse = attend(4, 128, 2, 8, 2, 900, 0.3, seed=21)
    need = seer.seer_workspace_bytes(seer.SEER_CALL_BLOCK_SPARSE_DECODE_QUANT, seer.seer_shape(2, 8, 2, 900, 128))
    with pytest.raises(ValueError, match="workspace"):
        seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), 900, workspace=torch.empty(need, dtype=torch.uint8))
    o2 = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), 900,
                                             workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    seer.seer_check_status()
    assert torch.equal(o, o2)
