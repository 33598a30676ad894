"""Calls on the quantised cache that a program may make in other ways than the
plain one: workspaces, two calls at once."""
import threading

import pytest
import torch

import long_context_prefill_attngate_b200 as seer
from test_gpu_kvcache import attend, bf16, gpu, make_cache  # noqa: F401

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


def test_gate_keys_of_two_widths_from_two_threads():
    """A call of one d_gate between another's set-up and its launch changes nothing."""
    B, Hkv, L, d = 1, 2, 200, 128
    cache, table = make_cache(B, Hkv, 4, d, 4, False, 0)
    seer.seer_kv_write(cache, bf16((B, Hkv, L, d), 1).cuda(), bf16((B, Hkv, L, d), 2).cuda())
    wk = {dg: bf16((Hkv, d, dg), dg, 0.1).cuda() for dg in (4, 256)}
    want = {dg: seer.seer_gate_key_cache_quant(cache, wk[dg], L) for dg in wk}
    torch.cuda.synchronize()
    errors, got = [], {}

    def work(dg):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3000):
                    got[dg] = seer.seer_gate_key_cache_quant(cache, wk[dg], L)
        except Exception as e:                              # noqa: BLE001 (told below, in the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(dg,)) for dg in (4, 256, 4, 256)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(torch.equal(got[dg], want[dg]) for dg in wk)
