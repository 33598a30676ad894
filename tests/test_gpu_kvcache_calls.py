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


@pytest.mark.parametrize("what", ["start", "start_pos", "table"])
def test_rows_that_the_cache_does_not_have_read_as_zero(what):
    """Where the call makes the output, not what the memory held before: rows behind the cache, below 0 and on a page
    that the table does not have; a device error besides."""
    B, Hkv, d, n = 1, 2, 128, 100
    cache, table = make_cache(B, Hkv, 2, d, 4, what == "table", 0)
    k = bf16((B, Hkv, 128, d), 1).cuda()
    seer.seer_kv_write(cache, k, k)
    held = seer.seer_kv_read(cache, 128)[0]
    args, at = {}, 0
    if what == "table":
        cache.block_table[0, 1] = -1
    elif what == "start":
        args, at = dict(start=torch.tensor([64], dtype=torch.int32, device="cuda")), 64
    else:
        args, at = dict(start_pos=64), 64
    torch.cuda.synchronize()
    for _ in range(4):                                      # what the allocator hands out next
        a = [torch.full((B, Hkv, n, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        del a
    out = seer.seer_kv_read(cache, n, **args)
    with pytest.raises(seer.SeerError):
        seer.seer_check_status()
    for t in out:
        assert torch.equal(t[:, :, :64], held[:, :, at:at + 64]) and not t[:, :, 64:].any()
    whole = seer.seer_kv_read(cache, 64)
    seer.seer_check_status()
    assert torch.equal(whole[0], held[:, :, :64])
