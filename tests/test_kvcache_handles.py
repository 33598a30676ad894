"""What the quantised-cache calls refuse of the handles that they are given, on
the CPU: nothing here launches a kernel."""
import pytest
import torch

import long_context_prefill_attngate_b200 as seer


@pytest.fixture
def cache():
    return seer.SeerKVCache.empty(2, 2, 200, 128, bits=4, device="cpu")


def test_workspace_is_checked_like_every_other_tensor(cache):
    q, m = torch.zeros((2, 4, 128), dtype=torch.bfloat16), torch.zeros((2, 4, 4), dtype=torch.uint8)
    need = seer.seer_workspace_bytes(seer.SEER_CALL_BLOCK_SPARSE_DECODE_QUANT, seer.seer_shape(2, 4, 2, 200, 128))
    with pytest.raises(ValueError, match="workspace"):
        seer.seer_block_sparse_decode_quant(q, cache, m, 200, workspace=torch.empty(2 * need, dtype=torch.uint8)[::2])
    with pytest.raises(ValueError, match="CUDA"):           # a good one: the cache is what is refused
        seer.seer_block_sparse_decode_quant(q, cache, m, 200, workspace=torch.empty(need, dtype=torch.uint8))


@pytest.mark.parametrize("name", ["pages", "block_table", "d", "bits", "Hkv", "B", "max_blocks"])
def test_a_cache_keeps_its_tensors_and_sizes(name):
    """The calls hold the tensors' addresses: what they were made from is not exchanged behind them."""
    pages = torch.zeros((8, 2, seer.seer_kv_record_bytes(4, 128)), dtype=torch.uint8)
    table = torch.arange(8, dtype=torch.int32).view(2, 4)
    c = seer.SeerKVCache(pages, 128, 4, block_table=table)
    was = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, {"pages": pages.clone(), "block_table": table.flip(1)}.get(name, 64))
    assert getattr(c, name) is was
    assert c.pages is pages and c.block_table is table and (c.d, c.bits, c.Hkv, c.B, c.max_blocks) == (128, 4, 2, 2, 4)
    c.block_table[0, 0] = 7                                 # their contents may change
    assert table[0, 0] == 7


@pytest.mark.parametrize("shape,stride", [((128, 64), 128 * 64), ((2, 128, 64), 2 * 128 * 64), ((2, 128, 64), 128 * 64 + 1),
                                          ((2, 128, 64), -8)])
def test_a_head_stride_that_leads_out_of_the_weights_is_refused(cache, shape, stride):
    wk = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="wk_head_stride"):
        seer.seer_gate_key_cache_quant(cache, wk, 200, wk_head_stride=stride)


@pytest.mark.parametrize("stride", [0, 64, 128 * 64])
def test_a_head_stride_within_the_weights_is_taken(cache, stride):
    with pytest.raises(ValueError, match="CUDA"):           # the cache is what is refused
        seer.seer_gate_key_cache_quant(cache, torch.zeros((2, 128, 64), dtype=torch.bfloat16), 200, wk_head_stride=stride)


def test_a_stream_of_another_device_is_refused():
    """What is given as the stream decides nothing else: the call would have run on the other device's current stream."""
    from long_context_prefill_attngate_b200 import kvcache

    class Stream:
        cuda_stream, device_index = 0, 1

    with pytest.raises(ValueError, match="stream"):
        kvcache._elsewhere(lambda: None, 0, Stream())


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1])
def test_positions_of_more_than_32_bits_are_refused(cache, n):
    """The C calls take ints: what does not fit would have named another position."""
    k = torch.zeros((2, 2, 5, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="start_pos"):
        seer.seer_kv_write(cache, k, k, start_pos=n)
    with pytest.raises(ValueError, match="start_pos"):
        seer.seer_kv_read(cache, 5, start_pos=n)
    with pytest.raises(ValueError, match="first_block"):
        seer.seer_gate_key_cache_quant(cache, torch.zeros((2, 128, 64), dtype=torch.bfloat16), 200, first_block=n)
