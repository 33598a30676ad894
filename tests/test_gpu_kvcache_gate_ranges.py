"""The gate's key rows of caches whose groups lie far apart or near the largest
values, against the 64-bit definition (tolerances as in test_gpu_kvcache.py)."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import long_context_prefill_attngate_b200 as seer
from test_gpu_kvcache import FORMATS, bf16, check_gate, gpu, make_cache, parts  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_of(bits, d, k, wk, maxmin):
    L = k.shape[2]
    cache, table = make_cache(1, 1, -(-L // 64), d, bits, False, 0)
    seer.seer_kv_write(cache, k.cuda(), k.cuda())
    kt = seer.seer_gate_key_cache_quant(cache, wk.cuda(), L, k_maxmin=maxmin)
    seer.seer_check_status()
    check_gate(kt, parts(cache, table)[0], wk, [L], 0, maxmin)


@pytest.mark.parametrize("bits,d", [(4, 128), (4, 64), (8, 128)])
@pytest.mark.parametrize("apart", [20, 45, 90, -45, -90])
@pytest.mark.parametrize("maxmin", [False, True])
def test_a_group_far_from_the_ones_that_the_weights_take(bits, d, apart, maxmin):
    """One group 2^apart times the others, and weights that are 0 for it."""
    G = ref.group(bits)
    k = bf16((1, 1, 300, d), 1).float()
    k[..., G:2 * G] *= 2.0 ** apart
    wk = bf16((1, 2 * d if maxmin else d, 32), 2, 0.1)
    for part in range(2 if maxmin else 1):
        wk[:, part * d + G:part * d + 2 * G] = 0
    rows_of(bits, d, k.to(torch.bfloat16), wk, maxmin)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("apart", [30, 60])
def test_tokens_far_apart(bits, d, apart):
    """Small tokens beside large ones of opposite sign: the mean is what is left."""
    k = bf16((1, 1, 128, d), 1).float() * 2.0 ** -apart
    k[:, :, 0], k[:, :, 64] = 1.0, -1.0
    k[:, :, 1], k[:, :, 65] = -1.0, 1.0
    rows_of(bits, d, k.to(torch.bfloat16), bf16((1, d, 32), 2, 0.1), False)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("e", [100, 119, 124, -80])
@pytest.mark.parametrize("maxmin", [False, True])
def test_blocks_of_values_near_the_largest_and_smallest(bits, d, e, maxmin):
    """A mean of 64 values below 2^126 is below it; the weights bring it back into range."""
    k = (bf16((1, 1, 200, d), 1).float().clamp(-3, 3) * 2.0 ** e + 2.0 ** e / 4).to(torch.bfloat16)
    wk = bf16((1, 2 * d if maxmin else d, 32), 2, 0.1).float()
    rows_of(bits, d, k, (wk * 2.0 ** (-e if e > 0 else 0)).to(torch.bfloat16), maxmin)
