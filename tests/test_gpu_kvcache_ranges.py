"""The quantised decode attention and row writer where the values of a group, a
token, a head or a block lie far apart, against the 64-bit definition.

Tolerances, from the arithmetic: p s enters the products in parts that leave at
most 2^-16 of it, scores are fp32 sums (e as in test_gpu_kvcache.py), and every
other sum of the output is fp32 over at most N tokens.  So o is within
2^-8 |o| + 2 (2^-16 + e + N 2^-24) sum p (s n + |z|) of the definition.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import long_context_prefill_attngate_b200 as seer
from test_gpu_kvcache import FORMATS, bf16, f64, gpu, make_cache, parts, shared  # noqa: F401

pytestmark = pytest.mark.gpu
# heads of a CTA: two, four, eight, and sixteen (for a batch)
HEADS = [(1, 2), (1, 4), (1, 8), (150, 16)]


def check(o, lse, q, kv, mask, lens, which=None, scale=None):
    B, _, d = q.shape
    for b in range(B) if which is None else which:
        want, wl, A, E = ref.decode(f64(q[b:b + 1]), *kv, mask[b:b + 1].numpy(), lens[b:b + 1], scale)
        got, gl = f64(o[b:b + 1]), f64(lse[b:b + 1])
        e = (d + 32) * 2.0 ** -24 * E + 2.0 ** -21
        tol = 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -16 + e + lens[b] * 2.0 ** -24)[..., None] * A
        err = np.abs(got - want)
        assert np.isfinite(got).all(), "not finite"
        assert np.all(err <= tol), f"o off by up to {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"
        assert np.all(np.abs(gl - wl) <= e + 2.0 ** -20 * (1 + np.abs(wl))), "lse"


def run(bits, d, B, Hq, k, v, q, mask, scale=0.0):
    """One KV head that every sequence of the batch shares."""
    L = k.shape[2]
    one, table = make_cache(1, 1, -(-L // 64), d, bits, True, 0)
    seer.seer_kv_write(one, k.cuda(), v.cuda())
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), shared(one, B), mask.cuda(), L, return_lse=True,
                                                 softmax_scale=scale)
    seer.seer_check_status()
    return o, lse, parts(one, table)


def ones(B, Hq, L):
    return torch.ones((B, Hq, -(-L // 64)), dtype=torch.uint8)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq", HEADS)
def test_probabilities_keep_their_bits(bits, d, B, Hq):
    """Every element's value is 0 (z = -1, s n = 1), so o is what the rounding of p s leaves: 31 tokens of 32 have p of
    1/2 + 2^-12 of the others', the middle of two numbers of 11 bits, all rounded the same way."""
    L, scale = 450, -float(np.log(0.5 + 2.0 ** -12))
    k = torch.zeros((1, 1, L, d))
    k[0, 0, :, 0] = -(torch.arange(L) % 32 != 5).float()
    q = torch.zeros((B, Hq, d))
    q[..., 0] = 1.0
    v = torch.zeros((1, 1, L, d))
    v[..., 0::32] = -1.0
    v[..., 1::32] = 2.0 ** bits - 2
    k, v, q = (x.to(torch.bfloat16) for x in (k, v, q))
    mask = ones(B, Hq, L)
    o, lse, kv = run(bits, d, B, Hq, k, v, q, mask, scale)
    assert np.all(kv[1][1][:, :, :L] == 1.0)
    check(o, lse, q, kv, mask, [L] * B, (0, B - 1), scale)


@pytest.mark.parametrize("bits,d", [(4, 128), (4, 64), (8, 128)])
@pytest.mark.parametrize("B,Hq", HEADS)
@pytest.mark.parametrize("apart", [24, 36, 90, -36, -90])
def test_groups_of_a_row_far_apart(bits, d, B, Hq, apart):
    """One group of every V row 2^apart times the others."""
    L, G = 450, ref.group(bits)
    k, v, q = bf16((1, 1, L, d), 1), bf16((1, 1, L, d), 2).float(), bf16((B, Hq, d), 3)
    v[..., G:2 * G] *= 2.0 ** apart
    mask = ones(B, Hq, L)
    o, lse, kv = run(bits, d, B, Hq, k, v.to(torch.bfloat16), q, mask)
    check(o, lse, q, kv, mask, [L] * B, (0, B - 1))


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq", HEADS)
@pytest.mark.parametrize("apart", [26, 40, 110, 180])
def test_block_of_large_values_that_other_heads_leave_out(bits, d, B, Hq, apart):
    """V of one block 2^apart times the others; every other head leaves it out, and its result is the ordinary one."""
    L = 450
    k, v, q = bf16((1, 1, L, d), 1), bf16((1, 1, L, d), 2).float(), bf16((B, Hq, d), 3)
    block = torch.arange(L) // 64 == 2
    v *= torch.where(block, 2.0 ** (apart - 60), 2.0 ** -60).view(1, 1, L, 1)
    mask = ones(B, Hq, L)
    mask[:, 1::2, 2] = 0
    o, lse, kv = run(bits, d, B, Hq, k, v.to(torch.bfloat16), q, mask)
    check(o, lse, q, kv, mask, [L] * B, (0, B - 1))


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq", HEADS)
@pytest.mark.parametrize("apart,below", [(30, 50), (40, 60), (80, 90)])
def test_large_values_of_small_weight(bits, d, B, Hq, apart, below):
    """Tokens whose V is 2^apart times the others' and whose p is 2^-below: next to nothing of the output."""
    L = 450
    k, v = torch.zeros((1, 1, L, d)), bf16((1, 1, L, d), 2).float()
    k[..., 0] = bf16((1, 1, L), 1).float()
    far = torch.arange(L) % 9 == 4
    k[0, 0, far, 0] = -below * float(np.log(2.0))
    v[0, 0, far] *= 2.0 ** apart
    q = torch.zeros((B, Hq, d))
    q[..., 0] = 1.0
    k, v, q = (x.to(torch.bfloat16) for x in (k, v, q))
    mask = ones(B, Hq, L)
    o, lse, kv = run(bits, d, B, Hq, k, v, q, mask, 1.0)
    check(o, lse, q, kv, mask, [L] * B, (0, B - 1), 1.0)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq", HEADS)
@pytest.mark.parametrize("apart", [30, 60])
def test_q_elements_far_apart(bits, d, B, Hq, apart):
    """Elements of q 2^-apart of the largest, against K elements 2^apart times the others: both halves of a score
    count."""
    L = 450
    k, v, q = bf16((1, 1, L, d), 1).float(), bf16((1, 1, L, d), 2), bf16((B, Hq, d), 3).float()
    far = torch.arange(d) >= 32 if bits == 4 else torch.arange(d) >= d // 2
    q[..., far] *= 2.0 ** -apart
    if bits == 4 or d == 128:                               # (the large elements in groups of their own)
        k[..., far] *= 2.0 ** apart
    else:
        k *= 2.0 ** apart
        q[..., ~far] = 0.0
        q[..., 0] = 2.0 ** -apart * 2.0 ** 10
    k, q = k.to(torch.bfloat16), q.to(torch.bfloat16)
    mask = ones(B, Hq, L)
    o, lse, kv = run(bits, d, B, Hq, k, v, q, mask)
    check(o, lse, q, kv, mask, [L] * B, (0, B - 1))


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("Hq", [2, 4, 8, 16])
def test_values_near_the_largest_with_scores_that_rise(bits, d, Hq):
    """V of 2^125 at a late token whose score is the largest, 20 times the first ones': a weighted sum that is in
    fp32's range stays there."""
    B, L = 150, 1500
    k, v = torch.zeros((1, 1, L, d)), bf16((1, 1, L, d), 2).float()
    k[0, 0, 1400, 0] = 3.0
    v[0, 0, 1400] = 2.0 ** 125
    v[0, 0, 1400, 1::2] = -2.0 ** 125
    q = torch.zeros((B, Hq, d))
    q[..., 0] = 1.0
    k, v, q = (x.to(torch.bfloat16) for x in (k, v, q))
    mask = ones(B, Hq, L)
    o, lse, kv = run(bits, d, B, Hq, k, v, q, mask, 1.0)
    check(o, lse, q, kv, mask, [L] * B, (0, B - 1), 1.0)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq", HEADS)
@pytest.mark.parametrize("e", [20, 30, 40, 60, 100])
def test_scores_beyond_fp32_steps_of_one(bits, d, B, Hq, e):
    """Scores of 2^e and more, each a 256th of the largest from the next: the largest key takes all."""
    L = 450
    k = torch.zeros((1, 1, L, d))
    top = torch.randperm(L, generator=torch.Generator().manual_seed(e))
    k[0, 0, :, 0] = (top % 128 + 64).float() * 2.0 ** (e // 2)
    k[0, 0, 333, 0] = 255.0 * 2.0 ** (e // 2)               # the largest of all
    q = torch.zeros((B, Hq, d))
    q[..., 0] = 2.0 ** (e - e // 2)
    k, q, v = k.to(torch.bfloat16), q.to(torch.bfloat16), bf16((1, 1, L, d), 2)
    o, lse, kv = run(bits, d, B, Hq, k, v, q, ones(B, Hq, L), 1.0)
    score = ref.values(*kv[0])[0, 0, :L] @ f64(q[0, 0])
    best = int(np.argmax(score))
    want = ref.values(*kv[1])[0, 0, best]
    assert best == 333 and np.sort(score)[-2] < score[best] * (1 - 2.0 ** -9)
    assert np.all(np.abs(f64(o) - want) <= (2.0 ** -8 + 2.0 ** -15) * np.abs(want) + 2.0 ** -15 * (np.abs(want).max()))
    assert np.all(np.abs(f64(lse) - score[best]) <= 2.0 ** -21 * score[best])
