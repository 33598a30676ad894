"""A decode step of sequences of their own lengths: gate scores, block mask and
the whole step over the quantised cache, each sequence as it is alone."""
import ctypes

import numpy as np
import pytest
import torch

import long_context_prefill_attngate_b200 as seer
from test_gpu_kvcache import bf16, check_decode, dev32, gpu, make_cache, parts  # noqa: F401

pytestmark = pytest.mark.gpu


def blocks(n):
    return -(-n // 64)


def clamp(lens, L):
    return [max(0, min(x, L)) for x in lens]


def mask_row(s, nb, k=None, threshold=None, first=True, last=True):
    """The mask row of one head by its definition: s fp32 [nb_all]."""
    m = np.zeros(len(s), np.uint8)
    if nb == 0:
        return m
    forced = [j for j, f in ((0, first), (nb - 1, last)) if f]
    if threshold is not None:
        m[:nb] = s[:nb] > np.float32(threshold)
        m[forced] = 1
        return m
    k = max(len(set(forced)), min(k, nb))
    order = sorted(range(nb), key=lambda j: (j not in forced, -s[j], j))
    m[order[:k]] = 1
    return m


SHAPES = [
    (5, 8, 2, 128, 64, 3000, [3000, 1999, 64, 0, 1]),
    (4, 6, 3, 64, 128, 700, [65, 700, 5000, -2]),               # beyond L and below 0
    (3, 4, 4, 128, 32, 64 * 1100, [64 * 1100 - 1, 64 * 1030, 100]),   # rows of more than 1024 blocks
    (1, 2, 1, 64, 64, 1, [1]),
]


@pytest.mark.parametrize("B,Hq,Hkv,d,dg,L,lens", SHAPES)
def test_gate_scores_of_each_sequence_alone(B, Hq, Hkv, d, dg, L, lens):
    nb = blocks(L)
    q, wq = bf16((B, Hq, d), 1).cuda(), bf16((Hq, d, dg), 2, 0.1).cuda()
    kt = torch.randn((B, Hkv, nb, dg), generator=torch.Generator().manual_seed(3)).cuda()
    lens_c = clamp(lens, L)
    for b, n in enumerate(lens_c):
        kt[b, :, blocks(n):] = float("nan")                     # not read
    s = torch.full((B, Hq, nb), 7.0, device="cuda")
    got = seer.seer_decode_gate_scores_cached(q, kt, wq, L, Hkv, scores=s, lens=dev32(lens))
    seer.seer_check_status()
    assert got is s
    for b, n in enumerate(lens_c):
        m = blocks(n)
        assert not s[b, :, m:].any()
        if n:
            alone = seer.seer_decode_gate_scores_cached(q[b:b + 1].contiguous(), kt[b:b + 1, :, :m].contiguous(), wq, n, Hkv)
            assert torch.equal(s[b, :, :m], alone[0])
            assert torch.all((s[b].sum(-1) - 1).abs() < 1e-5)
    even = seer.seer_decode_gate_scores_cached(q, torch.nan_to_num(kt), wq, L, Hkv, lens=dev32([L] * B))
    assert torch.equal(even, seer.seer_decode_gate_scores_cached(q, torch.nan_to_num(kt), wq, L, Hkv))


@pytest.mark.parametrize("B,Hq,Hkv,d,dg,L,lens", SHAPES)
@pytest.mark.parametrize("first,last", [(True, True), (False, False), (True, False), (False, True)])
def test_mask_rows_of_each_sequence_alone(B, Hq, Hkv, d, dg, L, lens, first, last):
    nb = blocks(L)
    s = torch.rand((B, Hq, nb), generator=torch.Generator().manual_seed(nb)).cuda()
    s[..., 1::3] = 0.5                                          # ties go to the lower block
    x, lens_c, ld = s.cpu().numpy(), clamp(lens, L), dev32(lens)
    flags = dict(force_first=first, force_diag=last, lens=ld)
    for density in (0.0, 0.1, 0.37, 1.0):
        m = seer.seer_decode_block_mask(s, "topk", density=density, mask=torch.full((B, Hq, nb), 9, dtype=torch.uint8, device="cuda"), **flags)
        seer.seer_check_status()
        want = [[mask_row(x[b, h], blocks(n), int(np.ceil(density * blocks(n))), None, first, last) for h in range(Hq)]
                for b, n in enumerate(lens_c)]
        assert np.array_equal(m.cpu().numpy(), np.array(want)), density
    m = seer.seer_decode_block_mask(s, "topk", k_fixed=3, **flags)
    want = [[mask_row(x[b, h], blocks(n), 3, None, first, last) for h in range(Hq)] for b, n in enumerate(lens_c)]
    assert np.array_equal(m.cpu().numpy(), np.array(want))
    m = seer.seer_decode_block_mask(s, "threshold", threshold=0.5, **flags)
    want = [[mask_row(x[b, h], blocks(n), None, 0.5, first, last) for h in range(Hq)] for b, n in enumerate(lens_c)]
    assert np.array_equal(m.cpu().numpy(), np.array(want))


@pytest.mark.parametrize("nb", [40, 1100])
def test_mask_counts_from_a_device_row(nb):
    """k_per_row through the C entry: row nb_b - 1 of it, and none for a sequence without a token."""
    B, Hq, lens = 3, 2, [64 * nb, 0, 64 * 17 + 1]
    s = torch.rand((B, Hq, nb), generator=torch.Generator().manual_seed(1)).cuda()
    k = (torch.arange(nb) % 7 + 3).to(torch.int32).cuda()
    m = torch.full((B, Hq, nb), 9, dtype=torch.uint8, device="cuda")
    ld = dev32(lens)
    sh = seer.seer_shape(B, Hq, 1, 64 * nb, 64)
    mp = seer.seer_mask_params(seer.SEER_MASK_TOPK, 0.0, 0.0, 0, k.data_ptr(), 1, 1)
    assert seer.lib().seer_decode_block_mask_lens(ctypes.byref(sh), s.data_ptr(), ctypes.byref(mp), ld.data_ptr(),
                                                  m.data_ptr(), torch.cuda.current_stream().cuda_stream) == seer.SEER_OK
    seer.seer_check_status()
    want = [[mask_row(s[b, h].cpu().numpy(), blocks(n), int(k[blocks(n) - 1]) if n else 0) for h in range(Hq)]
            for b, n in enumerate(lens)]
    assert np.array_equal(m.cpu().numpy(), np.array(want))


@pytest.mark.parametrize("bits,maxmin", [(4, False), (8, True)])
@pytest.mark.parametrize("density", [0.1, 0.4])
def test_decode_steps_of_a_ragged_batch(bits, maxmin, density):
    """Append, refresh, scores, mask, attend, token by token: scores and masks as those of each sequence alone, outputs
    within the attention's tolerance of the definition.  One slot is idle, one sequence crosses into a new block."""
    B, Hq, Hkv, d, dg, steps = 5, 8, 2, 128, 64, 3
    lens0 = [1500, 63, 0, 640, 1]
    L = 1600
    nb = blocks(L)
    cache, table = make_cache(B, Hkv, nb, d, bits, True, 3)
    k, v = bf16((B, Hkv, L, d), 1).cuda(), bf16((B, Hkv, L, d), 2).cuda()
    wk, wq = bf16((Hkv, 2 * d if maxmin else d, dg), 4, 0.1).cuda(), bf16((Hq, d, dg), 5, 0.1).cuda()
    seer.seer_kv_write(cache, k, v, count=dev32(lens0))
    kt = seer.seer_gate_key_cache_quant(cache, wk, L, lens=dev32(lens0), k_maxmin=maxmin)
    for i in range(steps):
        lens = [n + i + 1 if n else 0 for n in lens0]
        ld, one = dev32(lens), dev32([int(n > 0) for n in lens])
        q = bf16((B, Hq, d), 10 + i).cuda()
        at = torch.tensor([max(n - 1, 0) for n in lens], device="cuda").view(B, 1, 1, 1).expand(B, Hkv, 1, d)
        seer.seer_kv_write(cache, k.gather(2, at), v.gather(2, at), start=ld, count=one, start_pos=-1)
        seer.seer_gate_key_cache_quant(cache, wk, L, kt=kt, lens=ld, k_maxmin=maxmin)
        s = seer.seer_decode_gate_scores_cached(q, kt, wq, L, Hkv, lens=ld)
        m = seer.seer_decode_block_mask(s, "topk", density=density, lens=ld)
        o, lse = seer.seer_block_sparse_decode_quant(q, cache, m, L, lens=ld, return_lse=True)
        seer.seer_check_status()
        check_decode(o, lse, q, parts(cache, table), m.cpu(), lens)
        for b, n in enumerate(lens):
            if n == 0:
                assert not o[b].any() and not s[b].any() and not m[b].any()
                continue
            one_table = cache.block_table[b:b + 1, :blocks(n)].contiguous()
            alone = seer.SeerKVCache(cache.pages, d, bits, block_table=one_table)
            kt1 = seer.seer_gate_key_cache_quant(alone, wk, n, k_maxmin=maxmin)
            s1 = seer.seer_decode_gate_scores_cached(q[b:b + 1].contiguous(), kt1, wq, n, Hkv)
            m1 = seer.seer_decode_block_mask(s1, "topk", density=density)
            assert torch.equal(kt[b, :, :blocks(n)], kt1[0]) and torch.equal(s[b, :, :blocks(n)], s1[0])
            assert torch.equal(m[b, :, :blocks(n)], m1[0]) and m[b, :, blocks(n) - 1].all()
    seer.seer_check_status()


def test_captured_scores_and_mask_follow_the_lengths():
    B, Hq, Hkv, d, dg, L = 3, 4, 2, 64, 32, 900
    nb = blocks(L)
    q, wq = bf16((B, Hq, d), 1).cuda(), bf16((Hq, d, dg), 2, 0.1).cuda()
    kt = torch.randn((B, Hkv, nb, dg), generator=torch.Generator().manual_seed(3)).cuda()
    lens = dev32([900, 1, 300])

    def step():
        s = seer.seer_decode_gate_scores_cached(q, kt, wq, L, Hkv, lens=lens)
        return s, seer.seer_decode_block_mask(s, "topk", density=0.3, lens=lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for ln in ([900, 1, 300], [64, 65, 0], [0, 900, 899]):
        lens.copy_(dev32(ln))
        graph.replay()
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    seer.seer_check_status()
