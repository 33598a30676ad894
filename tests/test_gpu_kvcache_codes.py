"""Codes of rows whose elements lie far apart: x - z is no fp32 number there, and
the nearest integer to (x - z) / s is still the one that is stored."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import long_context_prefill_attngate_b200 as seer
from test_gpu_kvcache import FORMATS, f64, gpu, make_cache, parts  # noqa: F401

pytestmark = pytest.mark.gpu


def bf16_near(x):
    return torch.tensor(np.asarray(x, np.float64)).to(torch.bfloat16).double().numpy()


def far_groups(bits, seed):
    """Groups of G bf16 numbers: a minimum far below the others, elements far below the minimum, and quotients next to
    halves."""
    G, top = ref.group(bits), 2 ** bits - 1
    rng = np.random.default_rng(seed)
    halves = (np.arange(G) % top) + 0.5
    rows = []
    for k in (10, 14, 16, 17, 20, 24, 30, 40):
        for scale in (1.0, 1.25, 2.0 ** 60):
            tiny = scale * 2.0 ** -k
            a = np.minimum(halves, top) * scale             # ties but for the minimum of -tiny: one step up
            a[:2] = -tiny, top * scale
            b = np.where(np.arange(G) % 2, tiny, -tiny) * rng.uniform(1, 2, G) + (halves - (top - 1) / 2) * scale
            b[:2] = -(top - 1) / 2 * scale, (top + 1) / 2 * scale
            c = np.where(np.arange(G) % 3 == 0, tiny, np.where(np.arange(G) % 3 == 1, -tiny, 0.5 * scale)) + 0 * halves
            c[:2] = -0.5 * scale, (top - 0.5) * scale       # x + 1/2 far below an element: just past a half, or just not
            rows += [a, b, c, -a, -c]
    for _ in range(40):                                     # random significands and exponents
        r = rng.uniform(1, 2, G) * 2.0 ** rng.integers(-30, 1, G) * rng.choice((-1, 1), G)
        rows.append(r)
    return bf16_near(np.stack(rows))


def test_example_of_an_element_far_below_the_minimum():
    """-1, 29 and 2^-30: s = 2, (2^-30 + 1) / 2 is above a half, so n = 1."""
    x = np.full(32, 3.0)
    x[:3] = -1.0, 29.0, 2.0 ** -30
    n, s, z = ref.quantise(x[None], 4)
    assert (s, z) == (2.0, -1.0) and n[0, 2] == 1
    k = torch.tensor(np.tile(x, 4), dtype=torch.bfloat16).view(1, 1, 1, 128).cuda()
    cache, table = make_cache(1, 1, 1, 128, 4, False, 0)
    seer.seer_kv_write(cache, k, k)
    seer.seer_check_status()
    for gn, gs, gz in parts(cache, table):
        assert np.array_equal(gn[0, 0, 0], np.tile(n[0], 4))


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("seed", [0, 1])
def test_codes_of_groups_far_apart(bits, d, seed):
    groups = far_groups(bits, seed)
    per = d // ref.group(bits)
    order = np.random.default_rng(seed).permutation(len(groups) * per) % len(groups)
    x = groups[order].reshape(len(groups), d)
    k = torch.tensor(x).to(torch.bfloat16).view(1, 1, -1, d)
    n = k.shape[2]
    cache, table = make_cache(1, 1, -(-n // 64), d, bits, False, 0)
    seer.seer_kv_write(cache, k.cuda(), k.flip(2).contiguous().cuda())
    seer.seer_check_status()
    for (gn, gs, gz), src in zip(parts(cache, table), (k, k.flip(2))):
        wn, ws, wz = ref.quantise(f64(src), bits)
        assert np.array_equal(gs[:, :, :n], ws) and np.array_equal(gz[:, :, :n], wz)
        bad = gn[:, :, :n] != wn
        assert not bad.any(), f"{bad.sum()} of {bad.size} codes differ"
