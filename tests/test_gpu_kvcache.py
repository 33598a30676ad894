"""The quantised KV cache on the GPU against its definition in 64 bits
(kv_reference.py): rows written and read back, the gate's key rows, and the
block-sparse decode attention.

Tolerances, from the arithmetic:
 * codes, scales and zeros: equal.
 * values read back: one rounding to bf16, 2^-8 of the value (and 2^-24 before).
 * key rows: sums in fp32 over up to 64 tokens, then over dk features, each
   addition within 2^-24 of the sum of magnitudes; the rotation adds a few more.
 * attention: a probability's exponent is off by at most the fp32 sum of a
   score, (d + 32) 2^-24 of sum |q| (s n + |z|) * scale =: E, plus 2^-21 of the
   exponential; p s is rounded to fp16 (2^-11).  So o is within
   2^-8 |o| + 2 (2^-11 + E) sum p (s n + |z|), lse within E + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import long_context_prefill_attngate_b200 as seer
from long_context_prefill_attngate_b200 import build as seer_build

pytestmark = pytest.mark.gpu
THETA = 5e5
FORMATS = [(4, 128), (4, 64), (8, 128), (8, 64)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    seer_build.build()
    seer.lib()
    yield
    seer.seer_check_status()


def bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def dev32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make_cache(B, Hkv, blocks, d, bits, paged, seed, extra=3):
    """An all-0xFF cache (NaN params, largest codes); paged: pages in a random order, some unused."""
    n = B * blocks + (extra if paged else 0)
    pages = torch.full((n, Hkv, seer.seer_kv_record_bytes(bits, d)), 255, dtype=torch.uint8, device="cuda")
    if not paged:
        return seer.SeerKVCache(pages, d, bits, batch=B), np.arange(n).reshape(B, blocks)
    table = np.random.default_rng(seed).permutation(n)[:B * blocks].reshape(B, blocks)
    return seer.SeerKVCache(pages, d, bits, block_table=dev32(table)), table


def parts(cache, table):
    return ref.gather(cache.pages.cpu().numpy(), table, cache.bits, cache.d)


# ------------------------------------------------------------------ write, read

@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hkv,n,start,count,paged,token_major", [
    (1, 2, 130, [0], None, False, False),
    (3, 1, 70, [0, 61, 31], [70, 3, 0], True, True),       # a chunk that starts inside a page, one row, none
    (2, 3, 1, [63, 64], None, True, False),                # a decode step's token, last and first of a page
    (4, 2, 33, [1, 30, 95, 100], [33, 40, 1, -5], True, True),   # counts beyond n and below 0
    (1, 1, 257, [7], [250], False, True),
])
def test_write_and_read(bits, d, B, Hkv, n, start, count, paged, token_major):
    blocks = 5
    cache, table = make_cache(B, Hkv, blocks, d, bits, paged, 5)
    before = cache.pages.clone()
    k, v = bf16((B, Hkv, n, d), 1), bf16((B, Hkv, n, d), 2, 3.0)
    k[0, 0, 0, :32] = 0.5                                  # a constant group: s = 0
    v[0, 0, 0] *= torch.arange(d) % 2 * 1e-3 + 1e-30
    kd, vd = (t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if token_major else t.cuda() for t in (k, v))
    seer.seer_kv_write(cache, kd, vd, start=dev32(start), count=None if count is None else dev32(count))
    want = before.cpu().numpy()
    cnt = [n] * B if count is None else [max(0, min(c, n)) for c in count]
    kq, vq = ref.quantise(f64(k), bits), ref.quantise(f64(v), bits)
    for b in range(B):
        for h in range(Hkv):
            for t in range(cnt[b]):
                p = start[b] + t
                ref.pack(want, table[b, p // 64], h, p % 64, [x[b, h, t] for x in kq], [x[b, h, t] for x in vq], bits, d)
    got = cache.pages.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"

    ko, vo = (torch.full((B, Hkv, n, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    seer.seer_kv_read(cache, n, start=dev32(start), count=None if count is None else dev32(count), k=ko, v=vo)
    seer.seer_check_status()
    for out, q in ((ko, kq), (vo, vq)):
        x, w = f64(out), ref.values(*q)
        for b in range(B):
            assert np.all(x[b, :, cnt[b]:] == 7.0)          # rows behind the last one: as they were
            assert np.all(np.abs(x[b, :, :cnt[b]] - w[b, :, :cnt[b]]) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(w[b, :, :cnt[b]]))
    only = seer.seer_kv_read(cache, n, start=dev32(start), count=None if count is None else dev32(count))
    for b in range(B):
        assert torch.equal(only[0][b, :, :cnt[b]], ko[b, :, :cnt[b]]) and not only[1][b, :, cnt[b]:].any()


@pytest.mark.parametrize("bits,d", FORMATS)
def test_write_extreme_groups(bits, d):
    """Ties, constant groups, tiny and huge ranges, infinities and NaN, each in a group of its own."""
    G = ref.group(bits)
    top = 2 ** bits - 1
    rows = []
    ties = torch.arange(G).float() % (2 * top + 1) / 2.0    # s = 1: every odd half is a tie
    ties[0], ties[1] = 0.0, float(top)
    rows += [ties, ties - 8, ties * 2.0 ** -20, ties * 2.0 ** 90, -ties * 0.75]
    rows += [torch.zeros(G), torch.full((G,), -3.25), torch.linspace(-1, 1, G) * 2.0 ** -110,
             torch.linspace(-1, 1, G) * 2.0 ** -98, torch.linspace(-1, 1, G) * 2.0 ** 125,
             torch.linspace(0, 1, G) * 2.0 ** 126]
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.randn(G, generator=torch.Generator().manual_seed(3))
        r[5] = bad
        rows.append(r)
    wide = torch.randn(G, generator=torch.Generator().manual_seed(4))
    wide[3] = 1e4                                           # a group whose other elements share one level
    rows.append(wide)
    n = len(rows)
    x = torch.stack([torch.cat([rows[(i + j) % n] for j in range(d // G)]) for i in range(n)]).to(torch.bfloat16)
    k = x.view(1, 1, n, d)
    cache, table = make_cache(1, 1, 1, d, bits, False, 0)
    seer.seer_kv_write(cache, k.cuda(), k.flip(2).contiguous().cuda(), start_pos=11)
    (kn, ks, kz), (vn, vs, vz) = parts(cache, table)
    for (gn, gs, gz), src in (((kn, ks, kz), k), ((vn, vs, vz), k.flip(2))):
        wn, ws, wz = ref.quantise(f64(src), bits)
        assert np.array_equal(gs[:, :, 11:11 + n], ws) and np.array_equal(gz[:, :, 11:11 + n], wz, equal_nan=True)
        assert np.array_equal(gn[:, :, 11:11 + n], wn)
    ko, _ = seer.seer_kv_read(cache, n, start_pos=11)
    seer.seer_check_status()
    w = ref.values(*ref.quantise(f64(k), bits))
    got = f64(ko)
    assert np.array_equal(np.isnan(got), np.isnan(w))
    ok = ~np.isnan(w)
    # below bf16's normal range the rounding is of 2^-134 at most
    assert np.all(np.abs(got - w)[ok] <= (2.0 ** -8 + 2.0 ** -23) * np.abs(w[ok]) + 2.0 ** -133)


def test_long_cache_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of the pool: the last page of a large one."""
    bits, d, Hkv = 8, 128, 8
    rec = seer.seer_kv_record_bytes(bits, d)
    n = 2 ** 32 // (rec * Hkv) + 40
    pages = torch.empty((n, Hkv, rec), dtype=torch.uint8, device="cuda")
    table = dev32([[n - 1, 3]])
    cache = seer.SeerKVCache(pages, d, bits, block_table=table)
    k, v = bf16((1, Hkv, 100, d), 1), bf16((1, Hkv, 100, d), 2)
    seer.seer_kv_write(cache, k.cuda(), v.cuda())
    got = ref.gather(pages[[n - 1, 3]].cpu().numpy(), np.array([[0, 1]]), bits, d)
    for (gn, gs, gz), src in zip(got, (k, v)):
        wn, ws, wz = ref.quantise(f64(src), bits)
        assert np.array_equal(gn[:, :, :100], wn) and np.array_equal(gs[:, :, :100], ws)
    q = bf16((1, 16, d), 3)
    mask = torch.ones((1, 16, 2), dtype=torch.uint8)
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), 100, return_lse=True)
    check_decode(o, lse, q, got, mask, [100])


@pytest.mark.parametrize("what", ["beyond", "negative", "page"])
def test_bad_positions_and_pages_are_left_out(what):
    """A position past the cache, one below 0 or a table entry outside the pool: a device error, nothing touched
    by that row, the other rows done."""
    bits, d, B, Hkv, n = 4, 128, 2, 2, 4
    cache, table = make_cache(B, Hkv, 2, d, bits, True, 1)
    start = [0, {"beyond": 126, "negative": -2, "page": 64}[what]]
    good = {"beyond": [0, 1], "negative": [2, 3], "page": []}[what]
    if what == "page":
        cache.block_table[1, 1] = cache.pages.shape[0]
    k = bf16((B, Hkv, n, d), 1)
    want = cache.pages.cpu().numpy()
    kq = ref.quantise(f64(k), bits)
    for b, ts in ((0, range(n)), (1, good)):
        for t in ts:
            for h in range(Hkv):
                p = start[b] + t
                one = [x[b, h, t] for x in kq]
                ref.pack(want, table[b, p // 64], h, p % 64, one, one, bits, d)
    seer.seer_kv_write(cache, k.cuda(), k.cuda(), start=dev32(start))
    with pytest.raises(seer.SeerError) as e:
        seer.seer_check_status()
    assert e.value.status == seer.SEER_ERR_DEVICE and "block table" in str(e.value)
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    out = torch.full((B, Hkv, n, d), 7.0, dtype=torch.bfloat16, device="cuda")
    seer.seer_kv_read(cache, n, start=dev32(start), k=out, v=torch.empty_like(out))
    with pytest.raises(seer.SeerError):
        seer.seer_check_status()
    for t in range(n):
        assert (t in good) != bool((out[1, :, t] == 7.0).all())
    if what != "page":
        return
    # a key block on a bad page is inactive, for the attention and for the gate
    cache, table = make_cache(B, Hkv, 2, d, bits, True, 1)
    kv = bf16((B, Hkv, 128, d), 2)
    seer.seer_kv_write(cache, kv.cuda(), kv.cuda())
    held = parts(cache, table)
    cache.block_table[1, 1] = -1
    q, mask = bf16((B, 4, d), 3), torch.ones((B, 4, 2), dtype=torch.uint8)
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), 128, return_lse=True)
    with pytest.raises(seer.SeerError):
        seer.seer_check_status()
    check_decode(o, lse, q, held, mask, [128, 64])
    wk = bf16((Hkv, d, 64), 4, 0.1)
    kt = seer.seer_gate_key_cache_quant(cache, wk.cuda(), 128)
    with pytest.raises(seer.SeerError):
        seer.seer_check_status()
    check_gate(kt, held[0], wk, [128, 64], 0, False)


# ------------------------------------------------------------------ gate key rows

def check_gate(kt, k, wk, lens, first, maxmin, fill=None):
    w = f64(wk)
    want, A = ref.gate_keys(k, w, lens, first, THETA, maxmin)
    got = f64(kt)
    if first:
        assert np.all(got[:, :, :first] == fill)
    tol = (64 + w.shape[1] + 32) * 2.0 ** -24 * A + 1e-30
    bad = np.abs(got - want)[:, :, first:] > tol[:, :, first:]
    assert np.isfinite(got).all() and not bad.any(), f"{bad.sum()} of {bad.size} rows off"


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hkv,L,dg,first,maxmin,lens,paged", [
    (1, 2, 1, 64, 0, False, None, False),
    (2, 3, 64, 4, 0, True, None, True),
    (1, 2, 1000, 128, 0, False, None, True),
    (3, 1, 300, 12, 4, False, None, False),
    (4, 2, 200, 64, 1, True, [200, 65, 64, 0], True),
    (2, 8, 777, 256, 0, False, [777, 130], True),
    (1, 1, 5000, 64, 3, False, None, False),
])
def test_gate_key_rows(bits, d, B, Hkv, L, dg, first, maxmin, lens, paged):
    nb = -(-L // 64)
    cache, table = make_cache(B, Hkv, nb + 1, d, bits, paged, L)
    ln = [L] * B if lens is None else lens
    k = bf16((B, Hkv, L, d), L + d)
    seer.seer_kv_write(cache, k.cuda(), k.cuda(), count=dev32(ln))
    dk = 2 * d if maxmin else d
    wk = bf16((Hkv, dk, dg), dg, dk ** -0.5)
    kt = torch.full((B, Hkv, nb, dg), 7.0, device="cuda")
    got = seer.seer_gate_key_cache_quant(cache, wk.cuda(), L, kt=kt, first_block=first,
                                         lens=None if lens is None else dev32(lens), rope_theta=THETA, k_maxmin=maxmin)
    seer.seer_check_status()
    assert got is kt
    check_gate(kt, [x[:, :, :64 * nb] for x in parts(cache, table)[0]], wk, ln, first, maxmin, 7.0)


def test_gate_key_rows_shared_weights_and_nothing_to_do():
    cache, table = make_cache(2, 2, 3, 128, 4, False, 0)
    k = bf16((2, 2, 150, 128), 9)
    seer.seer_kv_write(cache, k.cuda(), k.cuda())
    wk = bf16((128, 64), 3, 0.1)
    kt = seer.seer_gate_key_cache_quant(cache, wk.cuda(), 150)
    seer.seer_check_status()
    check_gate(kt, parts(cache, table)[0], wk[None].expand(2, -1, -1), [150, 150], 0, False)
    same = kt.clone()
    seer.seer_gate_key_cache_quant(cache, wk.cuda(), 150, kt=kt, first_block=3)
    seer.seer_check_status()
    assert torch.equal(kt, same)


# ------------------------------------------------------------------ attention

def check_decode(o, lse, q, kv, mask, lens, scale=None):
    d = q.shape[-1]
    want, wl, A, E = ref.decode(f64(q), *kv, mask.numpy(), lens, scale)
    got, gl = f64(o), f64(lse)
    e = (d + 32) * 2.0 ** -24 * E + 2.0 ** -21
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), empty) and np.all(got[empty] == 0)
    tol = 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -11 + e[..., None]) * A
    err = np.abs(got - want)
    assert np.isfinite(got).all() and np.all(err <= tol), f"o off by {np.max(err - tol):.3e} over the tolerance"
    gl, wl, e = gl[~empty], wl[~empty], e[~empty]
    assert np.all(np.abs(gl - wl) <= e + 2.0 ** -20 * (1 + np.abs(wl))), "lse"


def attend(bits, d, B, Hq, Hkv, L, p, lens=None, paged=True, seed=0, kscale=1.0, vscale=1.0, scale=None, spare=1):
    nb = -(-L // 64)
    cache, table = make_cache(B, Hkv, nb + spare, d, bits, paged, seed)
    ln = [L] * B if lens is None else [max(0, min(x, L)) for x in lens]
    k, v = bf16((B, Hkv, L, d), seed + 1, kscale), bf16((B, Hkv, L, d), seed + 2, vscale)
    seer.seer_kv_write(cache, k.cuda(), v.cuda(), count=dev32(ln))
    q = bf16((B, Hq, d), seed + 3)
    mask = (torch.rand((B, Hq, nb), generator=torch.Generator().manual_seed(seed + 4)) < p).to(torch.uint8)
    mask *= torch.randint(1, 256, mask.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.uint8)
    o, lse = seer.seer_block_sparse_decode_quant(
        q.cuda(), cache, mask.cuda(), L, lens=None if lens is None else dev32(lens), return_lse=True,
        softmax_scale=0.0 if scale is None else scale)
    seer.seer_check_status()
    check_decode(o, lse, q, parts(cache, table), mask, ln, scale)
    return cache, q, mask, o, lse


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 96, 97, 128, 1000])
def test_decode_lengths(bits, d, L):
    attend(bits, d, 1, 8, 2, L, 1.0, paged=False, seed=L, spare=0)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (4, 2), (6, 2), (5, 1), (16, 2), (9, 1), (12, 1), (32, 2), (17, 1)])
def test_decode_group_sizes(bits, d, Hq, Hkv):
    attend(bits, d, 2, Hq, Hkv, 700, 0.4, seed=Hq)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("p", [0.0, 0.02, 0.3])
def test_decode_ragged_batch(bits, d, p):
    """Lengths from none to beyond L (clamped), pages in any order, rows whose mask leaves nothing."""
    attend(bits, d, 6, 8, 2, 2000, p, lens=[2000, 1337, 1, 0, 5000, -3], seed=11)


@pytest.mark.parametrize("bits,d,Hq,Hkv,L,lens", [
    (4, 128, 16, 8, 9000, [9000, 0, 64, 5000, 7]),
    (4, 64, 12, 6, 6000, [1, 6000, 1, 1]),
    (8, 128, 8, 8, 3000, [3000] * 4),
    (8, 64, 9, 1, 2500, [0] * 7),                           # nothing anywhere, groups of nine
    (4, 128, 2, 1, 1500, [(97 * i) % 1501 for i in range(64)]),   # as many sequences as are shared out
    (4, 128, 2, 1, 1200, [(97 * i) % 1201 for i in range(65)]),   # one more
    (8, 128, 4, 2, 3500, [3500 - 90 * i for i in range(37)]),
    (4, 64, 1, 1, 64 * 600, [64 * 600, 3, 0, 64 * 300, 64 * 600 - 1]),
])
def test_decode_batches_shared_out_by_length(bits, d, Hq, Hkv, L, lens):
    """CTAs in proportion to the lengths, which only the device knows."""
    attend(bits, d, len(lens), Hq, Hkv, L, 0.4, lens=lens, seed=len(lens))


@pytest.mark.parametrize("bits,d", FORMATS)
def test_decode_long_and_split(bits, d):
    """More blocks than one pass of the list takes, one KV head: many splits."""
    attend(bits, d, 1, 4, 1, 64 * 1100 + 5, 0.3, seed=12)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("nb", [1200, 1203])               # four blocks a lane where the rows are aligned, one where not
def test_decode_long_rows_and_bad_pages(bits, d, nb):
    """Rows of more blocks than a warp takes in one round, a short sequence beside a long one, and table entries of
    active blocks that name no page: those blocks count as inactive, and the device status says so."""
    B, Hq, Hkv, L = 2, 6, 2, 64 * nb
    lens = [L - 70, 130]
    cache, table = make_cache(B, Hkv, nb, d, bits, True, 3)
    k, v = bf16((B, Hkv, L, d), 1), bf16((B, Hkv, L, d), 2)
    seer.seer_kv_write(cache, k.cuda(), v.cuda(), count=dev32(lens))
    q = bf16((B, Hq, d), 3)
    mask = (torch.rand((B, Hq, nb), generator=torch.Generator().manual_seed(nb)) < 0.1).to(torch.uint8)
    mask[:, :, [0, 1, 700, nb - 2]] = 1
    held = parts(cache, table)
    args = (q.cuda(), cache, mask.cuda(), L)
    o, lse = seer.seer_block_sparse_decode_quant(*args, lens=dev32(lens), return_lse=True)
    seer.seer_check_status()
    check_decode(o, lse, q, held, mask, lens)
    for j, bad in ((1, -1), (700, cache.pages.shape[0]), (nb - 2, 2 ** 30)):
        cache.block_table[0, j] = bad
    o, lse = seer.seer_block_sparse_decode_quant(*args, lens=dev32(lens), return_lse=True)
    with pytest.raises(seer.SeerError):
        seer.seer_check_status()
    without = mask.clone()
    without[0, :, [1, 700, nb - 2]] = 0
    check_decode(o, lse, q, held, without, lens)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("kscale,vscale,scale", [(30.0, 1.0, None), (1.0, 1e-12, None), (1.0, 1e12, None),
                                                 (1e-3, 1.0, 5.0), (1.0, 1.0, 1e-3)])
def test_decode_ranges(bits, d, kscale, vscale, scale):
    attend(bits, d, 1, 4, 2, 500, 0.7, seed=13, kscale=kscale, vscale=vscale, scale=scale)


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq", [(1, 4), (1, 8), (150, 12)])
@pytest.mark.parametrize("kscale,vscale,scale", [(30.0, 1.0, None), (1.0, 1e12, None), (1e-3, 1e-12, 5.0)])
def test_decode_ranges_of_groups_of_any_size(bits, d, B, Hq, kscale, vscale, scale):
    attend(bits, d, B, Hq, 1, 400, 0.7, seed=14, kscale=kscale, vscale=vscale, scale=scale)


@pytest.mark.parametrize("bits,d", FORMATS)
def test_decode_token_scales_far_apart(bits, d):
    """V of neighbouring tokens 2^40 apart in magnitude, growing and shrinking along the cache; q far from 1."""
    B, Hq, Hkv, L = 1, 8, 2, 400
    cache, table = make_cache(B, Hkv, 7, d, bits, False, 0)
    k, v = bf16((B, Hkv, L, d), 1), bf16((B, Hkv, L, d), 2)
    v = (v.float() * 2.0 ** (torch.arange(L) % 5 * 10 - 20).view(1, 1, L, 1)).to(torch.bfloat16)
    seer.seer_kv_write(cache, k.cuda(), v.cuda())
    mask = torch.ones((B, Hq, 7), dtype=torch.uint8)
    for qs in (1.0, 1e-30, 1e-3):
        q = (bf16((B, Hq, d), 3).float() * qs).to(torch.bfloat16)
        o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), L, return_lse=True)
        seer.seer_check_status()
        check_decode(o, lse, q, parts(cache, table), mask, [L])
    q = (bf16((B, Hq, d), 3).float() * 2.0 ** 100).to(torch.bfloat16)   # scores of 2^100: one key takes all
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), L, return_lse=True, softmax_scale=2.0 ** -100)
    check_decode(o, lse, q, parts(cache, table), mask, [L], 2.0 ** -100)


@pytest.mark.parametrize("bits,d", FORMATS)
def test_decode_nan_stays_where_it_is(bits, d):
    """NaN in K or V reaches only heads that select the block, NaN in V only its group's elements, and nothing behind
    the length counts; NaN in q only its own head."""
    B, Hq, Hkv, L, G = 1, 4, 1, 300, ref.group(bits)
    cache, table = make_cache(B, Hkv, 5, d, bits, False, 0)
    k, v = bf16((B, Hkv, L, d), 1), bf16((B, Hkv, L, d), 2)
    kn, vn = k.clone(), v.clone()
    kn[0, 0, 70, 3] = float("nan")                          # block 1
    vn[0, 0, 140, d - 1] = float("inf")                     # block 2, the last group
    seer.seer_kv_write(cache, kn.cuda(), vn.cuda())
    mask = torch.ones((B, Hq, 5), dtype=torch.uint8)
    mask[0, 1, 1] = 0                                       # head 1 leaves out block 1, head 2 block 2, head 3 both
    mask[0, 2, 2] = 0
    mask[0, 3, 1:3] = 0
    q = bf16((B, Hq, d), 3)
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), L, return_lse=True)
    seer.seer_check_status()
    assert torch.isnan(o[0, 0]).all() and torch.isnan(o[0, 2]).all() and torch.isnan(lse[0, [0, 2]]).all()
    assert torch.isnan(o[0, 1, d - G:]).all() and torch.isfinite(o[0, 1, :d - G]).all()
    held = parts(cache, table)
    check_decode(o[:, 3:], lse[:, 3:], q[:, 3:], held, mask[:, 3:], [L])
    kq, vq = held
    vq = (vq[0], vq[1], np.where(np.isnan(vq[2]), 0.0, vq[2]))
    want = ref.decode(f64(q[:, 1:2]), kq, vq, mask[:, 1:2].numpy(), [L])[0][0, 0, :d - G]
    assert np.all(np.abs(f64(o[0, 1, :d - G]) - want) <= 2.0 ** -6 * (np.abs(want) + 0.1))
    q2 = q.clone()
    q2[0, 0, 5] = float("nan")
    q2[0, 1, 5] = float("inf")
    first = mask[..., :1].contiguous()
    o2, lse2 = seer.seer_block_sparse_decode_quant(q2.cuda(), cache, first.cuda(), 64, return_lse=True)
    seer.seer_check_status()
    assert torch.isnan(o2[0, :2]).all()
    check_decode(o2[:, 2:], lse2[:, 2:], q2[:, 2:], held, mask[:, 2:, :1], [64])


def shared(cache, B):
    """B sequences that all read the one sequence of `cache`."""
    return seer.SeerKVCache(cache.pages, cache.d, cache.bits, block_table=cache.block_table.repeat(B, 1))


def check_shared(o, lse, q, kv, mask, lens, which, scale=None):
    for b in which:
        check_decode(o[b:b + 1], lse[b:b + 1], q[b:b + 1], kv, mask[b:b + 1], lens[b:b + 1], scale)


# Batches large enough for sixteen heads a CTA where a KV head has more than eight.

@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("Hq,Hkv", [(9, 1), (16, 1), (20, 1), (34, 2)])
@pytest.mark.parametrize("p", [0.05, 0.5, 1.0])
def test_decode_wide_groups(bits, d, Hq, Hkv, p):
    B, L = 150, 450
    cache, table = make_cache(1, Hkv, 9, d, bits, True, Hq)
    k, v = bf16((1, Hkv, L, d), 1), bf16((1, Hkv, L, d), 2)
    seer.seer_kv_write(cache, k.cuda(), v.cuda())
    lens = [(i * 67) % 460 for i in range(B)]
    lens[:4] = [450, 0, 1, 32]
    q = bf16((B, Hq, d), 3)
    mask = (torch.rand((B, Hq, 8), generator=torch.Generator().manual_seed(Hq)) < p).to(torch.uint8) * 64
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), shared(cache, B), mask.cuda(), L, lens=dev32(lens), return_lse=True)
    seer.seer_check_status()
    check_shared(o, lse, q, parts(cache, table), mask, [min(x, L) for x in lens], range(B))


@pytest.mark.parametrize("bits,d", FORMATS)
def test_decode_wide_groups_shared_out_by_length(bits, d):
    B, Hq, Hkv, L = 20, 52, 4, 4000
    cache, table = make_cache(1, Hkv, 63, d, bits, True, 1)
    k, v = bf16((1, Hkv, L, d), 1), bf16((1, Hkv, L, d), 2)
    seer.seer_kv_write(cache, k.cuda(), v.cuda())
    lens = [L, 0, 17, L] + [200 * i for i in range(B - 4)]
    q = bf16((B, Hq, d), 3)
    mask = (torch.rand((B, Hq, 63), generator=torch.Generator().manual_seed(5)) < 0.3).to(torch.uint8)
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), shared(cache, B), mask.cuda(), L, lens=dev32(lens), return_lse=True)
    seer.seer_check_status()
    check_shared(o, lse, q, parts(cache, table), mask, lens, range(B))


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq,nb", [
    (16, 16, 800), (16, 16, 803),
    (150, 16, 800), (150, 16, 803), (4, 16, 1600), (4, 16, 1603),   # rows of more blocks than one round, one CTA per SM or two
    (1, 4, 1200), (1, 4, 1203),
])
def test_decode_long_rows_and_bad_pages_of_shared_caches(bits, d, B, Hq, nb):
    Hkv, L = 1, 64 * nb
    one, table = make_cache(1, Hkv, nb, d, bits, True, 3)
    k, v = bf16((1, Hkv, L, d), 1), bf16((1, Hkv, L, d), 2)
    seer.seer_kv_write(one, k.cuda(), v.cuda())
    cache, held = shared(one, B), parts(one, table)
    q = bf16((B, Hq, d), 3)
    mask = (torch.rand((B, Hq, nb), generator=torch.Generator().manual_seed(nb)) < 0.05).to(torch.uint8)
    mask[:, :, [1, 700, nb - 1]] = 1
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), L, return_lse=True)
    seer.seer_check_status()
    check_shared(o, lse, q, held, mask, [L] * B, {0, B - 1})
    cache.block_table[-1, 1], cache.block_table[-1, 700], cache.block_table[-1, nb - 1] = -1, one.pages.shape[0], 2 ** 30
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), L, return_lse=True)
    with pytest.raises(seer.SeerError):
        seer.seer_check_status()
    mask[-1, :, [1, 700, nb - 1]] = 0
    check_shared(o, lse, q, held, mask, [L] * B, {0, B - 1})


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hq", [(150, 16), (1, 16), (1, 8), (1, 4), (1, 2)])
def test_decode_nan_stays_where_it_is_in_groups_of_any_size(bits, d, B, Hq):
    L, G = 450, ref.group(bits)
    one, table = make_cache(1, 1, 8, d, bits, True, 0)
    k, v = bf16((1, 1, L, d), 1), bf16((1, 1, L, d), 2)
    k[0, 0, 70, 3] = float("nan")                           # block 1
    v[0, 0, 140, d - 1] = float("inf")                      # block 2, the last group
    seer.seer_kv_write(one, k.cuda(), v.cuda())
    mask = torch.ones((B, Hq, 8), dtype=torch.uint8)        # by h % 4: all, without block 1, without block 2, without both
    mask[:, 1::4, 1] = 0
    mask[:, 2::4, 2] = 0
    mask[:, 3::4, 1:3] = 0
    q = bf16((B, Hq, d), 3)
    q[:, 7:8, 5] = float("nan")
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), shared(one, B), mask.cuda(), L, return_lse=True)
    seer.seer_check_status()
    held = parts(one, table)
    assert torch.isnan(o[:, 0::4]).all() and torch.isnan(o[:, 2::4]).all() and torch.isnan(o[:, 7:8]).all()
    assert torch.isnan(o[:, 1::4, d - G:]).all() and torch.isfinite(o[:, 1::4, :d - G]).all()
    h = [x for x in (3, 11, 15) if x < Hq]
    if h:
        check_shared(o[:, h], lse[:, h], q[:, h], held, mask[:, h], [L] * B, {0, B // 2, B - 1})
    kq, vq = held                                           # the groups before the NaN, of a head that takes its block
    vq = (vq[0], vq[1], np.where(np.isnan(vq[2]), 0.0, vq[2]))
    want = ref.decode(f64(q[:1, 1:2]), kq, vq, mask[:1, 1:2].numpy(), [L])[0][0, 0, :d - G]
    assert np.all(np.abs(f64(o[0, 1, :d - G]) - want) <= 2.0 ** -6 * (np.abs(want) + 0.1))


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("Hq,B", [(4, 1), (16, 150), (2, 1), (8, 1)])
@pytest.mark.parametrize("step", [0.001, 0.01, 0.1, 3.0, -0.1])
def test_decode_scores_rising_along_the_cache(bits, d, Hq, B, step):
    """Maxima that move by less and by more than a step of the running maximum, token after token."""
    L = 450
    one, table = make_cache(1, 1, 8, d, bits, True, 0)
    q = bf16((B, Hq, d), 3)
    along = torch.zeros(d)
    along[0::8] = 1.0
    q[..., 0::8] = q[..., 0::8].abs() + 0.5                 # every head's scores rise
    k = (bf16((1, 1, L, d), 1).float() * 0.1 + step * torch.arange(L).view(1, 1, L, 1) * along).to(torch.bfloat16)
    v = bf16((1, 1, L, d), 2)
    v = (v.float() * 2.0 ** (torch.arange(L) % 7 * 3.0 - 9).view(1, 1, L, 1)).to(torch.bfloat16)
    seer.seer_kv_write(one, k.cuda(), v.cuda())
    mask = torch.ones((B, Hq, 8), dtype=torch.uint8)
    o, lse = seer.seer_block_sparse_decode_quant(q.cuda(), shared(one, B), mask.cuda(), L, return_lse=True)
    seer.seer_check_status()
    check_shared(o, lse, q, parts(one, table), mask, [L] * B, (0, B - 1))


def test_decode_outputs_written_over_poison_and_repeatable():
    cache, q, mask, o, lse = attend(4, 128, 2, 8, 2, 900, 0.3, seed=21)
    o2, l2 = torch.full_like(o, float("nan")), torch.full_like(lse, float("nan"))
    ws = torch.full((seer.seer_workspace_bytes(seer.SEER_CALL_BLOCK_SPARSE_DECODE_QUANT,
                                               seer.seer_shape(2, 8, 2, 900, 128)),), 255, dtype=torch.uint8, device="cuda")
    seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), 900, o=o2, lse=l2, workspace=ws)
    seer.seer_check_status()
    assert torch.equal(o, o2) and torch.equal(lse, l2)


# ------------------------------------------------------------------ together, as they are used

def decode_loop(cache, k, v, q, wk, wq, L0, steps, density, step=None):
    """Append a token, refresh its block's key rows, gate, mask, attend: the outputs of each step."""
    B, Hkv, _, d = k.shape
    seer.seer_kv_write(cache, k[:, :, :L0], v[:, :, :L0])
    nb = -(-(L0 + steps) // 64)
    kt = torch.zeros((B, Hkv, nb, wk.shape[-1]), device="cuda")
    kt[:, :, :-(-L0 // 64)] = seer.seer_gate_key_cache_quant(cache, wk, L0)
    outs = []
    for i in range(steps):
        L = L0 + i + 1
        n = -(-L // 64)
        seer.seer_kv_write(cache, k[:, :, L - 1:L], v[:, :, L - 1:L], start_pos=L - 1)
        now = kt[:, :, :n].contiguous()
        seer.seer_gate_key_cache_quant(cache, wk, L, kt=now, first_block=n - 1)
        kt[:, :, :n] = now
        s = seer.seer_decode_gate_scores_cached(q[:, :, i], now, wq, L, Hkv)
        m = seer.seer_decode_block_mask(s, "topk", density=density)
        outs.append((s, m, *seer.seer_block_sparse_decode_quant(q[:, :, i], cache, m, L, return_lse=True)))
    return outs


@pytest.mark.parametrize("bits", [4, 8])
def test_decode_loop_against_the_bf16_calls(bits):
    """The whole path token by token: scores, masks and outputs equal those of the bf16 calls on the values that the
    cache holds, up to the rounding of those values to bf16."""
    B, Hq, Hkv, d, dg, L0, steps = 2, 8, 2, 128, 64, 318, 5
    k, v = bf16((B, Hkv, L0 + steps, d), 1).cuda(), bf16((B, Hkv, L0 + steps, d), 2).cuda()
    q = bf16((steps, B, Hq, d), 3).cuda().permute(1, 2, 0, 3)
    q = [q[:, :, i].contiguous() for i in range(steps)]
    wk, wq = bf16((Hkv, d, dg), 4, 0.1).cuda(), bf16((Hq, d, dg), 5, 0.1).cuda()
    cache, table = make_cache(B, Hkv, 6, d, bits, True, 3)

    class Q:                                                # q[:, :, i] as the loop takes it
        def __getitem__(self, i):
            return q[i[2]]

    outs = decode_loop(cache, k, v, Q(), wk, wq, L0, steps, 0.5)
    seer.seer_check_status()
    held = parts(cache, table)
    kb, vb = seer.seer_kv_read(cache, L0 + steps)
    for i, (s, m, o, lse) in enumerate(outs):
        L = L0 + i + 1
        check_decode(o, lse, q[i], held, m.cpu(), [L] * B)
        # K rounded to bf16 moves a pooled key by 2^-8 of its magnitude at most; scores are a softmax of logits of that
        kc = kb[:, :, :L].contiguous()
        s_ref = seer.seer_decode_gate_scores(q[i], kc, wq, wk)
        assert torch.all((s - s_ref).abs() <= 0.02 * s_ref + 1e-6)
        o_ref, l_ref = seer.seer_block_sparse_decode(q[i], kc, vb[:, :, :L].contiguous(), m, return_lse=True)
        assert (o.float() - o_ref.float()).abs().max() <= 0.03 and (lse - l_ref).abs().max() <= 0.03
    seer.seer_check_status()


def test_captured_step_replays_with_new_lengths_and_rows():
    """One decode step in a CUDA graph: start, lens, rows, mask and table change between replays; two graphs that share
    a workspace, replayed in turn."""
    bits, B, Hq, Hkv, d, L = 4, 2, 8, 2, 128, 500
    nb = -(-L // 64)
    cache, table = make_cache(B, Hkv, nb, d, bits, True, 3)
    k0 = bf16((B, Hkv, L, d), 1).cuda()
    seer.seer_kv_write(cache, k0, k0)
    lens = dev32([100, 257])
    k1, v1, q = bf16((B, Hkv, 1, d), 2).cuda(), bf16((B, Hkv, 1, d), 3).cuda(), bf16((B, Hq, d), 4).cuda()
    wk = bf16((Hkv, d, 64), 5, 0.1).cuda()
    mask = torch.ones((B, Hq, nb), dtype=torch.uint8, device="cuda")
    ws = torch.empty(seer.seer_workspace_bytes(seer.SEER_CALL_BLOCK_SPARSE_DECODE_QUANT,
                                               seer.seer_shape(B, Hq, Hkv, L, d)), dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros_like(q), torch.zeros((B, Hq), device="cuda")) for _ in range(2)]
    kt = torch.zeros((B, Hkv, nb, 64), device="cuda")

    def step(i):
        seer.seer_kv_write(cache, k1, v1, start=lens, start_pos=-1)
        seer.seer_gate_key_cache_quant(cache, wk, L, kt=kt, lens=lens)
        seer.seer_block_sparse_decode_quant(q, cache, mask, L, lens=lens, o=outs[i][0], lse=outs[i][1], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            step(i)
    for r, (ln, i) in enumerate((([101, 258], 0), ([102, 259], 1), ([65, 500], 0), ([0, 1], 1))):
        lens.copy_(dev32(ln))
        k1.copy_(bf16(k1.shape, 30 + r))
        v1.copy_(bf16(k1.shape, 40 + r))
        mask.copy_((torch.rand(mask.shape, generator=torch.Generator().manual_seed(r)) < 0.6).to(torch.uint8))
        graphs[i].replay()
        torch.cuda.synchronize()
        if ln[0] == 0:                                      # position -1: refused on the device, the rest done
            with pytest.raises(seer.SeerError):
                seer.seer_check_status()
        else:
            seer.seer_check_status()
        held = parts(cache, table)
        check_decode(*outs[i], q, held, mask.cpu(), ln)
        check_gate(kt, held[0], wk, ln, 0, False)


def test_two_streams_at_once():
    """Calls on two streams of one cache and on a stream that is not the current one: the same results."""
    cache, q, mask, o, lse = attend(8, 128, 2, 8, 2, 3000, 0.5, seed=31)
    qd, md = q.cuda(), mask.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for r in range(20):
        got.append(seer.seer_block_sparse_decode_quant(qd, cache, md, 3000, return_lse=True, stream=streams[r % 2]))
    raw = seer.seer_kv_read(cache, 64, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, o) and torch.equal(b, lse)
    again = seer.seer_kv_read(cache, 64)
    assert torch.equal(raw[0], again[0]) and torch.equal(raw[1], again[1])


def test_decode_wait_timeout_is_reported_and_recoverable():
    """With the wait limit at 0 the first unfinished copy gives up: a status, no fault; the next call is exact.
    The cache is long enough that every warp waits for some of its copies."""
    cache, q, mask, o, lse = attend(4, 128, 2, 8, 2, 60000, 1.0, seed=41)
    try:
        seer.seer_set_wait_timeout_ns(0)
        seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), 60000)
        with pytest.raises(seer.SeerError) as e:
            seer.seer_check_status()
        assert e.value.status == seer.SEER_ERR_TIMEOUT
    finally:
        seer.seer_set_wait_timeout_ns(2_000_000_000)
    o2, l2 = seer.seer_block_sparse_decode_quant(q.cuda(), cache, mask.cuda(), 60000, return_lse=True)
    seer.seer_check_status()
    assert torch.equal(o, o2) and torch.equal(lse, l2)


# ------------------------------------------------------------------ kernels that start while the one before them ends

def chain(cache, kv, q, wk, wq, mask, L, between, side=None):
    """Rows over rows of the same places, each read, pooled and attended to by the call behind it."""
    B, Hq, d = q.shape
    n = kv[0][0].shape[2]
    outs = []
    for i, (k, v) in enumerate(kv):
        at = (i % 2) * (L - n)
        seer.seer_kv_write(cache, k, v, start_pos=at)
        between()
        rows = seer.seer_kv_read(cache, n, start_pos=at, k=torch.empty_like(k), v=torch.empty_like(v))
        between()
        kt = seer.seer_gate_key_cache_quant(cache, wk, L)
        between()
        scores = seer.seer_decode_gate_scores_cached(q, kt, wq, L, kt.shape[1])
        lse = torch.zeros((B, Hq), device="cuda")
        if side is not None:                                # a stream beside it reads the same cache
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                other = seer.seer_block_sparse_decode_quant(q, cache, mask, L)
        o = seer.seer_block_sparse_decode_quant(q, cache, mask, L, lse=lse)[0]
        between()
        if side is not None:
            torch.cuda.current_stream().wait_stream(side)
            outs.append(other)
        q = o                                               # the next step's token from this one's output
        outs += [*rows, kt, scores, o, lse]
    return outs


@pytest.mark.parametrize("bits,d", FORMATS)
@pytest.mark.parametrize("B,Hkv,g,L", [(8, 4, 4, 4096), (1, 2, 16, 700), (40, 4, 10, 2000)])
def test_calls_back_to_back(bits, d, B, Hkv, g, L):
    """The same bits whether each call's kernels follow at once, after a wait on the host, or from a captured graph."""
    nb, dg, steps = -(-L // 64), 64, 12
    n = L // 2
    kv = [(bf16((B, Hkv, n, d), 2 * i).cuda(), bf16((B, Hkv, n, d), 2 * i + 1).cuda()) for i in range(3)]
    kv = [kv[i % 3] for i in range(steps)]
    q, wk = bf16((B, Hkv * g, d), 7).cuda(), bf16((Hkv, d, dg), 8, 0.1).cuda()
    wq = bf16((Hkv * g, d, dg), 9, 0.1).cuda()
    mask = (torch.rand((B, Hkv * g, nb), generator=torch.Generator().manual_seed(1)) < 0.5).to(torch.uint8).cuda()

    def run(between=lambda: None, side=None):
        cache, _ = make_cache(B, Hkv, nb, d, bits, True, 4)
        seer.seer_kv_write(cache, torch.zeros((B, Hkv, L, d), dtype=torch.bfloat16, device="cuda"),
                           torch.zeros((B, Hkv, L, d), dtype=torch.bfloat16, device="cuda"))
        return chain(cache, kv, q, wk, wq, mask, L, between, side)

    want = run(torch.cuda.synchronize)
    seer.seer_check_status()
    for _ in range(3):
        got = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))
    cache, _ = make_cache(B, Hkv, nb, d, bits, True, 4)
    zero = torch.zeros((B, Hkv, L, d), dtype=torch.bfloat16, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        seer.seer_kv_write(cache, zero, zero)
        got = chain(cache, kv, q, wk, wq, mask, L, lambda: None, side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        seer.seer_check_status()
        assert all(torch.equal(a, b) for a, b in zip([x for i, x in enumerate(got) if i % 7], want, strict=True))
        assert all(torch.equal(got[7 * i], got[7 * i + 5]) for i in range(steps))
