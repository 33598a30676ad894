"""Host-side checks of the quantised-cache calls: refusals before any launch,
record sizes, the wrapper's checks.  No test here launches a kernel."""
import ctypes

import numpy as np
import pytest
import torch

import kv_reference as ref
import long_context_prefill_attngate_b200 as seer
from long_context_prefill_attngate_b200 import build as seer_build

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    seer_build.build()
    return seer.lib()


def shape(B=2, Hq=8, Hkv=2, S=100, d=128):
    return ctypes.byref(seer.seer_shape(B, Hq, Hkv, S, d))


def cache(bits=4, n_pages=8, max_blocks=4, pages=0x10000, table=None):
    return ctypes.byref(seer.seer_kv_cache(bits, n_pages, max_blocks, pages, table))


def rows(k=0x10000, v=0x10000, kt=128, vt=128):
    return ctypes.byref(seer.seer_kv_rows(k, v, 0, 0, kt, 0, 0, vt))


def calls(L, sh, c):
    gp = ctypes.byref(seer.seer_gate_params(64, 5e5, 0, 0, 0))
    return (lambda: L.seer_kv_write(sh, c, rows(), None, None, 0, None),
            lambda: L.seer_kv_read(sh, c, None, None, 0, P, P, None),
            lambda: L.seer_gate_key_cache_quant(sh, c, None, P, gp, 0, P, None),
            lambda: L.seer_block_sparse_decode_quant(sh, P, c, None, P, 0.0, P, P, P, 1 << 30, None))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_record_bytes(L, bits, d):
    assert seer.seer_kv_record_bytes(bits, d) == ref.record_bytes(bits, d)
    assert seer.seer_kv_record_bytes(bits, d) % 32 == 0          # halves stay 16-byte aligned


@pytest.mark.parametrize("bits,d", [(2, 128), (16, 128), (4, 96), (8, 0), (0, 64)])
def test_record_bytes_refuses(L, bits, d):
    with pytest.raises(seer.SeerError) as e:
        seer.seer_kv_record_bytes(bits, d)
    assert e.value.status == seer.SEER_ERR_UNSUPPORTED


@pytest.mark.parametrize("sh,c,status,msg", [
    (dict(d=96), {}, seer.SEER_ERR_UNSUPPORTED, "head dim"),
    (dict(S=0), {}, seer.SEER_ERR_INVALID_ARG, "positive"),
    (dict(Hq=7), {}, seer.SEER_ERR_INVALID_ARG, "multiple of Hkv"),
    ({}, dict(bits=3), seer.SEER_ERR_UNSUPPORTED, "bits"),
    ({}, dict(pages=None), seer.SEER_ERR_INVALID_ARG, "pages"),
    ({}, dict(pages=0x10008), seer.SEER_ERR_INVALID_ARG, "aligned"),
    ({}, dict(n_pages=0), seer.SEER_ERR_INVALID_ARG, "positive"),
    ({}, dict(max_blocks=0), seer.SEER_ERR_INVALID_ARG, "positive"),
    ({}, dict(max_blocks=16385, n_pages=1 << 20), seer.SEER_ERR_UNSUPPORTED, "max_blocks"),
    ({}, dict(n_pages=7), seer.SEER_ERR_INVALID_ARG, "block table"),
    (dict(B=65536, Hq=2), dict(n_pages=1 << 30), seer.SEER_ERR_UNSUPPORTED, "65535"),
])
def test_every_call_refuses_a_bad_cache(L, sh, c, status, msg):
    for call in calls(L, shape(**sh), cache(**c)):
        assert call() == status and msg in seer.seer_last_error()


def test_length_beyond_the_cache_is_refused(L):
    gate, decode = calls(L, shape(S=257), cache())[2:]
    for call in (gate, decode):
        assert call() == seer.SEER_ERR_INVALID_ARG and "4 per sequence" in seer.seer_last_error()


def test_null_and_misaligned_arguments(L):
    sh, c = shape(), cache()
    gp = ctypes.byref(seer.seer_gate_params(64, 5e5, 0, 0, 0))
    assert L.seer_kv_write(sh, None, rows(), None, None, 0, None) == seer.SEER_ERR_INVALID_ARG
    assert L.seer_kv_write(sh, c, None, None, None, 0, None) == seer.SEER_ERR_INVALID_ARG
    for bad in (rows(k=None), rows(v=0x10008), rows(kt=100), rows(vt=-8)):
        assert L.seer_kv_write(sh, c, bad, None, None, 0, None) == seer.SEER_ERR_INVALID_ARG
    assert L.seer_kv_read(sh, c, None, None, 0, None, None, None) == seer.SEER_ERR_INVALID_ARG
    assert L.seer_kv_read(sh, c, None, None, 0, ODD, P, None) == seer.SEER_ERR_INVALID_ARG
    g = lambda wk=P, kt=P, first=0, params=gp: L.seer_gate_key_cache_quant(  # noqa: E731
        sh, c, None, wk, params, first, kt, None)
    assert g(wk=None) == seer.SEER_ERR_INVALID_ARG and g(kt=None) == seer.SEER_ERR_INVALID_ARG
    assert g(params=None) == seer.SEER_ERR_INVALID_ARG
    assert g(first=-1) == seer.SEER_ERR_INVALID_ARG and g(first=3) == seer.SEER_ERR_INVALID_ARG
    assert g(params=ctypes.byref(seer.seer_gate_params(63, 5e5, 0, 0, 0))) == seer.SEER_ERR_UNSUPPORTED
    dec = lambda q=P, m=P, o=P, s=0.0, ws=P, n=1 << 30: L.seer_block_sparse_decode_quant(  # noqa: E731
        sh, q, c, None, m, s, o, None, ws, n, None)
    assert dec(q=None) == seer.SEER_ERR_INVALID_ARG and dec(m=None) == seer.SEER_ERR_INVALID_ARG
    assert dec(o=None) == seer.SEER_ERR_INVALID_ARG and dec(q=ODD) == seer.SEER_ERR_INVALID_ARG
    assert dec(s=float("nan")) == seer.SEER_ERR_INVALID_ARG and dec(s=float("inf")) == seer.SEER_ERR_INVALID_ARG
    assert dec(ws=None) == seer.SEER_ERR_WORKSPACE and dec(n=16) == seer.SEER_ERR_WORKSPACE


def test_workspace_size(L):
    sh = seer.seer_shape(1, 32, 8, 32768, 128)
    assert seer.seer_workspace_bytes(seer.SEER_CALL_BLOCK_SPARSE_DECODE_QUANT, sh) > 0


def test_wrapper_checks(L):
    """ValueErrors of the Python calls; a cache on the CPU is the last thing they refuse."""
    c = seer.SeerKVCache.empty(2, 2, 200, 128, bits=4, device="cpu")
    assert c.capacity == 256 and c.max_blocks == 4 and c.pages.shape == (8, 2, 10240)
    bf = dict(dtype=torch.bfloat16)
    k = torch.zeros((2, 2, 5, 128), **bf)
    q, m = torch.zeros((2, 4, 128), **bf), torch.zeros((2, 4, 4), dtype=torch.uint8)
    wk = torch.zeros((2, 128, 64), **bf)
    i32 = torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: seer.SeerKVCache(c.pages[:, :, :-16].contiguous(), 128, 4),
        lambda: seer.SeerKVCache(c.pages, 128, 8),
        lambda: seer.SeerKVCache(c.pages, 128, 4, batch=3),
        lambda: seer.SeerKVCache(c.pages, 128, 4, block_table=i32),
        lambda: seer.SeerKVCache(c.pages, 128, 4, block_table=torch.zeros((2, 4), dtype=torch.int64)),
        lambda: seer.SeerKVCache(c.pages.transpose(0, 1), 128, 4),
        lambda: seer.seer_kv_write(c, k.float(), k.float()),
        lambda: seer.seer_kv_write(c, k, k[:, :, :4]),
        lambda: seer.seer_kv_write(c, k[:1], k[:1]),
        lambda: seer.seer_kv_write(c, k.transpose(2, 3).contiguous().transpose(2, 3), k),
        lambda: seer.seer_kv_write(c, k, k, start=i32.long()),
        lambda: seer.seer_kv_write(c, k, k, count=i32[:1]),
        lambda: seer.seer_kv_read(c, 5, k=k[:, :, :4]),
        lambda: seer.seer_kv_read(c, 5, start=i32.float()),
        lambda: seer.seer_gate_key_cache_quant(c, wk[:, :64], 200),
        lambda: seer.seer_gate_key_cache_quant(c, wk[:1], 200),
        lambda: seer.seer_gate_key_cache_quant(c, wk, 200, kt=torch.zeros(2, 2, 3, 64)),
        lambda: seer.seer_block_sparse_decode_quant(q[:, :3].contiguous(), c, m, 200),
        lambda: seer.seer_block_sparse_decode_quant(q, c, m[..., :3].contiguous(), 200),
        lambda: seer.seer_block_sparse_decode_quant(q, c, m.bool(), 200),
        lambda: seer.seer_block_sparse_decode_quant(q, c, m, 200, lens=i32.long()),
        lambda: seer.seer_block_sparse_decode_quant(q, c, m, 200, o=q.float()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: seer.seer_kv_write(c, k, k, start=i32, count=i32), lambda: seer.seer_kv_read(c, 5),
                 lambda: seer.seer_gate_key_cache_quant(c, wk, 200, lens=i32),
                 lambda: seer.seer_block_sparse_decode_quant(q, c, m, 200, lens=i32)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_reference_layout_is_a_bijection():
    """Every byte of a record has one meaning, and packing is undone by unpacking."""
    rng = np.random.default_rng(0)
    for bits in (4, 8):
        for d in (64, 128):
            pl = ref._places(bits, d)
            assert sorted(np.concatenate([p for t in pl for p in t])) == list(range(ref.record_bytes(bits, d)))
            pages = rng.integers(0, 256, (1, 1, ref.record_bytes(bits, d)), dtype=np.uint8)
            x = ref.bf16_round(rng.standard_normal((2, d)))[0]
            kq, vq = (ref.quantise(y, bits) for y in x)
            ref.pack(pages, 0, 0, 37, kq, vq, bits, d)
            for got, want in zip(ref.unpack(pages, bits, d), (kq, vq)):
                for a, b in zip(got, want):
                    assert np.array_equal(a[0, 0, 37], b)
