"""The quantised KV cache of the decode step (include/seer.h, seer_kv_cache).

    cache = SeerKVCache.empty(B, Hkv, capacity, d, bits=4)
    seer_kv_write(cache, k, v)                                   # the prompt's rows
    kt = seer_gate_key_cache_quant(cache, wk, L)
    ...                                                          # then, a token at a time:
    seer_kv_write(cache, k_tok, v_tok, start_pos=L - 1)
    seer_gate_key_cache_quant(cache, wk, L, kt=kt, first_block=(L - 1) // 64)
    scores = seer_decode_gate_scores_cached(q_tok, kt, wq, L, Hkv)
    o = seer_block_sparse_decode_quant(q_tok, cache, seer_decode_block_mask(scores, density=0.1), L)

Like the other calls these marshal arguments only, and take their tensors as
they are on the stream they are given.  They run on the cache's device; what
they allocate belongs to the stream they run on.
"""
from __future__ import annotations

import ctypes

from . import _binding as B
from ._binding import _check, _need, _ptr, _torch


def seer_kv_record_bytes(bits: int, d: int) -> int:
    """Bytes of a cache record: one head's 64 tokens of K and V."""
    n = int(B.lib().seer_kv_record_bytes(int(bits), int(d)))
    if n == 0:
        raise B.SeerError(B.SEER_ERR_UNSUPPORTED, B.seer_last_error())
    return n


class SeerKVCache:
    """Pages u8 [n_pages, Hkv, record] and, for sequences that share them, a block table int32 [B, max_blocks]
    (without one, page b * max_blocks + j is block j of sequence b)."""

    def __init__(self, pages, d: int, bits: int, block_table=None, batch: int = 1):
        torch = _torch()
        _need(bits in (4, 8) and d in (64, 128), "a cache has 4 or 8 bits and a head dim of 64 or 128")
        _need(pages.dtype == torch.uint8 and pages.dim() == 3 and pages.is_contiguous(),
              "pages must be contiguous uint8 [n_pages, Hkv, record]")
        _need(pages.shape[2] == seer_kv_record_bytes(bits, d), "pages' last dimension must be the record's bytes")
        if block_table is not None:
            _need(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.is_contiguous(),
                  "block_table must be contiguous int32 [B, max_blocks]")
            _need(block_table.device == pages.device, "block_table must be on the pages' device")
            self.B, self.max_blocks = block_table.shape
        else:
            _need(batch >= 1 and pages.shape[0] % batch == 0, "pages must be batch * max_blocks without a block table")
            self.B, self.max_blocks = batch, pages.shape[0] // batch
        self.pages, self.block_table, self.d, self.bits, self.Hkv = pages, block_table, d, bits, pages.shape[1]
        self._c = B.seer_kv_cache(bits, pages.shape[0], self.max_blocks, _ptr(pages), _ptr(block_table))

    @classmethod
    def empty(cls, Bsz: int, Hkv: int, capacity: int, d: int, bits: int = 4, device="cuda"):
        """A cache of ceil(capacity / 64) blocks per sequence; its contents are whatever the memory held."""
        n = -(-capacity // B.BLOCK)
        pages = _torch().empty((Bsz * n, Hkv, seer_kv_record_bytes(bits, d)), dtype=_torch().uint8, device=device)
        return cls(pages, d, bits, batch=Bsz)

    @property
    def capacity(self) -> int:
        return self.max_blocks * B.BLOCK


def _on(device, stream, call):
    """call(stream pointer) with `device` current and, if a stream is given, that stream current too: what torch
    allocates in it then belongs to the stream that uses it."""
    torch = _torch()
    _need(device.type == "cuda", "the cache must be on a CUDA device")
    if stream is None and device.index == torch.cuda.current_device():
        return call(torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(device):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _per_sequence(cache, **named):
    for name, t in named.items():
        if t is not None:
            _need(t.dtype == _torch().int32 and t.shape == (cache.B,) and t.is_contiguous() and
                  t.device == cache.pages.device, f"{name} must be int32 [B] on the cache's device")


def _strides(t, name):
    st = [s if n > 1 else 0 for n, s in zip(t.shape[:3], t.stride())]
    _need(t.stride(3) == 1 and all(s % 8 == 0 for s in st) and t.data_ptr() % 16 == 0,
          f"{name}: the last dimension must be contiguous, the other strides multiples of 8, the start 16-byte aligned")
    return st


def seer_kv_write(cache, k, v, start=None, count=None, start_pos: int = 0, stream=None) -> None:
    """Quantise rows k, v (bf16 [B,Hkv,n,d], any row strides) into the cache at positions start[b] + start_pos + t,
    t < min(count[b], n) (start, count: device int32 [B]; absent: 0 and n)."""
    torch = _torch()
    _need(k.dim() == 4 and k.shape == v.shape and k.shape[0] == cache.B and k.shape[1] == cache.Hkv and
          k.shape[3] == cache.d, "k and v must be [B,Hkv,n,d] of the cache")
    _need(k.dtype == v.dtype == torch.bfloat16, "k and v must be bf16")
    _need(k.device == v.device == cache.pages.device, "k and v must be on the cache's device")
    _per_sequence(cache, start=start, count=count)
    rows = B.seer_kv_rows(_ptr(k), _ptr(v), *_strides(k, "k"), *_strides(v, "v"))
    sh = B.seer_shape(cache.B, cache.Hkv, cache.Hkv, k.shape[2], cache.d)
    _on(cache.pages.device, stream, lambda st: _check(B.lib().seer_kv_write(
        ctypes.byref(sh), ctypes.byref(cache._c), ctypes.byref(rows), _ptr(start), _ptr(count), int(start_pos), st)))


def seer_kv_read(cache, n: int, start=None, count=None, start_pos: int = 0, k=None, v=None, stream=None):
    """K and V (bf16 [B,Hkv,n,d]) as the cache holds them from position start[b] + start_pos on; rows from count[b] on
    are not written (zero where the tensor is not given)."""
    torch = _torch()
    shape = (cache.B, cache.Hkv, n, cache.d)
    for name, t in (("k", k), ("v", v)):
        _need(t is None or (t.dtype == torch.bfloat16 and tuple(t.shape) == shape and t.is_contiguous() and
                            t.device == cache.pages.device),
              f"{name} must be contiguous bf16 [B,Hkv,n,d] on the cache's device")
    _per_sequence(cache, start=start, count=count)
    sh = B.seer_shape(cache.B, cache.Hkv, cache.Hkv, int(n), cache.d)

    def call(st):
        make = torch.empty if count is None else torch.zeros
        ko, vo = (make(shape, dtype=torch.bfloat16, device=cache.pages.device) if t is None else t for t in (k, v))
        _check(B.lib().seer_kv_read(ctypes.byref(sh), ctypes.byref(cache._c), _ptr(start), _ptr(count), int(start_pos),
                                    _ptr(ko), _ptr(vo), st))
        return ko, vo

    return _on(cache.pages.device, stream, call)


def seer_gate_key_cache_quant(cache, wk, L: int, kt=None, first_block: int = 0, lens=None, rope_theta: float = 5e5,
                              stream=None, wk_head_stride: int | None = None, k_maxmin: bool = False):
    """seer_gate_key_cache on the quantised cache: key rows fp32 [B,Hkv,nb,d_gate] of blocks first_block.. of a cache
    of L tokens, or of lens[b] (device int32 [B]) tokens each."""
    torch = _torch()
    dev, dk = cache.pages.device, 2 * cache.d if k_maxmin else cache.d
    _need(wk.dtype == torch.bfloat16 and wk.is_contiguous() and wk.device == dev, "wk must be contiguous bf16 on the cache's device")
    _need(wk.dim() in (2, 3) and wk.shape[-2] == dk and (wk.dim() == 2 or wk.shape[0] == cache.Hkv),
          "wk must be [%d, d_gate] or [Hkv, %d, d_gate]" % (dk, dk))
    dg, nb = wk.shape[-1], -(-L // B.BLOCK)
    _per_sequence(cache, lens=lens)
    if wk_head_stride is None:
        wk_head_stride = 0 if wk.dim() == 2 else dk * dg
    shape = (cache.B, cache.Hkv, nb, dg)
    _need(kt is None or (kt.dtype == torch.float32 and kt.is_contiguous() and tuple(kt.shape) == shape and
                         kt.device == dev), "kt must be contiguous fp32 [B,Hkv,nb,d_gate] on the cache's device")
    sh = B.seer_shape(cache.B, cache.Hkv, cache.Hkv, int(L), cache.d)
    gp = B.seer_gate_params(int(dg), float(rope_theta), 0, int(wk_head_stride), int(bool(k_maxmin)))

    def call(st):
        out = torch.empty(shape, dtype=torch.float32, device=dev) if kt is None else kt
        _check(B.lib().seer_gate_key_cache_quant(ctypes.byref(sh), ctypes.byref(cache._c), _ptr(lens), _ptr(wk),
                                                 ctypes.byref(gp), int(first_block), _ptr(out), st))
        return out

    return _on(dev, stream, call)


def seer_block_sparse_decode_quant(q_tok, cache, mask, L: int, lens=None, softmax_scale: float = 0.0, o=None, lse=None,
                                   return_lse: bool = False, workspace=None, stream=None):
    """seer_block_sparse_decode on the quantised cache: q_tok bf16 [B,Hq,d], mask u8 [B,Hq,ceil(L/64)], sequences of L
    tokens or of lens[b] (device int32 [B]) each; returns o bf16 [B,Hq,d] (and lse)."""
    torch = _torch()
    dev, nb = cache.pages.device, -(-L // B.BLOCK)
    _need(q_tok.dim() == 3 and q_tok.shape[0] == cache.B and q_tok.shape[2] == cache.d, "q_tok must be [B,Hq,d] of the cache")
    Hq = q_tok.shape[1]
    _need(Hq % cache.Hkv == 0, "Hq must be a multiple of the cache's Hkv")
    _need(q_tok.dtype == torch.bfloat16 and mask.dtype == torch.uint8, "bf16 q_tok, u8 mask")
    _need(tuple(mask.shape) == (cache.B, Hq, nb), "mask must be [B,Hq,ceil(L/64)]")
    _need(q_tok.is_contiguous() and mask.is_contiguous(), "tensors must be contiguous")
    _need(q_tok.device == mask.device == dev, "q_tok and mask must be on the cache's device")
    _per_sequence(cache, lens=lens)
    _need(o is None or (o.dtype == torch.bfloat16 and o.shape == q_tok.shape and o.is_contiguous() and o.device == dev),
          "o must be contiguous bf16 [B,Hq,d] on the cache's device")
    _need(lse is None or (lse.dtype == torch.float32 and tuple(lse.shape) == (cache.B, Hq) and lse.is_contiguous() and
                          lse.device == dev), "lse must be contiguous fp32 [B,Hq] on the cache's device")
    sh = B.seer_shape(cache.B, Hq, cache.Hkv, int(L), cache.d)

    def call(st):
        out = torch.empty_like(q_tok) if o is None else o
        ls = torch.empty((cache.B, Hq), dtype=torch.float32, device=dev) if return_lse and lse is None else lse
        ws, wsb = B._workspace(B.SEER_CALL_BLOCK_SPARSE_DECODE_QUANT, sh, dev, workspace)
        _check(B.lib().seer_block_sparse_decode_quant(
            ctypes.byref(sh), _ptr(q_tok), ctypes.byref(cache._c), _ptr(lens), _ptr(mask), float(softmax_scale),
            _ptr(out), _ptr(ls), _ptr(ws), wsb, st))
        return (out, ls) if ls is not None else out

    return _on(dev, stream, call)
