"""The quantised KV cache of the decode step (include/seer.h, seer_kv_cache).

    cache = SeerKVCache.empty(B, Hkv, capacity, d, bits=4)
    seer_kv_write(cache, k, v)                                   # the prompt's rows
    kt = seer_gate_key_cache_quant(cache, wk, L)
    ...                                                          # then, a token at a time:
    seer_kv_write(cache, k_tok, v_tok, start_pos=L - 1)
    seer_gate_key_cache_quant(cache, wk, L, kt=kt, first_block=(L - 1) // 64)
    scores = seer_decode_gate_scores_cached(q_tok, kt, wq, L, Hkv)
    o = seer_block_sparse_decode_quant(q_tok, cache, seer_decode_block_mask(scores, density=0.1), L)

For sequences of their own lengths (device int32 [B], the new token counted) the four calls of a step take them as
lens=..., the write as start=lens, start_pos=-1 (with count=0 for idle slots, whose row would have no place), and L is
the longest.

Like the other calls these marshal arguments only, and take their tensors as
they are on the stream they are given.  They run on the cache's device; what
they allocate belongs to the stream they run on.  A decode step makes these
calls once per layer and token, so their checks are plain comparisons.
"""
from __future__ import annotations

import ctypes
import functools
import operator

import torch

from . import _binding as B
from ._binding import _check, _need, lib

try:                                                # without a Stream object, and for devices that tensors live on
    from torch._C import _cuda_getCurrentRawStream as _current_stream, _cuda_getDevice as _current_device
except ImportError:
    _current_device = torch.cuda.current_device

    def _current_stream(dev):
        return torch.cuda.current_stream(dev).cuda_stream

_byref = ctypes.byref
_bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@functools.lru_cache(maxsize=None)
def seer_kv_record_bytes(bits: int, d: int) -> int:
    """Bytes of a cache record: one head's 64 tokens of K and V."""
    n = int((B._lib or lib()).seer_kv_record_bytes(int(bits), int(d)))
    if n == 0:
        raise B.SeerError(B.SEER_ERR_UNSUPPORTED, B.seer_last_error())
    return n


@functools.lru_cache(maxsize=1024)
def _attention_workspace(Bsz: int, Hq: int, Hkv: int, d: int) -> int:
    """Bytes of the attention's workspace: the same for every L."""
    return B.seer_workspace_bytes(B.SEER_CALL_BLOCK_SPARSE_DECODE_QUANT, B.seer_shape(Bsz, Hq, Hkv, 1, d))


class SeerKVCache:
    """Pages u8 [n_pages, Hkv, record] and, for sequences that share them, a block table int32 [B, max_blocks]
    (without one, page b * max_blocks + j is block j of sequence b).

    The tensors' contents may change between calls, a table's entries among them; the tensors themselves and the sizes
    may not (the calls keep their addresses): another table or pool is another SeerKVCache."""

    __slots__ = ("_pages", "_block_table", "_d", "_bits", "_Hkv", "_B", "_max_blocks", "_dev", "_c")

    pages, block_table, d, bits, Hkv, B, max_blocks = (
        property(operator.attrgetter(n)) for n in ("_pages", "_block_table", "_d", "_bits", "_Hkv", "_B", "_max_blocks"))

    def __init__(self, pages, d: int, bits: int, block_table=None, batch: int = 1):
        _need((bits == 4 or bits == 8) and (d == 128 or d == 64), "a cache has 4 or 8 bits and a head dim of 64 or 128")
        _need(pages.dtype is _u8 and pages.dim() == 3 and pages.is_contiguous(),
              "pages must be contiguous uint8 [n_pages, Hkv, record]")
        n_pages, self._Hkv, record = pages.shape
        _need(record == seer_kv_record_bytes(bits, d), "pages' last dimension must be the record's bytes")
        self._dev = pages.get_device()
        if block_table is not None:
            _need(block_table.dtype is _i32 and block_table.dim() == 2 and block_table.is_contiguous(),
                  "block_table must be contiguous int32 [B, max_blocks]")
            _need(block_table.get_device() == self._dev, "block_table must be on the pages' device")
            self._B, self._max_blocks = block_table.shape
        else:
            _need(batch >= 1 and n_pages % batch == 0, "pages must be batch * max_blocks without a block table")
            self._B, self._max_blocks = batch, n_pages // batch
        self._pages, self._block_table, self._d, self._bits = pages, block_table, d, bits
        self._c = B.seer_kv_cache(bits, n_pages, self._max_blocks, pages.data_ptr(),
                                  None if block_table is None else block_table.data_ptr())

    @classmethod
    def empty(cls, Bsz: int, Hkv: int, capacity: int, d: int, bits: int = 4, device="cuda"):
        """A cache of ceil(capacity / 64) blocks per sequence; its contents are whatever the memory held."""
        n = -(-capacity // B.BLOCK)
        pages = torch.empty((Bsz * n, Hkv, seer_kv_record_bytes(bits, d)), dtype=_u8, device=device)
        return cls(pages, d, bits, batch=Bsz)

    @property
    def capacity(self) -> int:
        return self._max_blocks * B.BLOCK


def _elsewhere(fn, dev: int, stream, *args):
    """fn(*args) with device `dev` current and, if a stream is given, that stream current too: what torch allocates
    then belongs to the stream that uses it."""
    _need(dev >= 0, "the cache must be on a CUDA device")
    _need(getattr(stream, "device_index", dev) == dev, "the stream must be on the cache's device")
    with torch.cuda.device(dev):
        if stream is None:
            return fn(*args)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return fn(*args)


def _per_sequence(cache, name, t):
    """The pointer of an optional int32 [B] of the cache's device."""
    if t is None:
        return None
    if t.dtype is _i32 and t.shape == (cache._B,) and t.is_contiguous() and t.get_device() == cache._dev:
        return t.data_ptr()
    raise ValueError(name)


_INT32 = range(-2 ** 31, 2 ** 31)
_POS = "start_pos must be within 32 bits"
_START = "start must be int32 [B] on the cache's device"
_COUNT = "count must be int32 [B] on the cache's device"
_LENS = "lens must be int32 [B] on the cache's device"


def _strides(t, shape, message):
    sb, sh, st, sc = t.stride()
    if shape[0] == 1:
        sb = 0
    if shape[1] == 1:
        sh = 0
    if shape[2] == 1:
        st = 0
    _need(sc == 1 and not (sb | sh | st) & 7 and not t.data_ptr() & 15, message)
    return sb, sh, st


_LAYOUT = ("k and v: the last dimension must be contiguous, the other strides multiples of 8, the start 16-byte aligned")


def seer_kv_write(cache, k, v, start=None, count=None, start_pos: int = 0, stream=None) -> None:
    """Quantise rows k, v (bf16 [B,Hkv,n,d], any row strides) into the cache at positions start[b] + start_pos + t,
    t < min(count[b], n) (start, count: device int32 [B]; absent: 0 and n)."""
    shape = k.shape
    _need(len(shape) == 4 and shape == v.shape and shape[0] == cache._B and shape[1] == cache._Hkv and shape[3] == cache._d,
          "k and v must be [B,Hkv,n,d] of the cache")
    _need(k.dtype is _bf16 and v.dtype is _bf16, "k and v must be bf16")
    dev = cache._dev
    _need(k.get_device() == dev and v.get_device() == dev, "k and v must be on the cache's device")
    _need(start_pos in _INT32, _POS)
    sp, cp = _per_sequence(cache, _START, start), _per_sequence(cache, _COUNT, count)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(seer_kv_write, dev, stream, cache, k, v, start, count, start_pos)
    rows = B.seer_kv_rows(k.data_ptr(), v.data_ptr(), *_strides(k, shape, _LAYOUT), *_strides(v, shape, _LAYOUT))
    sh = B.seer_shape(cache._B, cache._Hkv, cache._Hkv, shape[2], cache._d)
    st = (B._lib or lib()).seer_kv_write(_byref(sh), _byref(cache._c), _byref(rows), sp, cp, int(start_pos),
                                         _current_stream(dev))
    if st:
        _check(st)


def seer_kv_read(cache, n: int, start=None, count=None, start_pos: int = 0, k=None, v=None, stream=None):
    """K and V (bf16 [B,Hkv,n,d]) as the cache holds them from position start[b] + start_pos on; rows from count[b] on
    and rows that the cache does not have are not written (zero where the tensor is not given)."""
    shape = (cache._B, cache._Hkv, n, cache._d)
    for t in (k, v):
        _need(t is None or (t.dtype is _bf16 and t.shape == shape and t.is_contiguous() and t.get_device() == cache._dev),
              "k and v must be contiguous bf16 [B,Hkv,n,d] on the cache's device")
    _need(start_pos in _INT32, _POS)
    sp, cp = _per_sequence(cache, _START, start), _per_sequence(cache, _COUNT, count)
    dev = cache._dev
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(seer_kv_read, dev, stream, cache, n, start, count, start_pos, k, v)
    # zeros where the call may leave rows out: behind counts, outside the cache, on pages that a table does not have
    whole = count is None and start is None and cache._block_table is None and 0 <= start_pos <= 64 * cache._max_blocks - n
    make = torch.empty if whole else torch.zeros
    if k is None:
        k = make(*shape, dtype=_bf16, device=cache._pages.device)
    if v is None:
        v = make(*shape, dtype=_bf16, device=cache._pages.device)
    sh = B.seer_shape(cache._B, cache._Hkv, cache._Hkv, int(n), cache._d)
    st = (B._lib or lib()).seer_kv_read(_byref(sh), _byref(cache._c), sp, cp, int(start_pos), k.data_ptr(), v.data_ptr(),
                                        _current_stream(dev))
    if st:
        _check(st)
    return k, v


def seer_gate_key_cache_quant(cache, wk, L: int, kt=None, first_block: int = 0, lens=None, rope_theta: float = 5e5,
                              stream=None, wk_head_stride: int | None = None, k_maxmin: bool = False):
    """seer_gate_key_cache on the quantised cache: key rows fp32 [B,Hkv,nb,d_gate] of blocks first_block.. of a cache
    of L tokens, or of lens[b] (device int32 [B]) tokens each."""
    dev, dk, ws = cache._dev, 2 * cache._d if k_maxmin else cache._d, wk.shape
    _need(wk.dtype is _bf16 and wk.is_contiguous() and wk.get_device() == dev, "wk must be contiguous bf16 on the cache's device")
    _need(len(ws) in (2, 3) and ws[-2] == dk and (len(ws) == 2 or ws[0] == cache._Hkv),
          "wk must be [dk, d_gate] or [Hkv, dk, d_gate], dk = d (2 d with max+min pooling)")
    dg = ws[-1]
    if wk_head_stride is None:
        wk_head_stride = 0 if len(ws) == 2 else dk * dg
    _need(0 <= wk_head_stride and (cache._Hkv - 1) * wk_head_stride + dk * dg <= wk.numel(),
          "wk_head_stride leads out of wk")
    shape = (cache._B, cache._Hkv, -(-L // B.BLOCK), dg)
    _need(kt is None or (kt.dtype is _f32 and kt.shape == shape and kt.is_contiguous() and kt.get_device() == dev),
          "kt must be contiguous fp32 [B,Hkv,nb,d_gate] on the cache's device")
    _need(0 <= first_block <= shape[2], "first_block must be within the blocks of L")
    lp = _per_sequence(cache, _LENS, lens)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(seer_gate_key_cache_quant, dev, stream, cache, wk, L, kt, first_block, lens, rope_theta, None,
                          wk_head_stride, k_maxmin)
    if kt is None:
        kt = torch.empty(*shape, dtype=_f32, device=cache._pages.device)
    sh = B.seer_shape(cache._B, cache._Hkv, cache._Hkv, int(L), cache._d)
    gp = B.seer_gate_params(dg, float(rope_theta), 0, int(wk_head_stride), int(bool(k_maxmin)))
    st = (B._lib or lib()).seer_gate_key_cache_quant(_byref(sh), _byref(cache._c), lp, wk.data_ptr(), _byref(gp),
                                                     int(first_block), kt.data_ptr(), _current_stream(dev))
    if st:
        _check(st)
    return kt


def seer_block_sparse_decode_quant(q_tok, cache, mask, L: int, lens=None, softmax_scale: float = 0.0, o=None, lse=None,
                                   return_lse: bool = False, workspace=None, stream=None):
    """seer_block_sparse_decode on the quantised cache: q_tok bf16 [B,Hq,d], mask u8 [B,Hq,ceil(L/64)], sequences of L
    tokens or of lens[b] (device int32 [B]) each; returns o bf16 [B,Hq,d] (and lse)."""
    dev, qs = cache._dev, q_tok.shape
    _need(len(qs) == 3 and qs[0] == cache._B and qs[2] == cache._d, "q_tok must be [B,Hq,d] of the cache")
    Hq = qs[1]
    _need(Hq % cache._Hkv == 0, "Hq must be a multiple of the cache's Hkv")
    _need(q_tok.dtype is _bf16 and mask.dtype is _u8, "bf16 q_tok, u8 mask")
    _need(mask.shape == (cache._B, Hq, -(-L // B.BLOCK)), "mask must be [B,Hq,ceil(L/64)]")
    _need(q_tok.is_contiguous() and mask.is_contiguous(), "tensors must be contiguous")
    _need(q_tok.get_device() == dev and mask.get_device() == dev, "q_tok and mask must be on the cache's device")
    _need(o is None or (o.dtype is _bf16 and o.shape == qs and o.is_contiguous() and o.get_device() == dev),
          "o must be contiguous bf16 [B,Hq,d] on the cache's device")
    _need(lse is None or (lse.dtype is _f32 and lse.shape == (cache._B, Hq) and lse.is_contiguous() and
                          lse.get_device() == dev), "lse must be contiguous fp32 [B,Hq] on the cache's device")
    _need(workspace is None or (workspace.is_contiguous() and workspace.get_device() == dev),
          "workspace must be contiguous on the cache's device")
    lp = _per_sequence(cache, _LENS, lens)
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(seer_block_sparse_decode_quant, dev, stream, q_tok, cache, mask, L, lens, softmax_scale, o, lse,
                          return_lse, workspace)
    if o is None:
        o = torch.empty_like(q_tok)
    if lse is None and return_lse:
        lse = torch.empty(cache._B, Hq, dtype=_f32, device=cache._pages.device)
    if workspace is None:
        need = _attention_workspace(cache._B, Hq, cache._Hkv, cache._d)
        workspace = cache._pages.new_empty(need)
    else:
        need = workspace.numel() * workspace.element_size()
    sh = B.seer_shape(cache._B, Hq, cache._Hkv, int(L), cache._d)
    st = (B._lib or lib()).seer_block_sparse_decode_quant(
        _byref(sh), q_tok.data_ptr(), _byref(cache._c), lp, mask.data_ptr(), float(softmax_scale), o.data_ptr(),
        None if lse is None else lse.data_ptr(), workspace.data_ptr(), need, _current_stream(dev))
    if st:
        _check(st)
    return o if lse is None else (o, lse)
