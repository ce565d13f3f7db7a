"""The 4-bit KV cache: pages of block-scaled FP4 keys and values, the
attention that reads them, and the moves of the pages (``fp4_kv_*`` in
``include/fp4.h``, which states the layouts and the rules).

A serving step appends the new tokens' keys and values and attends::

    cache = new_kv_cache(pages, page_size, kv_heads, head_dim, "nvfp4", layers,
                         rht=True)
    batch = KVBatch(page_table, kv_lens, cu_q, max_q)   # lengths with the new tokens
    kv_append(cache, k, v, batch, layer)
    out = kv_attention(q, cache, batch, layer)

Prompts, chunks of prompts, several drafted tokens and single tokens are the
same two calls.  Tables stay on the device: ``kv_fork``, ``kv_free`` and
``kv_compact`` rewrite them there, nothing is read back.

Calls allocate the outputs and workspaces that are not passed in, on the
stream of the call, and raise on a refused argument.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

import block_scaled_bit_fp4_amd as fp4

KV_FORMATS = ("nvfp4", "mxfp4", "mxfp4_oas")
PAGE_SIZES = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128, 256)


class KVCache(NamedTuple):
    """All layers of a cache.  codes [layers, pages, heads, page_size,
    head_dim / 2] and scales [layers, pages, heads, page_size, head_dim /
    block], uint8; ``k_scale`` / ``v_scale``: float32 factors [layers]
    (NVFP4: the tensor scales; None for the MX formats)."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    fmt: str = "nvfp4"
    rht: bool = False
    rht_seed: int = 0


class KVBatch(NamedTuple):
    """The tokens of a call.  ``page_table`` int32 [sequences, columns] (-1: no
    page), ``kv_lens`` int32 [sequences] (new tokens included), ``cu_q`` int32
    [sequences + 1] (first new token of each sequence); ``max_q``: at least the
    most new tokens of a sequence; ``max_kv``: at least the longest length (0:
    what the columns can hold)."""
    page_table: torch.Tensor
    kv_lens: torch.Tensor
    cu_q: torch.Tensor
    max_q: int
    max_kv: int = 0


class _Cache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("layers", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("rht", ctypes.c_int32), ("rht_seed", ctypes.c_uint64), ("pages", ctypes.c_int64),
                ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class _Batch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("table_ld", ctypes.c_int64),
                ("kv_lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("columns", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32)]


def bind(L):
    """Argument types of the cache's entry points."""
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    C, B = ctypes.POINTER(_Cache), ctypes.POINTER(_Batch)
    L.fp4_kv_append.argtypes = [C, i32, B, vp, i64, i64, vp, i64, i64, i32, i64, vp]
    L.fp4_kv_gather.argtypes = [C, i32, B, vp, vp, i64, i64, i32, i64, vp]
    L.fp4_kv_attention_workspace_bytes.argtypes = [C, B, i32, i64, i32, i32]
    L.fp4_kv_attention_workspace_bytes.restype = sz
    L.fp4_kv_attention.argtypes = [C, i32, B, vp, i64, i64, i32, i64, ctypes.c_float, i32, i32, vp,
                                   i32, i64, i64, vp, vp, sz, vp]
    L.fp4_kv_copy_pages.argtypes = [C, vp, vp, vp, i32, vp]
    L.fp4_kv_fork.argtypes = [C, vp, i64, i64, i32, vp, vp, vp, vp, i32, vp, vp, sz, vp]
    L.fp4_kv_free.argtypes = [vp, i64, i64, i32, vp, vp, i64, i32, vp, i32, i32, i32, vp]
    L.fp4_kv_compact.argtypes = [C, vp, i64, i64, i32, vp, vp, vp, vp, sz, vp]
    for f in (L.fp4_kv_append, L.fp4_kv_gather, L.fp4_kv_attention, L.fp4_kv_copy_pages,
              L.fp4_kv_fork, L.fp4_kv_free, L.fp4_kv_compact):
        f.restype = i32


def new_kv_cache(pages: int, page_size: int, heads: int, head_dim: int, fmt: str = "nvfp4",
                 layers: int = 1, k_scale=1.0 / 448, v_scale=1.0 / 448, rht: bool = False,
                 rht_seed: int = 0, device="cuda") -> KVCache:
    """An empty cache.  ``k_scale`` / ``v_scale`` (NVFP4): a float for all
    layers, or one float32 per layer; the largest magnitude a layer can hold is
    6 * 448 times its factor (the default: 6), so a calibration's amax gives
    amax / (6 * 448)."""
    if fmt not in KV_FORMATS:
        raise ValueError("a cache is held in one of %s" % (KV_FORMATS,))
    if page_size not in PAGE_SIZES or head_dim not in HEAD_DIMS:
        raise ValueError("page_size is one of %s, head_dim one of %s" % (PAGE_SIZES, HEAD_DIMS))
    shape = (layers, pages, heads, page_size)

    def part(n):
        return torch.zeros(*shape, n, dtype=torch.uint8, device=device)

    def factor(v):
        if fmt != "nvfp4":
            return None
        t = torch.as_tensor(v, dtype=torch.float32, device=device)
        return t.expand(layers).contiguous()

    n, b = head_dim // 2, head_dim // fp4.BLOCK[fmt]
    return KVCache(part(n), part(b), part(n), part(b), factor(k_scale), factor(v_scale), fmt,
                   bool(rht), int(rht_seed))


def _need(ok, msg):
    if not ok:
        raise ValueError(msg)


def _ints(t, name, dims=1, device=None):
    if not (torch.is_tensor(t) and t.dtype == torch.int32 and t.dim() == dims and t.is_cuda
            and (t.numel() == 0 or t.shape[-1] == 1 or t.stride(-1) == 1)):
        raise ValueError("%s must be a %d-D int32 device tensor with dense rows" % (name, dims))
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    return t


def _cache(c: KVCache) -> _Cache:
    kc = c.k_codes
    if c.fmt not in KV_FORMATS:
        raise ValueError("a cache is held in one of %s" % (KV_FORMATS,))
    if kc.dim() != 5:
        raise ValueError("codes are [layers, pages, heads, page_size, head_dim / 2]")
    layers, pages, heads, page, half = kc.shape
    scales = (layers, pages, heads, page, 2 * half // fp4.BLOCK[c.fmt])
    if c.v_codes.shape != kc.shape or c.k_scales.shape != scales or c.v_scales.shape != scales:
        raise ValueError("the cache's arrays do not agree in shape")
    dev = kc.device
    for t in (kc, c.k_scales, c.v_codes, c.v_scales):
        if t.dtype != torch.uint8 or not t.is_contiguous() or not t.is_cuda or t.device != dev:
            raise ValueError("the cache's arrays are dense uint8 tensors on one device")
    ks = vs = None
    if c.fmt == "nvfp4":
        for t in (c.k_scale, c.v_scale):
            if t is not None and not (t.dtype == torch.float32 and t.numel() == layers
                                      and t.is_contiguous() and t.device == dev):
                raise ValueError("k_scale and v_scale are float32 [layers] on the cache's device")
        ks, vs = fp4._ptr(c.k_scale), fp4._ptr(c.v_scale)
    return _Cache(fp4.FORMATS[c.fmt], layers, heads, 2 * half, page, int(bool(c.rht)),
                  int(c.rht_seed) & (2**64 - 1), pages, kc.data_ptr(), c.k_scales.data_ptr(),
                  c.v_codes.data_ptr(), c.v_scales.data_ptr(), ks, vs)


def _batch(b: KVBatch, device) -> _Batch:
    t, n = b.page_table, b.kv_lens
    _ints(t, "page_table", 2, device)
    _ints(n, "kv_lens", 1, device)
    _ints(b.cu_q, "cu_q", 1, device)
    size = t.shape[0]
    if n.shape[0] != size or b.cu_q.shape[0] != size + 1:
        raise ValueError("page_table, kv_lens and cu_q are of different batches")
    return _Batch(t.data_ptr(), t.stride(0) if size > 1 else max(t.shape[1], 1), n.data_ptr(),
                  b.cu_q.data_ptr(), size, t.shape[1], int(b.max_q), int(b.max_kv))


def _rows(t, name, heads, dim, dtypes, device):
    """A [tokens, heads, head_dim] tensor with a dense last dimension; its
    strides (of a dimension of one, none that matter)."""
    if not torch.is_tensor(t) or t.dim() != 3 or t.shape[2] != dim or (heads and t.shape[1] != heads):
        raise ValueError("%s must be [tokens, %s, %d]" % (name, heads or "heads", dim))
    if t.dtype not in dtypes:
        raise TypeError("%s has type %s" % (name, t.dtype))
    if t.device != device or t.stride(2) != 1:
        raise ValueError("%s must be on %s with a dense last dimension" % (name, device))
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def _raise(st, name):
    if st != fp4.FP4_OK:
        raise fp4.FP4Error(st, name)


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, batch: KVBatch, layer: int = 0,
              stream=None) -> None:
    """Quantize the new tokens' keys and values ([tokens, heads, head_dim], BF16
    or FP32, any strides that keep rows 16-byte aligned: views of a fused
    projection, say) into their places in a layer."""
    c = _cache(cache)
    dev = cache.k_codes.device
    b = _batch(batch, dev)
    ks = _rows(k, "k", c.heads, c.head_dim, fp4.DTYPES, dev)
    vs = _rows(v, "v", c.heads, c.head_dim, fp4.DTYPES, dev)
    _need(k.shape == v.shape and k.dtype == v.dtype, "k and v must agree in shape and type")
    _raise(fp4.load().fp4_kv_append(c, layer, b, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0],
                                    vs[1], fp4.DTYPES[k.dtype], k.shape[0], fp4._stream(stream)),
           "fp4_kv_append")


def kv_gather(cache: KVCache, batch: KVBatch, tokens: int, layer: int = 0,
              out_dtype=torch.bfloat16, out=None, stream=None):
    """The keys and values that the batch's new tokens have in the cache, as
    (k, v) [tokens, heads, head_dim].  Tokens that the cache does not hold read
    as zeros; rows of no sequence are left as they are.  ``out``: a pair of
    tensors of equal strides to write."""
    c = _cache(cache)
    dev = cache.k_codes.device
    b = _batch(batch, dev)
    if out is None:
        with fp4._Alloc(stream) as al:
            shape = (tokens, c.heads, c.head_dim)
            out = (al.empty(shape, out_dtype, dev, "k"), al.empty(shape, out_dtype, dev, "v"))
    k, v = out
    s = _rows(k, "out[0]", c.heads, c.head_dim, fp4.DTYPES, dev)
    _need(s == _rows(v, "out[1]", c.heads, c.head_dim, fp4.DTYPES, dev) and k.dtype == v.dtype
          and k.shape == v.shape and k.shape[0] == tokens,
          "the outputs must agree in shape, type and strides")
    _raise(fp4.load().fp4_kv_gather(c, layer, b, k.data_ptr(), v.data_ptr(), s[0], s[1],
                                    fp4.DTYPES[k.dtype], tokens, fp4._stream(stream)),
           "fp4_kv_gather")
    return k, v


def kv_attention_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int, tokens: int,
                                 window: int = 0, sinks: int = 0) -> int:
    """Bytes of the workspace that ``kv_attention`` needs (0: none)."""
    c = _cache(cache)
    b = _batch(batch, cache.k_codes.device)
    return int(fp4.load().fp4_kv_attention_workspace_bytes(c, b, q_heads, tokens, window, sinks))


def kv_attention(q: torch.Tensor, cache: KVCache, batch: KVBatch, layer: int = 0,
                 scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                 out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                 lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Causal attention of the new tokens (q: [tokens, q_heads, head_dim] BF16)
    over the cache, which holds their own keys already.  ``scale``: None is 1 /
    sqrt(head_dim).  ``window`` > 0: a token sees the last ``window`` positions,
    itself included, and the first ``sinks``.  ``lse``: a dense float32 [tokens,
    q_heads] tensor that takes the logarithm of each row's sum of exponentials.
    Rows of no sequence are not written."""
    c = _cache(cache)
    dev = cache.k_codes.device
    b = _batch(batch, dev)
    qs = _rows(q, "q", 0, c.head_dim, (torch.bfloat16,), dev)
    tokens, q_heads = q.shape[0], q.shape[1]
    L = fp4.load()
    with fp4._Alloc(stream) as al:
        if out is None:
            out = al.empty((tokens, q_heads, c.head_dim), out_dtype, dev, "out")
        os_ = _rows(out, "out", q_heads, c.head_dim, fp4.DTYPES, dev)
        _need(out.shape[0] == tokens, "out must have q's shape")
        if lse is not None:
            _need(lse.dtype == torch.float32 and lse.shape == (tokens, q_heads)
                  and lse.is_contiguous() and lse.device == dev,
                  "lse must be a dense float32 [tokens, q_heads] tensor on the cache's device")
        if workspace is None:
            n = L.fp4_kv_attention_workspace_bytes(c, b, q_heads, tokens, window, sinks)
            if n:
                workspace = al.empty(n, torch.uint8, dev, "the workspace")
        st = L.fp4_kv_attention(
            c, layer, b, q.data_ptr(), qs[0], qs[1], q_heads, tokens,
            1.0 / math.sqrt(c.head_dim) if scale is None else scale, window, sinks,
            out.data_ptr(), fp4.DTYPES[out.dtype], os_[0], os_[1], fp4._ptr(lse),
            fp4._ptr(workspace), fp4._nbytes(workspace), fp4._stream(stream))
    _raise(st, "fp4_kv_attention")
    return out


def _tables(table, refs, device, lens=None):
    _ints(table, "page_table", 2, device)
    _ints(refs, "refs", 1, device)
    if lens is not None:
        _ints(lens, "lens", 1, device)
        _need(lens.shape[0] == table.shape[0], "lens must have a length for every sequence")
    ld = table.stride(0) if table.shape[0] > 1 else max(table.shape[1], 1)
    return table.data_ptr(), ld, table.shape[0], table.shape[1]


def kv_copy_pages(cache: KVCache, src: torch.Tensor, dst: torch.Tensor,
                  tokens: Optional[torch.Tensor] = None, stream=None) -> None:
    """Page ``dst[i]`` takes page ``src[i]`` in every layer (its first
    ``tokens[i]`` tokens, if given).  int32 device tensors; pages of ``dst`` are
    distinct and none of ``src``; ids out of range are skipped."""
    c = _cache(cache)
    dev = cache.k_codes.device
    _ints(src, "src", 1, dev)
    _ints(dst, "dst", 1, dev)
    _need(src.shape == dst.shape, "src and dst must be of one length")
    if tokens is not None:
        _ints(tokens, "tokens", 1, dev)
        _need(tokens.shape == src.shape, "tokens must be as long as src")
    _raise(fp4.load().fp4_kv_copy_pages(c, src.data_ptr(), dst.data_ptr(), fp4._ptr(tokens),
                                        src.shape[0], fp4._stream(stream)), "fp4_kv_copy_pages")


def kv_fork(cache: KVCache, page_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
            parents: torch.Tensor, children: torch.Tensor,
            workspace: Optional[torch.Tensor] = None, failed: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """Sequence ``children[i]`` becomes a copy of ``parents[i]``: full pages are
    shared (``refs`` + 1), a partly filled last page is copied into the lowest
    free page.  Returns a one-element int32 device tensor: the forks that found
    no free page (their children are left empty).  Children are distinct, hold
    no pages and are no parents of the same call."""
    c = _cache(cache)
    dev = cache.k_codes.device
    t = _tables(page_table, refs, dev, lens)
    _ints(parents, "parents", 1, dev)
    _ints(children, "children", 1, dev)
    _need(parents.shape == children.shape, "parents and children must be of one length")
    _need(refs.shape[0] == c.pages, "refs must have a count for every page")
    n = parents.shape[0]
    with fp4._Alloc(stream) as al:
        if failed is None:
            failed = al.empty(1, torch.int32, dev, "failed")
        _ints(failed, "failed", 1, dev)
        if workspace is None:
            workspace = al.empty(16 * max(n, 1), torch.uint8, dev, "the workspace")
        st = fp4.load().fp4_kv_fork(c, *t, lens.data_ptr(), refs.data_ptr(), parents.data_ptr(),
                                    children.data_ptr(), n, failed.data_ptr(),
                                    workspace.data_ptr(), fp4._nbytes(workspace),
                                    fp4._stream(stream))
    _raise(st, "fp4_kv_fork")
    return failed


def kv_free(page_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, seqs: torch.Tensor,
            page_size: int, window: int = 0, sinks: int = 0, stream=None) -> None:
    """Give pages of the (distinct) sequences ``seqs`` back: all of them (the
    length becomes 0), or with ``window`` > 0 those that hold none of the last
    ``window`` tokens and none of the first ``sinks``."""
    t = _tables(page_table, refs, page_table.device, lens)
    _ints(seqs, "seqs", 1, page_table.device)
    _raise(fp4.load().fp4_kv_free(*t, lens.data_ptr(), refs.data_ptr(), refs.shape[0], page_size,
                                  seqs.data_ptr(), seqs.shape[0], window, sinks,
                                  fp4._stream(stream)), "fp4_kv_free")


def kv_compact(cache: KVCache, page_table: torch.Tensor, refs: torch.Tensor,
               workspace: Optional[torch.Tensor] = None, place: Optional[torch.Tensor] = None,
               used: Optional[torch.Tensor] = None, stream=None):
    """Pack the pages in use into the lowest ids, with as few moves as that
    takes; ``page_table`` and ``refs`` are rewritten.  Returns (place, used):
    each page's new id (-1: it was free) and, in one element, the number of
    pages in use."""
    c = _cache(cache)
    dev = cache.k_codes.device
    t = _tables(page_table, refs, dev)
    _need(refs.shape[0] == c.pages, "refs must have a count for every page")
    with fp4._Alloc(stream) as al:
        if place is None:
            place = al.empty(c.pages, torch.int32, dev, "place")
        if used is None:
            used = al.empty(1, torch.int32, dev, "used")
        _ints(place, "place", 1, dev)
        _ints(used, "used", 1, dev)
        _need(place.shape[0] == c.pages, "place must have an id for every page")
        if workspace is None:
            workspace = al.empty(4 * (c.pages + 3), torch.uint8, dev, "the workspace")
        st = fp4.load().fp4_kv_compact(c, *t, refs.data_ptr(), place.data_ptr(), used.data_ptr(),
                                       workspace.data_ptr(), fp4._nbytes(workspace),
                                       fp4._stream(stream))
    _raise(st, "fp4_kv_compact")
    return place, used
