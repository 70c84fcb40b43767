"""A key/value cache in pages (``include/fa_paged.h``): append, one-token
attention, page copies. Argument marshalling only, as in the rest of the
package; the arithmetic runs in the CUDA kernels of ``libfa.so``.

K and V pages are views ``[pages, H_kv, page_size, d]`` of bf16 or e4m3
(torch.float8_e4m3fn) tensors with equal strides: contiguous, or a transposed
``[pages, page_size, H_kv, d]`` tensor, or slices of one that holds both.
``block_table`` is int32 ``[sequences, pages per sequence]``.
"""
from __future__ import annotations

import math
import struct

from .rotary import (HEADS, NO_HEADS, ROTARY, _failed, heads_of, on_device, positions_of,
                     rotary_of)

# fa_paged_cache_t: two pointers, three strides, five int32, two floats, int32;
# fa_block_table_t: pointer, stride, two int32 (include/fa_paged.h)
CACHE = "PPqqqiiiiiffi"
TABLE = "Pqii"
_APPEND = struct.Struct("@" + CACHE + TABLE + 4 * HEADS + "Pqq" + "P" + ROTARY + "4i")
_DECODE = struct.Struct("@" + CACHE + TABLE + "PqqPPP" + "iifi")
_COPY = struct.Struct("@" + CACHE)


def cache_of(k_cache, v_cache, k_descale, v_descale):
    """fa_paged_cache_t fields of the two page tensors."""
    import torch
    dt = k_cache.dtype
    if dt == torch.bfloat16:
        elem = 2
    elif dt == torch.float8_e4m3fn:
        elem = 1
    else:
        raise TypeError("cache pages must be bfloat16 or float8_e4m3fn")
    if v_cache.dtype != dt:
        raise TypeError("K and V pages must have one type")
    if not k_cache.is_cuda or v_cache.device != k_cache.device:
        raise ValueError("K and V pages must be on one CUDA device (no CPU fallback)")
    s = k_cache.shape
    st = k_cache.stride()
    if len(s) != 4 or v_cache.shape != s or v_cache.stride() != st or st[3] != 1:
        raise ValueError("K and V pages: [pages, H_kv, page_size, d] views with equal strides "
                         f"and a contiguous last axis expected, got {tuple(s)} {st} and "
                         f"{tuple(v_cache.shape)} {v_cache.stride()}")
    return (k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], s[0], s[2], s[1], s[3],
            elem, float(k_descale), float(v_descale), 0)


def table_of(block_table, device):
    """fa_block_table_t fields."""
    import torch
    if block_table.dtype != torch.int32 or block_table.device != device or \
            block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [sequences, pages] on the cache's device, "
                         "rows contiguous")
    return (block_table.data_ptr(), block_table.stride(0), block_table.shape[0],
            block_table.shape[1])


def _int32_vector(t, what, n, device):
    import torch
    if t.dtype != torch.int32 or t.device != device or t.dim() != 1 or \
            (n is not None and t.shape[0] != n) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 vector"
                         f"{'' if n is None else f' [{n}]'} on the cache's device")
    return t.data_ptr()


def paged_append(k, v, k_cache, v_cache, block_table, positions, q=None, freqs=None,
                 interleaved=False, rotary_scale=1.0, norm_eps=None, q_weight=None,
                 k_weight=None, k_descale=1.0, v_descale=1.0, seq=None, q_out=None, stream=None,
                 check=True):
    """Write new tokens' keys and values, bf16 views k, v [B, H_kv, N, d], into
    the cache and return the queries for them.

    Token (b, n) goes to key positions[b, n] (int32 [B, N] or [N]) of sequence
    seq[b] (int32 [B]; default b). Keys are normed and turned first as in
    :func:`qk_rotary` (norm_eps, k_weight, freqs; both None: stored as they
    come), and so is q [B, H, N, d] if given, into q_out (allocated unless
    given; may be q). e4m3 pages hold value / descale, saturated. Tokens with a
    negative position are padding: nothing of them is written. Tokens whose
    page the table does not give are dropped from the cache.
    """
    import torch
    from . import FA_OK, load_library
    cache = cache_of(k_cache, v_cache, k_descale, v_descale)
    dev, H_kv, d = k_cache.device, cache[7], cache[8]
    B, N = k.shape[0], k.shape[-2]
    kh, vh = heads_of(k, "k", B, H_kv, N, d), heads_of(v, "v", B, H_kv, N, d)
    qh, H = NO_HEADS, 0
    if q is not None:
        qh, H = heads_of(q, "q", B, None, N, d), q.shape[1]
    for t in (k, v, q, q_out):
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on the cache's device")
    table = table_of(block_table, dev)
    pos = positions_of(positions, B, N, dev)
    sp = 0 if seq is None else _int32_vector(seq, "seq", B, dev)
    rot = rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, dev)
    with on_device(dev, stream) as s:
        oh = NO_HEADS
        if q is not None:
            if q_out is None:
                q_out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev)
            oh = heads_of(q_out, "q_out", B, H, N, d)
        st = load_library().fa_paged_append(
            _APPEND.pack(*cache, *table, *kh, *vh, *qh, *oh, *pos, sp, *rot, B, H, N, 0), s)
    if check and st != FA_OK:
        _failed(st, "fa_paged_append")
    return q_out


def paged_decode_attention(q, k_cache, v_cache, block_table, kv_len, scale=None, k_descale=1.0,
                           v_descale=1.0, out=None, lse=None, workspace=None, stream=None,
                           check=True):
    """O [B, H, 1, d] (bf16) and lse [B, H, 1] (fp32) of one query row per head,
    q [B, H, 1, d], against the first kv_len[b] (int32 [B]) keys of the pages
    that block_table row b lists: :func:`decode_attention` over a paged cache.
    A sequence without keys gets O = 0 and lse = -inf. The workspace is
    allocated with torch unless given as a CUDA uint8 tensor of at least
    fa_paged_decode_workspace_bytes(B, H, H_kv, d) bytes.
    """
    import torch
    from . import FA_OK, load_library
    cache = cache_of(k_cache, v_cache, k_descale, v_descale)
    dev, d = k_cache.device, cache[8]
    qh = heads_of(q, "q", q.shape[0], None, 1, d)
    B, H = q.shape[0], q.shape[1]
    for t in (q, out, lse, workspace):
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on the cache's device")
    table = table_of(block_table, dev)
    lens = _int32_vector(kv_len, "kv_len", B, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    lib = load_library()
    with on_device(dev, stream) as s:
        if out is None:
            out = torch.empty((B, H, 1, d), dtype=torch.bfloat16, device=dev)
        elif out.dtype != torch.bfloat16 or tuple(out.shape) != (B, H, 1, d) or \
                not out.is_contiguous():
            raise ValueError(f"out must be a contiguous bfloat16 [{B}, {H}, 1, {d}]")
        if lse is None:
            lse = torch.empty((B, H, 1), dtype=torch.float32, device=dev)
        elif lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, 1) or \
                not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 [{B}, {H}, 1]")
        need = lib.fa_paged_decode_workspace_bytes(B, H, cache[7], d)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws, ws_bytes = (None, 0) if workspace is None else \
            (workspace.data_ptr(), workspace.numel() * workspace.element_size())
        st = lib.fa_paged_decode(
            _DECODE.pack(*cache, *table, qh[0], qh[1], qh[2], out.data_ptr(), lse.data_ptr(),
                         lens, B, H, float(scale), 0), ws, ws_bytes, s)
    if check and st != FA_OK:
        _failed(st, "fa_paged_decode")
    return out, lse


def copy_pages(k_cache, v_cache, src, dst, stream=None, check=True):
    """Copy pages src[i] to dst[i] (int32 vectors) of both caches, for
    copy-on-write forks and for compaction. Pages may be read several times; no
    dst may appear twice or among src (src[i] == dst[i] changes nothing). Pairs
    with a page outside the cache are skipped."""
    from . import FA_OK, load_library
    cache = cache_of(k_cache, v_cache, 1.0, 1.0)
    dev = k_cache.device
    sp = _int32_vector(src, "src", None, dev)
    n = src.shape[0]
    dp = _int32_vector(dst, "dst", n, dev)
    with on_device(dev, stream) as s:
        st = load_library().fa_copy_pages(_COPY.pack(*cache), sp, dp, n, s)
    if check and st != FA_OK:
        _failed(st, "fa_copy_pages")
