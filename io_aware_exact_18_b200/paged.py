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

import torch

from . import FA_OK, FAError, load_library
from ._marshal import (BF16, E4M3, F32, HEADS, I32, NO_HEADS, ROTARY, four, heads_of, on,
                       out_heads, positions_of, rotary_of, stream_of, vector_of, workspace_of)

# fa_paged_cache_t: two pointers, three strides, five int32, two floats, int32;
# fa_block_table_t: pointer, stride, two int32 (include/fa_paged.h)
CACHE = "PPqqqiiiiiffi"
TABLE = "Pqii"
_APPEND = struct.Struct("@" + CACHE + TABLE + 4 * HEADS + "Pqq" + "P" + ROTARY + "4i")
_DECODE = struct.Struct("@" + CACHE + TABLE + "PqqPPP" + "iifi")
_COPY = struct.Struct("@" + CACHE)


def cache_of(k_cache, v_cache, k_descale, v_descale):
    """fa_paged_cache_t fields of the two page tensors."""
    dt = k_cache.dtype
    if dt is BF16:
        elem = 2
    elif dt is E4M3:
        elem = 1
    else:
        raise TypeError("cache pages must be bfloat16 or float8_e4m3fn")
    if v_cache.dtype is not dt:
        raise TypeError("K and V pages must have one type")
    if not k_cache.is_cuda or v_cache.device != k_cache.device:
        raise ValueError("K and V pages must be on one CUDA device (no CPU fallback)")
    s = k_cache.shape
    st = k_cache.stride()
    if len(s) != 4 or v_cache.shape != s or v_cache.stride() != st or st[3] != 1:
        raise ValueError("K and V pages: [pages, H_kv, page_size, d] views with equal strides "
                         f"and a contiguous last axis expected, got {list(s)} {st} and "
                         f"{list(v_cache.shape)} {v_cache.stride()}")
    return (k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], s[0], s[2], s[1], s[3],
            elem, k_descale, v_descale, 0)


def table_of(block_table, device):
    """fa_block_table_t fields."""
    s = block_table.shape
    if block_table.dtype is not I32 or block_table.device != device or len(s) != 2 or \
            (s[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table must be int32 [sequences, pages] on {device}, "
                         "rows contiguous")
    return block_table.data_ptr(), block_table.stride(0), s[0], s[1]


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
    given; may be q). e4m3 pages hold value / descale, saturated (descales above
    2^-128). K and V pages must share no element. Tokens with a
    negative position are padding: nothing of them is written, and an allocated
    q_out holds arbitrary values in their rows. Tokens whose page the table does
    not give are dropped from the cache. Two tokens of a call must not go to the
    same slot.
    """
    cache = cache_of(k_cache, v_cache, k_descale, v_descale)
    dev, H_kv, d = k_cache.device, cache[7], cache[8]
    B, _, N, _ = four(k, "k")
    ks = (B, H_kv, N, d)
    kh, vh = heads_of(k, "k", ks, dev), heads_of(v, "v", ks, dev)
    table = table_of(block_table, dev)
    pos = positions_of(positions, B, N, dev)
    sp = 0 if seq is None else vector_of(seq, "seq", B, dev)
    rot = rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, dev)
    qh = oh = NO_HEADS
    H = 0
    with on(dev, stream):
        if q is not None:
            H = four(q, "q")[1]
            qh = heads_of(q, "q", (B, H, N, d), dev)
            q_out, oh = out_heads(q_out, "q_out", B, H, N, d, dev)
        elif q_out is not None:
            raise ValueError("q_out is given, but no q")
        st = load_library().fa_paged_append(
            _APPEND.pack(*cache, *table, *kh, *vh, *qh, *oh, *pos, sp, *rot, B, H, N, 0),
            stream_of(dev, stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_paged_append")
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
    cache = cache_of(k_cache, v_cache, k_descale, v_descale)
    dev, d = k_cache.device, cache[8]
    B, H, _, _ = four(q, "q")
    qs = (B, H, 1, d)
    qp, qsb, qsh, _ = heads_of(q, "q", qs, dev)
    table = table_of(block_table, dev)
    lens = vector_of(kv_len, "kv_len", B, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    lib = load_library()
    with on(dev, stream):
        if out is None:
            out = torch.empty(B, H, 1, d, dtype=BF16, device=dev)
        elif out.dtype is not BF16 or out.shape != qs or out.device != dev or \
                not out.is_contiguous():
            raise ValueError(f"out must be a contiguous bfloat16 {list(qs)} on {dev}")
        if lse is None:
            lse = torch.empty(B, H, 1, dtype=F32, device=dev)
        elif lse.dtype is not F32 or lse.shape != qs[:3] or lse.device != dev or \
                not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 {list(qs[:3])} on {dev}")
        ws, ws_bytes, workspace = workspace_of(
            workspace, lib.fa_paged_decode_workspace_bytes(B, H, cache[7], d), dev)
        st = lib.fa_paged_decode(
            _DECODE.pack(*cache, *table, qp, qsb, qsh, out.data_ptr(), lse.data_ptr(), lens, B, H,
                         scale, 0), ws, ws_bytes, stream_of(dev, stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_paged_decode")
    return out, lse


def copy_pages(k_cache, v_cache, src, dst, stream=None, check=True):
    """Copy pages src[i] to dst[i] (int32 vectors) of both caches, for
    copy-on-write forks and for compaction. Pages may be read several times; no
    dst may appear twice or among src (src[i] == dst[i] changes nothing). Pairs
    with a page outside the cache are skipped."""
    cache = cache_of(k_cache, v_cache, 1.0, 1.0)
    dev = k_cache.device
    n = src.numel()
    sp, dp = vector_of(src, "src", n, dev), vector_of(dst, "dst", n, dev)
    with on(dev, stream):
        st = load_library().fa_copy_pages(_COPY.pack(*cache), sp, dp, n, stream_of(dev, stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_copy_pages")
