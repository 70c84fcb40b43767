"""Per-head norm and rotary position of queries and keys (``include/fa_rotary.h``).

Like the rest of the package these functions only marshal arguments: views are
passed with their strides, outputs and workspaces are allocated with torch, the
arithmetic runs in the CUDA kernels of ``libfa.so``.
"""
from __future__ import annotations

import math
import struct

import torch

from . import FA_OK, FAError, load_library
from ._marshal import (F32, HEADS, NO_HEADS, ROTARY, device_of, four, heads_of, on, out_heads,
                       positions_of, rotary_of, stream_of, workspace_of)

_QK = struct.Struct("@" + 4 * HEADS + "Pqq" + ROTARY + "6i")
_QK_BWD = struct.Struct("@" + 6 * HEADS + "Pqq" + ROTARY + "PP" + "6i")


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0,
                       original_length=None, low=1.0, high=32.0, device="cuda"):
    """Radians per position of the rotary_dim / 2 pairs, fp64 on `device`:
    f_i = base^(-2 i / rotary_dim), stretched for contexts `factor` times longer
    than the trained one by

    * ``None``: not at all;
    * ``"linear"``: every f_i / factor;
    * ``"ntk"``: a larger base, base * factor^(r / (r - 2)), which leaves the
      fastest pair as it is and divides the slowest by factor;
    * ``"ramp"``: pairs that turn at least `high` times over original_length
      stay, those that turn at most `low` times are divided by factor, and those
      between are blended linearly in their number of turns.
    """
    r = int(rotary_dim)
    if r < 0 or r % 16 != 0:
        raise ValueError(f"rotary_dim must be a multiple of 16, got {rotary_dim}")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor > 0):
        raise ValueError("base and factor must be finite and positive")
    if scaling == "ntk" and r > 2:
        base = base * factor ** (r / (r - 2))
    i = torch.arange(0, r, 2, dtype=torch.float64)
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -i / max(r, 1))
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if not original_length or not high > low:
            raise ValueError("ramp scaling needs original_length and high > low")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / factor
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device)


def qk_rotary(q, k, positions, freqs, interleaved=False, rotary_scale=1.0, norm_eps=None,
              q_weight=None, k_weight=None, q_out=None, k_out=None, stream=None, check=True):
    """q_out, k_out = norm (if norm_eps is given) and rotary position of bf16
    CUDA views q [B, H, N, d] and k [B, H_kv, N, d].

    positions: int32 [B, N] or [N]. freqs: fp64 [r / 2] radians per position
    (:func:`rotary_frequencies`), or None to norm only; the first r elements of
    each head are turned, in pairs (i, i + r/2) or, interleaved, (2i, 2i + 1).
    Frequencies must be finite.
    q_weight, k_weight: norm weights [d], both bf16 or both fp32, None for
    ones. Outputs are allocated contiguous unless given; an output may be its
    input.
    """
    dev = device_of(q, "q")
    qs, ks = four(q, "q"), four(k, "k")
    B, H, N, d = qs
    H_kv = ks[1]
    qh, kh = heads_of(q, "q", qs, dev), heads_of(k, "k", (B, H_kv, N, d), dev)
    rot = rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, dev)
    pos = positions_of(positions, B, N, dev)
    with on(dev, stream):
        q_out, oq = out_heads(q_out, "q_out", B, H, N, d, dev)
        k_out, ok = out_heads(k_out, "k_out", B, H_kv, N, d, dev)
        st = load_library().fa_qk_rotary(
            _QK.pack(*qh, *kh, *oq, *ok, *pos, *rot, B, H, H_kv, N, d, 0),
            stream_of(dev, stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_qk_rotary")
    return q_out, k_out


def qk_rotary_bwd(dq_out, dk_out, q, k, positions, freqs, interleaved=False, rotary_scale=1.0,
                  norm_eps=None, q_weight=None, k_weight=None, dq=None, dk=None, workspace=None,
                  stream=None, check=True):
    """dq, dk, dq_weight, dk_weight of a call qk_rotary(q, k, ...) for the
    gradients dq_out, dk_out of its outputs (bf16 views).

    With a norm, q and k are the forward's inputs and the weight gradients are
    fp32 [d], summed over batch, heads and tokens (given for absent weights
    too). Without one, q and k may be None and the weight gradients are None.
    """
    dev = device_of(dq_out, "dq_out")
    qs, ks = four(dq_out, "dq_out"), four(dk_out, "dk_out")
    B, H, N, d = qs
    H_kv = ks[1]
    gq = heads_of(dq_out, "dq_out", qs, dev)
    gk = heads_of(dk_out, "dk_out", (B, H_kv, N, d), dev)
    norm = norm_eps is not None
    if norm:
        if q is None or k is None:
            raise ValueError("the norm's backward needs q and k")
        xq, xk = heads_of(q, "q", qs, dev), heads_of(k, "k", ks, dev)
    else:
        xq = xk = NO_HEADS
    rot = rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, dev)
    pos = positions_of(positions, B, N, dev)
    lib = load_library()
    with on(dev, stream):
        dq, oq = out_heads(dq, "dq", B, H, N, d, dev)
        dk, ok = out_heads(dk, "dk", B, H_kv, N, d, dev)
        dwq = dwk = None
        pwq = pwk = need = 0
        if norm:
            dwq = torch.empty(d, dtype=F32, device=dev)
            dwk = torch.empty(d, dtype=F32, device=dev)
            pwq, pwk = dwq.data_ptr(), dwk.data_ptr()
            need = lib.fa_qk_rotary_bwd_workspace_bytes(B, H, H_kv, N, d, 1)
        ws, ws_bytes, workspace = workspace_of(workspace, need, dev)
        st = lib.fa_qk_rotary_bwd(
            _QK_BWD.pack(*gq, *gk, *xq, *xk, *oq, *ok, *pos, *rot, pwq, pwk,
                         B, H, H_kv, N, d, 0), ws, ws_bytes, stream_of(dev, stream))
    if check and st != FA_OK:
        raise FAError(st, "fa_qk_rotary_bwd")
    return dq, dk, dwq, dwk
