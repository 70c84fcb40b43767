"""Per-head norm and rotary position of queries and keys (``include/fa_rotary.h``).

Like the rest of the package these functions only marshal arguments: views are
passed with their strides, outputs and workspaces are allocated with torch, the
arithmetic runs in the CUDA kernels of ``libfa.so``.
"""
from __future__ import annotations

import math
import struct

# fa_heads_t: pointer and three strides; fa_rotary_t: three pointers, four
# int32, two floats (include/fa_rotary.h)
HEADS = "Pqqq"
ROTARY = "PPPiiiiff"
_QK = struct.Struct("@" + 4 * HEADS + "Pqq" + ROTARY + "6i")
_QK_BWD = struct.Struct("@" + 6 * HEADS + "Pqq" + ROTARY + "PP" + "6i")
NO_HEADS = (0, 0, 0, 0)


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
    import torch
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


def heads_of(t, what, B=None, heads=None, N=None, d=None):
    """fa_heads_t fields of a bf16 CUDA [B, heads, N, d] view (any strides but
    a contiguous last axis), its sizes checked where given."""
    import torch
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what} must be bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (no CPU fallback)")
    s = t.shape
    if len(s) != 4 or (B is not None and (s[0] != B or s[2] != N or s[3] != d)) or \
            (heads is not None and s[1] != heads):
        want = [B, heads, N, d] if B is not None else "[B, heads, N, d]"
        raise ValueError(f"{what}: {want} expected, got {tuple(s)}")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{what}: the last axis must be contiguous")
    return t.data_ptr(), st[0], st[1], st[2]


def positions_of(positions, B, N, device):
    """Pointer and strides of int32 CUDA positions [B, N] (or [N], repeated)."""
    import torch
    if positions.dtype != torch.int32 or positions.device != device:
        raise ValueError("positions must be int32 on the device of q and k")
    if positions.dim() == 1 and positions.shape[0] == N:
        return positions.data_ptr(), 0, positions.stride(0)
    if tuple(positions.shape) != (B, N):
        raise ValueError(f"positions: [{B}, {N}] or [{N}] expected, got "
                         f"{tuple(positions.shape)}")
    st = positions.stride()
    return positions.data_ptr(), st[0], st[1]


def rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, device):
    """fa_rotary_t fields."""
    import torch
    fp, r = 0, 0
    if freqs is not None:
        if freqs.dtype != torch.float64 or freqs.device != device or freqs.dim() != 1 or \
                not freqs.is_contiguous():
            raise ValueError("freqs must be a contiguous fp64 vector on the device of q and k")
        fp, r = freqs.data_ptr(), 2 * freqs.shape[0]
    qw = kw = w32 = 0
    if q_weight is not None or k_weight is not None:
        if norm_eps is None:
            raise ValueError("norm weights are given, but no norm_eps")
        kinds = set()
        for w in (q_weight, k_weight):
            if w is None:
                continue
            if w.device != device or tuple(w.shape) != (d,) or not w.is_contiguous():
                raise ValueError(f"norm weights must be contiguous [{d}] on the device of q and k")
            kinds.add(w.dtype)
        if kinds == {torch.float32}:
            w32 = 1
        elif kinds != {torch.bfloat16}:
            raise TypeError("norm weights must be both bfloat16 or both float32")
        qw = 0 if q_weight is None else q_weight.data_ptr()
        kw = 0 if k_weight is None else k_weight.data_ptr()
    return (fp, qw, kw, r, int(bool(interleaved)), int(norm_eps is not None), w32,
            float(rotary_scale), 0.0 if norm_eps is None else float(norm_eps))


class on_device:
    """The context of a call: the tensors' device made current, and, where the
    caller names a stream, torch's allocations made for that stream."""

    def __init__(self, device, stream):
        import torch
        self.guards = []
        if device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(device))
        if stream is not None:
            self.guards.append(torch.cuda.stream(
                torch.cuda.ExternalStream(int(stream), device=device)))
        self.device, self.stream = device, stream

    def __enter__(self):
        import torch
        for g in self.guards:
            g.__enter__()
        return self.stream if self.stream is not None else \
            torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _failed(status, what):
    from . import FAError
    raise FAError(status, what)


def qk_rotary(q, k, positions, freqs, interleaved=False, rotary_scale=1.0, norm_eps=None,
              q_weight=None, k_weight=None, q_out=None, k_out=None, stream=None, check=True):
    """q_out, k_out = norm (if norm_eps is given) and rotary position of bf16
    CUDA views q [B, H, N, d] and k [B, H_kv, N, d].

    positions: int32 [B, N] or [N]. freqs: fp64 [r / 2] radians per position
    (:func:`rotary_frequencies`), or None to norm only; the first r elements of
    each head are turned, in pairs (i, i + r/2) or, interleaved, (2i, 2i + 1).
    q_weight, k_weight: norm weights [d], both bf16 or both fp32, None for
    ones. Outputs are allocated contiguous unless given; an output may be its
    input.
    """
    import torch
    from . import FA_OK, load_library
    qh = heads_of(q, "q")
    B, H, N, d = q.shape
    kh = heads_of(k, "k", B, None, N, d)
    if k.device != q.device:
        raise ValueError("q and k must be on one device")
    rot = rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, q.device)
    pos = positions_of(positions, B, N, q.device)
    with on_device(q.device, stream) as s:
        if q_out is None:
            q_out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q.device)
        if k_out is None:
            k_out = torch.empty((B, k.shape[1], N, d), dtype=torch.bfloat16, device=q.device)
        st = load_library().fa_qk_rotary(
            _QK.pack(*qh, *kh, *heads_of(q_out, "q_out", B, H, N, d),
                     *heads_of(k_out, "k_out", B, k.shape[1], N, d), *pos, *rot,
                     B, H, k.shape[1], N, d, 0), s)
    if check and st != FA_OK:
        _failed(st, "fa_qk_rotary")
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
    import torch
    from . import FA_OK, load_library
    gq = heads_of(dq_out, "dq_out")
    B, H, N, d = dq_out.shape
    gk = heads_of(dk_out, "dk_out", B, None, N, d)
    H_kv, dev = dk_out.shape[1], dq_out.device
    norm = norm_eps is not None
    if norm:
        if q is None or k is None:
            raise ValueError("the norm's backward needs q and k")
        xq, xk = heads_of(q, "q", B, H, N, d), heads_of(k, "k", B, H_kv, N, d)
    else:
        xq = xk = NO_HEADS
    for t in (dk_out, q, k):
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on one device")
    rot = rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, dev)
    pos = positions_of(positions, B, N, dev)
    lib = load_library()
    with on_device(dev, stream) as s:
        if dq is None:
            dq = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev)
        if dk is None:
            dk = torch.empty((B, H_kv, N, d), dtype=torch.bfloat16, device=dev)
        dw, wp, ws_bytes = (None, None), (0, 0), 0
        if norm:
            both = torch.empty((2, d), dtype=torch.float32, device=dev)
            dw = (both[0], both[1])
            wp = (dw[0].data_ptr(), dw[1].data_ptr())
            need = lib.fa_qk_rotary_bwd_workspace_bytes(B, H, H_kv, N, d, 1)
            if workspace is None and need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if workspace is not None:
            ws_bytes = workspace.numel() * workspace.element_size()
        st = lib.fa_qk_rotary_bwd(
            _QK_BWD.pack(*gq, *gk, *xq, *xk, *heads_of(dq, "dq", B, H, N, d),
                         *heads_of(dk, "dk", B, H_kv, N, d), *pos, *rot, *wp,
                         B, H, H_kv, N, d, 0),
            None if workspace is None else workspace.data_ptr(), ws_bytes, s)
    if check and st != FA_OK:
        _failed(st, "fa_qk_rotary_bwd")
    return dq, dk, dw[0], dw[1]
