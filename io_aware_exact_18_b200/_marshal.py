"""What the bindings of ``include/fa_rotary.h`` and ``include/fa_paged.h`` share:
tensors checked and turned into the fields of the C structs, and the device and
stream of a call. A call's cost on the host is a few microseconds, which is what
the smallest calls take on the device, so these helpers do each thing once.
"""
from __future__ import annotations

import torch

# The stream of a device as an integer: the short way where this torch has it
# (60 ns; the public one makes a Stream object, 1.3 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

BF16, F32, F64, I32, U8 = (torch.bfloat16, torch.float32, torch.float64, torch.int32,
                           torch.uint8)
E4M3 = torch.float8_e4m3fn

# fa_heads_t: pointer and three strides; fa_rotary_t: three pointers, four
# int32, two floats (include/fa_rotary.h)
HEADS = "Pqqq"
ROTARY = "PPPiiiiff"
NO_HEADS = (0, 0, 0, 0)


def device_of(t, what, dtype=BF16):
    """The CUDA device that a call's other tensors have to be on."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (no CPU fallback)")
    return t.device


def heads_of(t, what, shape, device):
    """fa_heads_t fields of a bf16 [B, heads, N, d] view of this shape."""
    if t.dtype is not BF16:
        raise TypeError(f"{what} must be bfloat16")
    if t.shape != shape:
        raise ValueError(f"{what}: {list(shape)} expected, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")
    sb, sh, sn, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{what}: the last axis must be contiguous")
    return t.data_ptr(), sb, sh, sn


def out_heads(t, what, B, heads, N, d, device):
    """(tensor, fa_heads_t fields) of a bf16 output: the caller's, or a new one."""
    if t is not None:
        return t, heads_of(t, what, (B, heads, N, d), device)
    t = torch.empty(B, heads, N, d, dtype=BF16, device=device)
    return t, (t.data_ptr(), heads * N * d, N * d, d)


def four(t, what):
    """The shape of a [B, heads, N, d] tensor."""
    s = t.shape
    if len(s) != 4:
        raise ValueError(f"{what}: [B, heads, N, d] expected, got {list(s)}")
    return s


def positions_of(positions, B, N, device):
    """Pointer and strides of int32 positions [B, N] (or [N], repeated)."""
    if positions.dtype is not I32 or positions.device != device:
        raise ValueError(f"positions must be int32 on {device}")
    s = positions.shape
    if s == (B, N):
        sb, sn = positions.stride()
        return positions.data_ptr(), sb, sn
    if s == (N,):
        return positions.data_ptr(), 0, positions.stride(0)
    raise ValueError(f"positions: [{B}, {N}] or [{N}] expected, got {list(s)}")


def rotary_of(freqs, interleaved, rotary_scale, norm_eps, q_weight, k_weight, d, device):
    """fa_rotary_t fields."""
    fp, r = 0, 0
    if freqs is not None:
        if freqs.dtype is not F64 or freqs.device != device or freqs.dim() != 1 or \
                not freqs.is_contiguous():
            raise ValueError(f"freqs must be a contiguous fp64 vector on {device}")
        fp, r = freqs.data_ptr(), 2 * freqs.shape[0]
    if norm_eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("norm weights are given, but no norm_eps")
        return fp, 0, 0, r, 1 if interleaved else 0, 0, 0, rotary_scale, 0.0
    pointers, kind = [0, 0], None
    for i, w in enumerate((q_weight, k_weight)):
        if w is None:
            continue
        if w.device != device or w.shape != (d,) or not w.is_contiguous():
            raise ValueError(f"norm weights must be contiguous [{d}] on {device}")
        if (w.dtype is not BF16 and w.dtype is not F32) or (kind or w.dtype) is not w.dtype:
            raise TypeError("norm weights must be both bfloat16 or both float32")
        kind = w.dtype
        pointers[i] = w.data_ptr()
    return (fp, pointers[0], pointers[1], r, 1 if interleaved else 0, 1,
            1 if kind is F32 else 0, rotary_scale, norm_eps)


def vector_of(t, what, n, device):
    """Pointer of a contiguous int32 vector of n entries."""
    if t.dtype is not I32 or t.device != device or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 vector [{n}] on {device}")
    return t.data_ptr()


def workspace_of(workspace, need, device):
    """(pointer, bytes, tensor) of a call's workspace, allocated if needed."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=U8, device=device)
        return workspace.data_ptr(), need, workspace
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


class _Guard:
    """The tensors' device made current, and, where the caller names a stream,
    torch's allocations made for that stream."""

    def __init__(self, device, stream):
        self.guards = [torch.cuda.device(device)]
        if stream is not None:
            self.guards.append(torch.cuda.stream(
                torch.cuda.ExternalStream(int(stream), device=device)))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


class _Nothing:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_NOTHING = _Nothing()


_current_device = torch.cuda.current_device


def on(device, stream):
    """The context to allocate and launch in."""
    if stream is None and device.index == _current_device():
        return _NOTHING
    return _Guard(device, stream)


def stream_of(device, stream):
    return _raw_stream(device.index) if stream is None else int(stream)
