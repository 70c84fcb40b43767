"""Per-head norm and rotary position in fp64 numpy, from the definition: the
oracle of fa_qk_rotary, its backward and the append's keys. No code is shared
with the library."""
import numpy as np


def turn(y, positions, freqs, interleaved, scale=1.0, inverse=False):
    """y [B, heads, N, d] with each pair turned by position * frequency."""
    y = np.asarray(y, dtype=np.float64)
    out = y.copy()
    half = len(freqs)
    angle = np.asarray(positions, dtype=np.float64)[:, None, :, None] * \
        np.asarray(freqs, dtype=np.float64)
    c, s = scale * np.cos(angle), scale * np.sin(angle) * (-1.0 if inverse else 1.0)
    if interleaved:
        a, b = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        a, b = slice(0, half), slice(half, 2 * half)
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def norm(x, eps, w=None):
    """x / sqrt(mean x^2 + eps) * w over the last axis (eps None: x)."""
    x = np.asarray(x, dtype=np.float64)
    if eps is None:
        return x
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * np.asarray(w, dtype=np.float64)


def forward(x, positions, freqs, interleaved, scale=1.0, eps=None, w=None):
    return turn(norm(x, eps, w), positions, freqs, interleaved, scale)


def backward(dy, x, positions, freqs, interleaved, scale=1.0, eps=None, w=None):
    """(dx, dw): the gradient of sum(dy * forward(x)); dw None without a norm."""
    g = turn(dy, positions, freqs, interleaved, scale, inverse=True)
    if eps is None:
        return g, None
    x = np.asarray(x, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dw = (g * n).reshape(-1, x.shape[-1]).sum(0)
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdims=True)), dw
