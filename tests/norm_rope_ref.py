"""Plain fp64 norms with rotary positions and their gradient (numpy): what the tests of attn_norm_rope go by."""
import numpy as np


def rotate(x, positions, freqs, axes, pairing, sign=1.0):
    """x [..., tokens, heads, d] rotated; positions [axes, ..., tokens].  With it the sum of the magnitudes of the two
    terms of each element (one term where it does not turn)."""
    y, mag = x.copy(), np.abs(x)
    n = len(freqs)
    for p in range(n):
        i, j = (2 * p, 2 * p + 1) if pairing == "adjacent" else (p, p + n)
        angle = np.asarray(positions[axes[p]], dtype=np.longdouble) * np.longdouble(freqs[p])
        c, s = np.cos(angle).astype(np.float64)[..., None], sign * np.sin(angle).astype(np.float64)[..., None]
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., j] * c + x[..., i] * s
        mag[..., i] = mag[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, mag


def size(x, eps):
    return np.sqrt((x * x).sum(-1, keepdims=True) / x.shape[-1] + eps)


def forward(x, w, eps, positions, freqs, axes, pairing):
    """y and the magnitudes behind each of its elements; x [..., tokens, heads, d], w [d] or None."""
    n = x / size(x, eps)
    return rotate(n if w is None else n * w, positions, freqs, axes, pairing)


def backward(dy, x, w, eps, positions, freqs, axes, pairing):
    """dx and dw, and the magnitudes of the terms that each is a sum of."""
    n = x / size(x, eps)
    w = np.ones(x.shape[-1]) if w is None else w
    g, mag = rotate(dy, positions, freqs, axes, pairing, -1.0)
    d = x.shape[-1]
    dot = (g * w * n).sum(-1, keepdims=True) / d
    dx = (g * w - n * dot) / size(x, eps)
    dx_mag = (mag * np.abs(w) + np.abs(n) * (mag * np.abs(w * n)).sum(-1, keepdims=True) / d) / size(x, eps)
    lead = tuple(range(x.ndim - 1))
    return dx, dx_mag, (g * n).sum(lead), (mag * np.abs(n)).sum(lead)
