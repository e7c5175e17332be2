"""Plain definitions, in numpy and 64 bits, of the operators between the
projections, the cache and the next token: head norm with rotation, sampling,
attention behind a shared prefix."""
import numpy as np

from cache_ref import e4m3_value


def rope(x, w, eps, positions, axis, inv_freq, interleaved):
    """(z, |a| + |b| of each element's pair, largest angle) of x [M, H, D]."""
    M, H, D = x.shape
    half = len(inv_freq)
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((x * x).mean(2, keepdims=True) + eps) * w
    positions = np.asarray(positions, np.int64).reshape(-1, M)
    z, size, far = y.copy(), np.abs(y), 0.0
    for i in range(half):
        ax = 0 if axis is None else int(axis[i])
        # (extended precision, so that the reference's own angle is not the limit)
        t = (positions[ax].astype(np.longdouble) if ax < len(positions) else np.zeros(M, np.longdouble)) * np.longdouble(inv_freq[i])
        far = max(far, float(np.abs(t).max()) if M else 0.0)
        c, s = (f(t).astype(np.float64)[:, None] for f in (np.cos, np.sin))
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        z[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        z[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
        size[:, :, a] = size[:, :, b] = np.abs(y[:, :, a]) + np.abs(y[:, :, b])
    return z, size, far
