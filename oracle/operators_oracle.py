"""Float64 oracle of the operators around the layer (numpy, CPU): per-head norms
with the position rotation and their gradients, the paged cache, attention of
new tokens over it.  Written from the formulas; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

D = 64


def rotation_angles(positions, axes, base):
    """Angles [..., 32] of the channel pairs: axes 1: pair i is channels (i, i + 32); axes 2: pairs 0..15 are
    (i, i + 16) by the first coordinate, 16..31 are (32 + i, 48 + i) by the second."""
    p = np.asarray(positions, dtype=np.float64)
    half = 32 // axes
    f = float(base) ** (-np.arange(half) / half)
    return np.concatenate([p[..., a:a + 1] * f for a in range(axes)], axis=-1)


def _pairs(axes):
    if axes == 1:
        return np.arange(32), np.arange(32) + 32
    i = np.concatenate([np.arange(16), 32 + np.arange(16)])
    return i, i + 16


def rotate(x, angles, axes, back=False):
    """x [..., 64] turned by angles [..., 32] (broadcast over the heads by the caller)."""
    a, b = _pairs(axes)
    c, s = np.cos(angles), np.sin(angles) * (-1.0 if back else 1.0)
    y = np.empty(np.broadcast_shapes(x.shape, angles.shape[:-1] + (D,)))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def normed(x, norm, eps):
    """Normalised rows (no weight) and the factor of each row."""
    if norm == "none":
        return x.astype(np.float64), np.ones(x.shape[:-1] + (1,))
    x = x.astype(np.float64)
    if norm == "layer":
        x = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def norm_rope(x, norm, eps, weight=None, bias=None, positions=None, axes=0, base=1.0):
    """x [..., tokens, heads, 64], positions [..., tokens, axes]."""
    y, _ = normed(x, norm, eps)
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    if axes:
        y = rotate(y, rotation_angles(positions, axes, base)[..., None, :], axes)
    return y


def norm_rope_backward(x, dy, norm, eps, weight=None, positions=None, axes=0, base=1.0):
    """dx, dweight, dbias (sums over all rows) of norm_rope; dy like its output."""
    g = np.asarray(dy, dtype=np.float64)
    if axes:
        g = rotate(g, rotation_angles(positions, axes, base)[..., None, :], axes, back=True)
    if norm == "none":
        return g, None, None
    h, r = normed(x, norm, eps)
    lead = tuple(range(g.ndim - 1))
    u = g * weight
    dx = u - h * (u * h).mean(-1, keepdims=True)
    if norm == "layer":
        dx = dx - u.mean(-1, keepdims=True)
    return dx * r, (g * h).sum(lead), g.sum(lead)


def cache_append(pages, rows, table, start, cu):
    """pages [P][heads][page][64] with the sequences' new rows [tokens][heads][64] written; the places that were left out."""
    pages = pages.copy()
    out = []
    n_pages, _, size, _ = pages.shape
    for b in range(len(start)):
        for t in range(cu[b], cu[b + 1]):
            at = start[b] + t - cu[b]
            page = table[b][at // size] if 0 <= at < table.shape[1] * size else -1
            if 0 <= page < n_pages:
                pages[page, :, at % size] = rows[t]
            else:
                out.append((b, t))
    return pages, out


def cache_attention(q, k_pages, v_pages, table, lengths, cu, causal, scale=0.125):
    """out [tokens][heads][64], lse [heads][tokens], and mean |v| under the same weights (the bound of a rounding of the
    weights); rows of no sequence are NaN in all three."""
    n_pages, hk, size, _ = k_pages.shape
    tokens, hq, _ = q.shape
    out, mag = (np.full((tokens, hq, D), np.nan) for _ in range(2))
    lse = np.full((hq, tokens), np.nan)
    for b in range(len(lengths)):
        n = cu[b + 1] - cu[b]
        if n <= 0:
            continue
        length = int(min(lengths[b], table.shape[1] * size))
        slot = np.arange(length)
        page = table[b][slot // size]
        there = (page >= 0) & (page < n_pages)
        page = np.where(there, page, 0)
        limit = lengths[b] - n + 1 + np.arange(n) if causal else np.full(n, length)
        seen = there[None] & (slot[None] < limit[:, None])
        for h in range(hq):
            k = np.where(there[:, None], k_pages[page, h // (hq // hk), slot % size], 0.0)
            v = np.where(there[:, None], v_pages[page, h // (hq // hk), slot % size], 0.0)
            s = np.where(seen, (q[cu[b]:cu[b + 1], h] @ k.T) * scale, -np.inf)
            top = s.max(-1, keepdims=True) if length else np.full((n, 1), -np.inf)
            p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
            w = p.sum(-1, keepdims=True)
            safe = np.where(w > 0, w, 1.0)
            out[cu[b]:cu[b + 1], h] = (p @ v) / safe
            mag[cu[b]:cu[b + 1], h] = (p @ np.abs(v)) / safe
            with np.errstate(divide="ignore"):
                lse[h, cu[b]:cu[b + 1]] = (top + np.log(w))[:, 0]
    return out, lse, mag
