"""Plain fp64 CPU forms of the query/key preparation and the cache writes.

TEST INFRASTRUCTURE ONLY, like ``flex_oracle``: written from the formulas
(root-mean-square norm per head, rotation in pairs by pos * inv_freq, e4m3
rounding under a power-of-two scale per block of slots and head), one row or
one block at a time, and sharing nothing with the CUDA library.
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def pairs(rot, interleaved):
    """Index arrays (a, b) of the rotated pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, pos, inv_freq, interleaved, sign=1.0):
    """x (H, N, D) of one sequence turned by sign * pos * inv_freq."""
    y = np.array(x, np.float64)
    f = np.asarray(inv_freq, np.float64)
    a, b = pairs(2 * f.size, interleaved)
    t = sign * np.asarray(pos, np.float64)[:, None] * f[None, :]
    c, s = np.cos(t), np.sin(t)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, pos=None, inv_freq=None, interleaved=False, norm=False, weight=None, eps=1e-6):
    """Rows x (B, H, N, D); pos (B or 1, N)."""
    x = np.asarray(x, np.float64)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * np.asarray(weight, np.float64)
    if inv_freq is None:
        return x
    pos = np.asarray(pos)
    return np.stack([rotate(x[b], pos[b if pos.shape[0] > 1 else 0], inv_freq, interleaved) for b in range(x.shape[0])])


def norm_rope_backward(x, dy, pos=None, inv_freq=None, interleaved=False, norm=False, weight=None, eps=1e-6):
    """(dx, dweight) of sum(norm_rope(x) * dy)."""
    g = np.asarray(dy, np.float64)
    if inv_freq is not None:
        pos = np.asarray(pos)
        g = np.stack([rotate(g[b], pos[b if pos.shape[0] > 1 else 0], inv_freq, interleaved, -1.0)
                      for b in range(g.shape[0])])
    if not norm:
        return g, None
    x = np.asarray(x, np.float64)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1, 2))
    dx = r * (g * w - x * r ** 2 * (g * w * x).mean(-1, keepdims=True))
    return dx, dw


def e4m3_round(x):
    """Nearest e4m3 value, ties to even, magnitudes above 448 to 448."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    _, e = np.frexp(np.maximum(a, 2.0 ** -60))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.sign(x) * np.minimum(np.rint(a / step) * step, E4M3_MAX)


def e4m3_step(x):
    """Distance between neighbouring e4m3 values at |x|."""
    _, e = np.frexp(np.maximum(np.abs(np.asarray(x, np.float64)), 2.0 ** -60))
    return np.ldexp(1.0, np.maximum(e - 1, -6) - 3)


def block_scale(amax):
    """2^ceil(log2(amax / 448)), 2^-126 at least; 0 for 0."""
    if amax == 0:
        return 0.0
    m, e = np.frexp(amax / E4M3_MAX)
    return float(np.ldexp(1.0, max(int(e) - (1 if m == 0.5 else 0), -126)))


def append(rows, pool, scale, block, table, page, start, count):
    """One sequence's rows (H, N, D) into ``pool`` (outer, H, page, D; values,
    or e4m3 codes when ``scale`` is given) in place; ``table`` lists its pages.
    Returns the unrounded quotients of the new slots: {slot: (H, D)}."""
    wrote = {}
    if scale is None:
        for n in range(count):
            j = start + n
            pool[table[j // page], :, j % page] = rows[:, n]
        return wrote
    H = rows.shape[0]
    for blk in range(start // block, (start + count - 1) // block + 1 if count else start // block):
        lo, hi = max(blk * block, start), min((blk + 1) * block, start + count)
        outer, at = table[blk * block // page], blk * block % page
        for h in range(H):
            new = rows[h, lo - start:hi - start]
            fin = np.abs(new[np.isfinite(new)])
            s = block_scale(fin.max() if fin.size else 0.0)
            if blk * block < start:
                old = float(scale[outer, h, at // block])
                if s > old:
                    k = lo - blk * block
                    pool[outer, h, at:at + k] = e4m3_round(pool[outer, h, at:at + k] * (old / s))
                s = max(s, old)
            scale[outer, h, at // block] = s
            for j in range(lo, hi):
                q = rows[h, j - start] / s if s > 0 else np.zeros_like(rows[h, j - start])
                wrote.setdefault(j, np.zeros((H, q.size)))[h] = q
                pool[outer, h, j % page] = e4m3_round(q)
    return wrote
