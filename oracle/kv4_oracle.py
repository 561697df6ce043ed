"""Plain fp64 oracle of the paged 4-bit key/value cache: quantization to E2M1 codes with
E4M3 scales, page sums, page selection, attention. Shares no code with the library."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the 127 finite non-negative E4M3 values, ascending (code = index)
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def _nearest(x, grid):
    """Index of the nearest grid value, of two equally near ones the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    a, b = x - grid[hi - 1], grid[hi] - x
    lower = (a < b) | ((a == b) & ((hi - 1) % 2 == 0))
    return np.where(lower, hi - 1, hi)


def quantize(x, head_scale=None):
    """x [..., H, d] fp32 -> (codes [..., H, d] 0..15, scale codes [..., H, d/16])."""
    x = np.asarray(x, dtype=np.float32)
    if head_scale is not None:
        x = x / np.asarray(head_scale, dtype=np.float32)[:, None]      # one fp32 rounding
    g = x.astype(np.float64).reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s = _nearest(np.minimum(np.abs(g).max(-1) / 6, 448.0), E4M3)
    v = E4M3[s][..., None]
    c = np.where(v > 0, _nearest(np.abs(g) / np.where(v > 0, v, 1.0), E2M1), 0)
    c = c + 8 * ((g < 0) & (v > 0))
    return c.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def dequantize(codes, scales):
    """The stored values without the head's scale, fp64."""
    mag = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return mag * np.repeat(E4M3[scales], 16, axis=-1)


def page_sum(values):
    """values [block, d] -> the sum over the page in units of 2^-10 (whole numbers)."""
    return np.rint(values.sum(0) * 1024).astype(np.int64)


def select_row(q, ksums, block, scale, p, k_min):
    """q [G, d] of one row and KV head, ksums [o, d] of the pages before its own (with the head's scale) ->
    ascending list, the own page o last."""
    o = len(ksums)
    if o == 0:
        return [0]
    s = (q.astype(np.float64) @ ksums.astype(np.float64).T) * (scale / (1024.0 * block))
    e = np.exp(s - s.max(-1, keepdims=True))
    mass = (e / e.sum(-1, keepdims=True)).mean(0)
    order = np.argsort(-mass, kind="stable")
    n = o
    if p < 1:
        reach = np.nonzero(np.cumsum(mass[order]) >= p)[0]
        n = int(reach[0]) + 1 if len(reach) else o
    cnt = min(o, max(n, k_min))
    return sorted(int(j) for j in order[:cnt]) + [o]


def attend_row(q, k, v, scale):
    """q [d], k, v [n, d] (the tokens the row sees) -> (out [d], lse, sum of the weights times |v| [d],
    largest sum of |q||k| scale)."""
    if len(k) == 0:
        z = np.zeros(q.shape[-1])
        return z, -np.inf, z, 0.0
    q = q.astype(np.float64)
    s = (k @ q) * scale
    m = s.max()
    e = np.exp(s - m)
    w = e / e.sum()
    return w @ v, m + np.log(e.sum()), w @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * scale)
