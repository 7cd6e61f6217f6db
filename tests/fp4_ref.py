"""4-bit latent rows in numpy float64, from the format's definition: groups of 16 codes
(e2m1, even channel in a byte's low half) under one e4m3 scale."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)])


def nearest(x, grid):
    """Index of the nearest entry of an ascending grid whose index parity is its last bit; a tie goes to the even one."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def quantize(rows, cache_scale=1.0):
    """(codes, scales) as uint8 arrays of float64 rows [..., d_c]."""
    x = np.asarray(rows, np.float64) / cache_scale
    x = np.where(np.isnan(x), 0.0, x)
    g = x.reshape(*x.shape[:-1], -1, 16)
    s = nearest(np.clip(np.minimum(np.abs(g).max(-1), 2688.0) / 6, E4M3[1], None), E4M3)
    with np.errstate(invalid="ignore"):
        q = np.minimum(np.abs(g), 1e30) / E4M3[s][..., None]
    mag = nearest(np.minimum(q, 6.0), GRID)
    code = np.where((g < 0) & (mag > 0), mag + 8, mag).reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.astype(np.uint8)


def values(codes, scales, cache_scale=1.0):
    """The float64 rows that packed bytes stand for."""
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).astype(int)
    e = np.where(n >= 8, -GRID[n & 7], GRID[n & 7])
    return e * np.repeat(E4M3[scales], 16, axis=-1) * cache_scale
