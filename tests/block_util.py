"""64-bit definitions of the block formats, for the tests of the few-token
products and of the quantized cache (numpy, written apart from the library)."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)])
E4M3[127] = np.nan
E4M3 = np.concatenate([E4M3, -E4M3])
BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}


def values(q, s, fmt, gs=1.0):
    """Element and scale bytes [..., bytes], [..., blocks] -> float64 [..., K]."""
    q, s = np.asarray(q, np.uint8), np.asarray(s, np.uint8)
    if fmt == "mxfp8":
        v = E4M3[q]
    else:
        v = E2M1[np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)]
    scale = E4M3[s] * float(gs) if fmt == "nvfp4" else np.exp2(s.astype(np.float64) - 127)
    return v * np.repeat(scale, BLOCK[fmt], axis=-1)


def to_mxfp8(x):
    """float64 [..., K] -> (E4M3 bytes, E8M0 codes) by search: the smallest code at
    which the block does not saturate, then the nearest element, ties to even."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    codes = np.arange(255)
    code = np.searchsorted(448.0 * np.exp2(codes - 127.0), top)  # the first with top <= 448 * scale
    v = np.abs(b) / np.exp2(code - 127.0)[..., None]
    grid = E4M3[:127]
    hi = np.clip(np.searchsorted(grid, v), 1, 126)
    lo = hi - 1
    d = (v - grid[lo]) - (grid[hi] - v)
    k = np.where(d < 0, lo, np.where(d > 0, hi, np.where(lo % 2 == 0, lo, hi)))
    q = k + 128 * np.signbit(b)
    return q.reshape(x.shape).astype(np.uint8), code.astype(np.uint8)


def weights(rng, N, K, fmt):
    """Random 4-bit weights: every nibble, scales within a few powers of two of each other."""
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    if fmt == "nvfp4":
        return q, rng.integers(0x20, 0x50, (N, K // 16), dtype=np.uint8)
    return q, rng.integers(118, 126, (N, K // 32), dtype=np.uint8)
