"""fp64 definitions of the cache format in 4 bits: E2M1 codes, an E4M3 scale per
16 columns, one factor per tensor.  numpy only."""

import numpy as np

BLOCK = 16
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3(code):
    e, m = (code >> 3) & 15, code & 7
    if code & 127 == 127:
        return np.nan
    x = m * 2.0 ** -9 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)
    return -x if code & 128 else x


SCALES = np.array([_e4m3(c) for c in range(256)])


def _nearest(x, steps):
    """Index of the nearest of the ascending `steps`, ties to the even index."""
    middle = (steps[1:] + steps[:-1]) / 2
    low, high = np.searchsorted(middle, x, "left"), np.searchsorted(middle, x, "right")
    return np.where(low % 2 == 0, low, high)


def encode(x, descale):
    """codes uint8 [..., d / 2] and scales uint8 [..., d / 16] of x [..., d]: the scale
    nearest to max |x| / (6 descale), at most 448, the codes nearest to x / (s
    descale), at most 6.  The borders are compared as products with descale, which
    64 bits hold exactly."""
    D = float(np.float32(descale))
    x = np.asarray(x, dtype=np.float64).reshape(x.shape[:-1] + (-1, BLOCK))
    mag = np.abs(x)
    nan = np.isnan(x).any(-1)
    top = np.where(np.isnan(mag), 0.0, mag).max(-1)
    s = _nearest(top, 6 * SCALES[:127] * D)
    codes = np.zeros(x.shape, dtype=np.uint8)
    middle = (LEVELS[1:] + LEVELS[:-1]) / 2 * (SCALES[s] * D)[..., None, None]
    mag = np.where(np.isnan(mag), 0.0, mag)[..., None]
    low, high = (mag > middle).sum(-1), (mag >= middle).sum(-1)
    codes = np.where(low % 2 == 0, low, high) + 8 * np.signbit(x)
    codes = np.where((nan | (s == 0))[..., None], 0, codes).astype(np.uint8)
    codes = codes.reshape(codes.shape[:-2] + (-1,))
    return codes[..., ::2] | codes[..., 1::2] << 4, np.where(nan, 127, s).astype(np.uint8)


def decode(codes, scales, descale):
    """The values [..., d] in 64 bits."""
    signed = np.concatenate([LEVELS, -LEVELS])
    x = np.stack([signed[codes & 15], signed[codes >> 4]], -1).reshape(codes.shape[:-1] + (-1,))
    return x * np.repeat(SCALES[scales], BLOCK, -1) * float(np.float32(descale))
