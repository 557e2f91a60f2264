"""8-bit floating point with a power-of-two scale for each block of 128 columns, in float64."""
import numpy as np

BLOCK = 128
KINDS = {"e4m3": (4, 3, 7, 0x7E, 119), "e5m2": (5, 2, 15, 0x7B, 112)}  # exponent bits, mantissa bits, bias, last finite code, top exponent


def values(kind):
    """The 256 codes' values; NaN where a code is none (e5m2's infinities are kept)."""
    eb, mb, bias, last, _ = KINDS[kind]
    v = np.full(256, np.nan)
    for c in range(128):
        e, m = c >> mb, c & ((1 << mb) - 1)
        if c <= last:
            v[c] = (m / 2 ** mb) * 2.0 ** (1 - bias) if e == 0 else (1 + m / 2 ** mb) * 2.0 ** (e - bias)
        elif kind == "e5m2" and m == 0:
            v[c] = np.inf
        v[c + 128] = -v[c]
    return v


def nearest(v, kind):
    """Codes of v, inside the type's range: the nearest value, ties to the even code; NaN where v is."""
    last = KINDS[kind][3]
    pos = values(kind)[:last + 1]
    a = np.minimum(np.abs(np.nan_to_num(v)), pos[-1])
    hi = np.clip(np.searchsorted(pos, a), 1, last)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isnan(v), 0x7F, c + 128 * np.signbit(v))
    return c.astype(np.uint8)


def encode(X, kind, block_rows=1):
    """(codes uint8 [R, C rounded up], biased exponents uint8 [ceil(R / block_rows), ceil(C / 128)])."""
    X = np.asarray(X, dtype=np.float64)
    R, C = X.shape
    top, most = values(kind)[KINDS[kind][3]], KINDS[kind][4]
    nr, nc = -(-R // block_rows), -(-C // BLOCK)
    codes, exps = np.zeros((R, nc * BLOCK), np.uint8), np.zeros((nr, nc), np.uint8)
    for i in range(nr):
        for j in range(nc):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            x = X[at]
            live = np.abs(x[np.isfinite(x)])
            e = -126
            while e < most and live.size and live.max() > top * 2.0 ** e:
                e += 1
            exps[i, j] = e + 127
            codes[at][:, :x.shape[1]] = nearest(np.where(np.isfinite(x), x / 2.0 ** e, np.nan), kind)
    return codes, exps


def decode(codes, exps, kind, cols, block_rows=1):
    s = np.repeat(np.repeat(2.0 ** (exps.astype(np.int64) - 127), block_rows, axis=0)[:codes.shape[0]], BLOCK, axis=1)
    return (values(kind)[codes] * s)[:, :cols]
