"""8-bit activation checkpoints in float64: blocks of 32 columns, int8 codes, power-of-two scales."""
import numpy as np

BLOCK = 32


def encode(X):
    """(codes int8 [T, K], biased exponents uint8 [T, ceil(K/32)]) of finite X [T, K]."""
    X = np.asarray(X, dtype=np.float64)
    T, K = X.shape
    nb = -(-K // BLOCK)
    codes, exps = np.zeros((T, K), np.int8), np.zeros((T, nb), np.uint8)
    for b in range(nb):
        x = X[:, b * BLOCK:(b + 1) * BLOCK]
        top = np.abs(x).max(axis=1) if K else np.zeros(T)
        e = np.full(T, -126)
        for k in range(-126, 122):  # the smallest exponent that covers the block
            e = np.where(top > 127 * 2.0 ** k, min(k + 1, 121), e)
        exps[:, b] = e + 127
        q = np.rint(x / (2.0 ** e)[:, None])  # rint rounds halves to even
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.clip(q, -127, 127)
    return codes, exps


def decode(codes, exps):
    K = codes.shape[1]
    scale = np.repeat(2.0 ** (exps.astype(np.int64) - 127), BLOCK, axis=1)[:, :K]
    return codes.astype(np.float64) * scale
