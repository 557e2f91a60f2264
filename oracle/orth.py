"""Newton-Schulz steps on a matrix in float64, step by step on the matrix itself."""
import numpy as np


def orthogonalize(G, steps, coeffs, eps):
    a, b, c = coeffs
    X = np.asarray(G, dtype=np.float64)
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (np.sqrt((X ** 2).sum()) + eps)
    for _ in range(steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.T if tall else X
