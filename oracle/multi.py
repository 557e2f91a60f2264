"""Many adapters beside one projection in float64: every token with the adapter its id names."""
import numpy as np


def forward(X, Ws, A, B, ids):
    """(Y, U) of X [T, K], dense Ws [N, K], A [n, r, K], B [n, N, r], ids [T]."""
    n, r = A.shape[:2]
    Y, U = X @ Ws.T, np.zeros((X.shape[0], r))
    for t, g in enumerate(ids):
        if 0 <= g < n:
            U[t] = A[g] @ X[t]
            Y[t] += B[g] @ U[t]
    return Y, U


def backward(dY, X, U, P, A, B, ids):
    """dX, dA, dB, dU with dense P [K, N]."""
    n, r = A.shape[:2]
    dX, dU = dY @ P.T, np.zeros((dY.shape[0], r))
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for t, g in enumerate(ids):
        if 0 <= g < n:
            dU[t] = dY[t] @ B[g]
            dX[t] += dU[t] @ A[g]
            dA[g] += np.outer(dU[t], X[t])
            dB[g] += np.outer(dY[t], U[t])
    return dict(dX=dX, dA=dA, dB=dB, dU=dU)
