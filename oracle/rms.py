"""Root-mean-square norm of X + R over rows in float64, and its gradients."""
import numpy as np


def forward(X, R, gamma, eps):
    H = np.asarray(X, dtype=np.float64) + (0.0 if R is None else np.asarray(R, dtype=np.float64))
    rstd = 1.0 / np.sqrt((H ** 2).sum(axis=1) / H.shape[1] + eps)
    return H * rstd[:, None] * gamma, H, rstd


def backward(dY, H, gamma, rstd, dH=None):
    xh = H * rstd[:, None]
    g = dY * gamma
    dX = rstd[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    return dX + (0.0 if dH is None else dH), (dY * xh).sum(axis=0)
