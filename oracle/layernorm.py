"""TEST INFRASTRUCTURE ONLY: layer norm over the last axis and its gradients in fp64 numpy, row by
row from the definition (no code shared with the GPU library)."""
from __future__ import annotations

import numpy as np


def forward(s, w, b=None, eps=1e-5):
    """(y, mean, rstd) of the rows s (M, D)."""
    s = np.asarray(s, np.float64)
    mean = s.mean(-1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(-1) + eps)
    y = (s - mean[:, None]) * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def grads(dy, s, w, mean, rstd, dres=None):
    """ds, dweight, dbias of sum(dy * y) + sum(dres * s) with the given statistics of s."""
    dy, s, w = (np.asarray(v, np.float64) for v in (dy, s, w))
    n = (s - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    t = dy * w
    ds = (t - t.mean(-1, keepdims=True) - n * (t * n).mean(-1, keepdims=True)) * np.asarray(rstd, np.float64)[:, None]
    if dres is not None:
        ds = ds + dres
    return dict(ds=ds, dweight=(dy * n).sum(0), dbias=dy.sum(0))
