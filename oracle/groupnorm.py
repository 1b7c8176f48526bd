"""TEST INFRASTRUCTURE ONLY: the group norm over a row's channels with its activation, and its gradients, in
fp64 numpy from the definition (no code shared with the GPU library).

    v = x silu(z) ("before") or x;   n = (v - mean) rstd per group (mean only if centred)
    o = n w + b;   y = o, o silu(z) ("after") or silu(o) ("silu")
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def dsilu(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def _forward(x, w, b, groups, eps, z, gate, centre):
    x = np.asarray(x, np.float64)
    m, d = x.shape
    v = (x * z * sigmoid(z) if gate == "before" else x).reshape(m, groups, d // groups)
    mean = v.mean(-1) if centre else np.zeros((m, groups))
    c = v - mean[..., None]
    rstd = 1.0 / np.sqrt(np.square(c).mean(-1) + eps)
    n = (c * rstd[..., None]).reshape(m, d)
    o = n * w + (0.0 if b is None else b)
    y = o * z * sigmoid(z) if gate == "after" else o * sigmoid(o) if gate == "silu" else o
    return y, mean, rstd, n, o


def norm(x, w, b, groups, eps, z=None, gate="none", centre=True):
    return _forward(x, w, b, groups, eps, z, gate, centre)[:3]


def grads(dy, x, w, b, groups, eps, z=None, gate="none", centre=True):
    """(dict of gradients, the sizes of their terms: of dweight's and dbias's the root of the sum of squares over rows,
    of those that dv's projection may cancel the first term's)."""
    y, mean, rstd, n, o = _forward(x, w, b, groups, eps, z, gate, centre)
    m, d = n.shape
    out, do = {}, np.asarray(dy, np.float64)
    if gate == "after":
        out["dz"] = do * o * dsilu(z)
        do = do * z * sigmoid(z)
    elif gate == "silu":
        do = do * dsilu(o)
    dn, ng = (do * w).reshape(m, groups, -1), n.reshape(m, groups, -1)
    dv = dn - ng * (dn * ng).mean(-1, keepdims=True)
    if centre:
        dv = dv - dn.mean(-1, keepdims=True)
    dv, term = (dv * rstd[..., None]).reshape(m, d), (dn * rstd[..., None]).reshape(m, d)
    size = dict(dweight=np.sqrt(np.square(do * n).sum(0)), dbias=np.sqrt(np.square(do).sum(0)), dx=term)
    if gate == "before":
        out["dz"], size["dz"] = dv * x * dsilu(z), term * x * dsilu(z)
        dv, size["dx"] = dv * z * sigmoid(z), term * z * sigmoid(z)
    out["dx"] = dv
    out["dweight"], out["dbias"] = (do * n).sum(0), do.sum(0)
    return out, size
