"""TEST INFRASTRUCTURE ONLY: the gated linear recurrence and its gradients in fp64 numpy, token by
token from the definition (no code shared with the GPU library).

    u_t = A sigmoid(r_t), a_t = exp(u_t), b_t = sqrt(1 - a_t^2) sigmoid(g_t) x_t
    h_t = a_t h_{t-1} + b_t,  y_t = h_t silu(z_t)
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    v = np.asarray(v, np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def _coefficients(r, g, A):
    s, i = sigmoid(r), sigmoid(g)
    u = np.asarray(A, np.float64) * s
    return s, i, np.exp(u), np.sqrt(-np.expm1(2.0 * u))


def step(state, x, r, g, A, z=None):
    """(y, new state) of one token."""
    _, i, a, beta = _coefficients(r, g, A)
    h = a * np.asarray(state, np.float64) + beta * i * np.asarray(x, np.float64)
    return (h if z is None else h * np.asarray(z, np.float64) * sigmoid(z)), h


def _lengths(seq_lens, bsz, L):
    return [L] * bsz if seq_lens is None else [int(min(max(n, 0), L)) for n in seq_lens]


def scan(x, r, g, A, z=None, h0=None, seq_lens=None):
    """y (bsz, L, D), zero past each length, and the state after each length (bsz, D)."""
    bsz, L, D = x.shape
    y = np.zeros((bsz, L, D))
    last = np.zeros((bsz, D)) if h0 is None else np.array(h0, np.float64)
    for b, n in enumerate(_lengths(seq_lens, bsz, L)):
        for t in range(n):
            y[b, t], last[b] = step(last[b], x[b, t], r[b, t], g[b, t], A, None if z is None else z[b, t])
    return y, last


def grads(dy, x, r, g, A, z=None, h0=None, seq_lens=None, dlast=None):
    """Gradients of sum(dy * y) + sum(dlast * last): a dict dx, dr, dg, dz, dA, dinitial_state."""
    bsz, L, D = x.shape
    A = np.asarray(A, np.float64)
    out = {k: np.zeros((bsz, L, D)) for k in ("dx", "dr", "dg", "dz")}
    out["dA"], out["dinitial_state"] = np.zeros(D), np.zeros((bsz, D))
    for b, n in enumerate(_lengths(seq_lens, bsz, L)):
        states = [np.zeros(D) if h0 is None else np.asarray(h0[b], np.float64)]
        for t in range(n):
            states.append(step(states[-1], x[b, t], r[b, t], g[b, t], A)[1])
        carry = np.zeros(D) if dlast is None else np.asarray(dlast[b], np.float64).copy()
        for t in range(n - 1, -1, -1):
            s, i, a, beta = _coefficients(r[b, t], g[b, t], A)
            xt, d = np.asarray(x[b, t], np.float64), np.asarray(dy[b, t], np.float64)
            if z is not None:
                zt = np.asarray(z[b, t], np.float64)
                sz = sigmoid(zt)
                out["dz"][b, t] = d * states[t + 1] * sz * (1.0 + zt * (1.0 - sz))
                d = d * zt * sz
            lam = d + carry
            carry = a * lam
            out["dx"][b, t] = lam * beta * i
            out["dg"][b, t] = lam * beta * xt * i * (1.0 - i)
            with np.errstate(divide="ignore", invalid="ignore"):
                dbeta = np.where(beta > 0, a * a / beta, 0.0)   # -d beta / d log a
            du = lam * (a * states[t] - i * xt * dbeta)
            out["dr"][b, t] = du * A * s * (1.0 - s)
            out["dA"] += du * s
        out["dinitial_state"][b] = carry
    if z is None:
        del out["dz"]
    return out
