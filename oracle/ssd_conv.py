"""TEST INFRASTRUCTURE ONLY: the state space dual layer with its causal convolution, and its gradients, in
fp64 numpy, token by token from the definition (no code shared with the GPU library).

    u_t = silu(conv_b + sum_k conv_w[:, k] row_{t - (W-1) + k}), rounded by `rounded` (x, B, C its parts)
    dt_t = softplus(raw_t + dt_bias),   S_t = exp(A dt_t) S_{t-1} + dt_t x_t B_t^T,   y_t = S_t C_t + D x_t
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    v = np.asarray(v, np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def softplus_of(v):
    v = np.asarray(v, np.float64)
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def lengths(seq_lens, bsz, L):
    return [L] * bsz if seq_lens is None else [int(min(max(n, 0), L)) for n in seq_lens]


class Layer:
    """One layer's inputs; `rounded` maps u to the values that the layer sees (identity by default)."""

    def __init__(self, xbc, conv_w, conv_b, dt, A, D, dt_bias, dstate, ngroups, conv_state=None, h0=None, seq_lens=None,
                 softplus=True, rounded=lambda u: u):
        f = lambda a: None if a is None else np.asarray(a, np.float64)
        self.xbc, self.w, self.cb, self.raw, self.A, self.D, self.bias = map(f, (xbc, conv_w, conv_b, dt, A, D, dt_bias))
        bsz, L, row = self.xbc.shape
        self.N, self.G, self.H, self.W = dstate, ngroups, self.A.shape[0], self.w.shape[1]
        self.P = (row - 2 * ngroups * dstate) // self.H
        self.lens = lengths(seq_lens, bsz, L)
        self.first = np.zeros((bsz, self.W - 1, row)) if conv_state is None else f(conv_state)
        self.h0 = np.zeros((bsz, self.H, self.P, dstate)) if h0 is None else f(h0)
        self.softplus = softplus
        self.full = np.concatenate([self.first, self.xbc], 1)            # token t at t + W - 1
        self.pre = (0.0 if self.cb is None else self.cb) + sum(self.w[:, k] * self.full[:, k:k + L] for k in range(self.W))
        self.u = rounded(self.pre * sigmoid(self.pre))
        v = self.raw + (0.0 if self.bias is None else self.bias)
        self.dt = softplus_of(v) if softplus else v
        self.sig = sigmoid(v) if softplus else np.ones_like(v)

    def parts(self, b, t):
        hp = self.H * self.P
        u, per = self.u[b, t], self.H // self.G
        x = u[:hp].reshape(self.H, self.P)
        B = np.repeat(u[hp:hp + self.G * self.N].reshape(self.G, self.N), per, 0)
        C = np.repeat(u[hp + self.G * self.N:].reshape(self.G, self.N), per, 0)
        return x, B, C

    def advance(self, b, t, S):
        x, B, _ = self.parts(b, t)
        return np.exp(self.A * self.dt[b, t])[:, None, None] * S + (self.dt[b, t][:, None] * x)[:, :, None] * B[:, None, :]

    def scan(self):
        """y (zero past each length), the last states, the convolution's last rows."""
        bsz, L = self.xbc.shape[:2]
        y, last = np.zeros((bsz, L, self.H, self.P)), self.h0.copy()
        rows = np.zeros_like(self.first)
        for b, n in enumerate(self.lens):
            for t in range(n):
                x, _, C = self.parts(b, t)
                last[b] = self.advance(b, t, last[b])
                y[b, t] = np.einsum("hpn,hn->hp", last[b], C) + (0.0 if self.D is None else self.D[:, None] * x)
            rows[b] = self.full[b, n:n + self.W - 1]
        return y, last, rows

    def grads(self, dy, dlast=None):
        """(gradients of sum(dy y) + sum(dlast last), root of the sums of squares of the terms of those that are
        sums over tokens)."""
        bsz, L, row = self.xbc.shape
        dy = np.asarray(dy, np.float64)
        H, P, G, N, W = self.H, self.P, self.G, self.N, self.W
        du, ddt = np.zeros((bsz, L, row)), np.zeros((bsz, L, H))
        lam_first = np.zeros_like(self.h0) if dlast is None else np.array(dlast, np.float64)
        tA, tD = np.zeros((bsz, L, H)), np.zeros((bsz, L, H))
        for b, n in enumerate(self.lens):
            states = [self.h0[b]]
            for t in range(n):
                states.append(self.advance(b, t, states[-1]))
            lam = lam_first[b]
            for t in range(n - 1, -1, -1):
                x, B, C = self.parts(b, t)
                g, d = dy[b, t], self.dt[b, t]
                dC = np.einsum("hp,hpn->hn", g, states[t + 1])
                lam = lam + g[:, :, None] * C[:, None, :]
                lB = np.einsum("hpn,hn->hp", lam, B)
                dx = d[:, None] * lB + (0.0 if self.D is None else self.D[:, None] * g)
                dB = np.einsum("hp,hpn->hn", d[:, None] * x, lam)
                a = np.exp(self.A * d)[:, None, None]
                dlog = np.einsum("hpn,hpn->h", lam * a, states[t])
                ddt[b, t] = ((lB * x).sum(-1) + self.A * dlog) * self.sig[b, t]
                tA[b, t], tD[b, t] = d * dlog, (g * x).sum(-1)
                du[b, t, :H * P] = dx.reshape(-1)
                du[b, t, H * P:H * P + G * N] = dB.reshape(G, H // G, N).sum(1).reshape(-1)
                du[b, t, H * P + G * N:] = dC.reshape(G, H // G, N).sum(1).reshape(-1)
                lam = a * lam
            lam_first[b] = lam
        s = sigmoid(self.pre)
        gr = du * (s * (1.0 + self.pre * (1.0 - s)))
        dfull = np.zeros_like(self.full)
        terms = np.zeros((bsz, L, row, W))
        for k in range(W):
            dfull[:, k:k + L] += self.w[:, k] * gr
            terms[..., k] = gr * self.full[:, k:k + L]
        out = dict(dxbc=dfull[:, W - 1:], dconv_state=dfull[:, :W - 1], ddt=ddt, dinitial_state=lam_first)
        scale = {}
        for k, t in (("dA", tA), ("dD", tD), ("ddt_bias", ddt), ("dconv_b", gr), ("dconv_w", terms)):
            out[k], scale[k] = t.sum((0, 1)), np.sqrt(np.square(t).sum((0, 1)))
        return out, scale

