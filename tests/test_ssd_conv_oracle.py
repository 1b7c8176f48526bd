"""The fp64 oracles of the state space dual layer with its convolution (oracle/ssd_conv.py) and of the group norm
(oracle/groupnorm.py) pinned by the layer's own oracle, closed forms and differences, so that they can check the
GPU kernels.

Tolerances: fp64 sums of at most a few hundred terms of size one, relative error below 1e-12.  Central differences
with step 1e-5 have an error of step^2 / 6 times a third derivative of at most 1e3 (2e-8) plus rounding 1e-16 *
|loss| / step (|loss| < 1e3: 1e-8): bound 1e-6 of a directional derivative of size one."""
import numpy as np
import pytest

from oracle import groupnorm, ssd_conv


def _case(bsz, L, H, P, G, N, seed, W=4):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)
    row = H * P + 2 * G * N
    return dict(xbc=n(bsz, L, row), conv_w=0.5 * n(row, W), conv_b=0.1 * n(row), dt=n(bsz, L, H) - 1.0,
                A=-np.exp(n(H)), D=n(H), dt_bias=0.3 * n(H), conv_state=n(bsz, W - 1, row), h0=n(bsz, H, P, N),
                dstate=N, ngroups=G)


def test_against_the_layers_oracle(oracle_mod):
    """Without history, the layer's C oracle on the convolution's output gives the same y and states."""
    c = _case(2, 23, 4, 8, 2, 8, 1)
    del c["conv_state"], c["h0"]
    lay = ssd_conv.Layer(**c)
    y, last, _ = lay.scan()
    hp = 4 * 8
    x = lay.u[..., :hp].reshape(2, 23, 4, 8)
    B, C = (lay.u[..., hp + k * 16:hp + (k + 1) * 16].reshape(2, 23, 2, 8) for k in (0, 1))
    f = lambda a: np.ascontiguousarray(a, np.float32)
    ry, rl = oracle_mod.ssd(f(x), f(c["dt"]), f(c["A"]), f(B), f(C), D=f(c["D"]), dt_bias=f(c["dt_bias"]), softplus=True)
    # (that oracle takes fp32 inputs: 2^-24 of each)
    assert np.allclose(y, ry, rtol=0, atol=2e-6 * np.sqrt(np.mean(ry ** 2)) * 8)
    assert np.allclose(last, rl, rtol=0, atol=2e-6 * np.sqrt(np.mean(rl ** 2)) * 8)


def test_constant_inputs_closed_form():
    """Constant u and dt: S_n = a^n S_0 + dt x B^T (1 - a^n) / (1 - a)."""
    H, P, N, L = 2, 8, 8, 12
    c = _case(1, L, H, P, 1, N, 2, W=1)
    c.update(xbc=np.ones_like(c["xbc"]) * np.linspace(-1, 1, c["xbc"].shape[-1]), dt=np.full((1, L, H), 0.2))
    lay = ssd_conv.Layer(**c)
    _, last, _ = lay.scan()
    x, B, _ = lay.parts(0, 0)
    d = lay.dt[0, 0]
    a = np.exp(c["A"] * d)[:, None, None]
    ref = a ** L * c["h0"][0] + (d[:, None] * x)[:, :, None] * B[:, None, :] * (1 - a ** L) / (1 - a)
    assert np.allclose(last[0], ref, rtol=1e-12, atol=1e-12)


def test_pieces_and_lengths():
    c = _case(3, 15, 2, 8, 1, 8, 3)
    y, last, rows = ssd_conv.Layer(**c, seq_lens=[15, 0, 7]).scan()
    for b, n in enumerate([15, 0, 7]):
        assert not y[b, n:].any()
        one = {k: v[b:b + 1] if k in ("xbc", "dt", "conv_state", "h0") else v for k, v in c.items()}
        cut = lambda d, lo, hi: dict(d, xbc=d["xbc"][:, lo:hi], dt=d["dt"][:, lo:hi])
        k = n // 2
        y1, s1, r1 = ssd_conv.Layer(**cut(one, 0, k)).scan()
        y2, s2, r2 = ssd_conv.Layer(**dict(cut(one, k, n), conv_state=r1, h0=s1)).scan()
        assert np.allclose(np.concatenate([y1, y2], 1)[0], y[b, :n], rtol=1e-12, atol=1e-12)
        assert np.allclose(s2[0], last[b], rtol=1e-12, atol=1e-12) and np.array_equal(r2[0], rows[b])


@pytest.mark.parametrize("W", [1, 2, 4])
@pytest.mark.parametrize("softplus", [True, False])
def test_gradients_against_differences(W, softplus):
    c = _case(2, 9, 4, 8, 2, 8, 4 + W, W=W)
    if not softplus:
        c["dt"] = np.abs(c["dt"])
        c["dt_bias"] = np.abs(c["dt_bias"])
    rng = np.random.default_rng(9)
    lens = [9, 5]
    wy, wl = rng.standard_normal((2, 9, 4, 8)), rng.standard_normal(c["h0"].shape)
    wy[1, 5:] = 0.0

    def loss(c):
        y, last, _ = ssd_conv.Layer(**c, seq_lens=lens, softplus=softplus).scan()
        return (y * wy).sum() + (last * wl).sum()
    g, _ = ssd_conv.Layer(**c, seq_lens=lens, softplus=softplus).grads(wy, wl)
    names = dict(xbc="dxbc", conv_w="dconv_w", conv_b="dconv_b", dt="ddt", A="dA", D="dD", dt_bias="ddt_bias", h0="dinitial_state")
    if W > 1:
        names["conv_state"] = "dconv_state"
    for k, name in names.items():
        v = rng.standard_normal(c[k].shape)
        v /= np.sqrt((v ** 2).sum())
        h = 1e-5
        diff = (loss(dict(c, **{k: c[k] + h * v})) - loss(dict(c, **{k: c[k] - h * v}))) / (2 * h)
        assert abs(diff - (g[name] * v).sum()) <= 1e-6 * max(1.0, np.sqrt((g[name] ** 2).sum())), k


@pytest.mark.parametrize("gate", ["none", "before", "after", "silu"])
@pytest.mark.parametrize("centre", [True, False])
def test_group_norm_gradients_against_differences(gate, centre):
    rng = np.random.default_rng(11)
    m, d, groups = 3, 24, 3
    c = dict(x=rng.standard_normal((m, d)), w=rng.standard_normal(d), b=rng.standard_normal(d))
    if gate in ("before", "after"):
        c["z"] = rng.standard_normal((m, d))
    wy = rng.standard_normal((m, d))
    loss = lambda c: (groupnorm.norm(groups=groups, eps=1e-3, gate=gate, centre=centre, **c)[0] * wy).sum()
    g, _ = groupnorm.grads(wy, groups=groups, eps=1e-3, gate=gate, centre=centre, **c)
    for k, name in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("z", "dz")):
        if k not in c:
            continue
        v = rng.standard_normal(c[k].shape)
        v /= np.sqrt((v ** 2).sum())
        h = 1e-5
        diff = (loss(dict(c, **{k: c[k] + h * v})) - loss(dict(c, **{k: c[k] - h * v}))) / (2 * h)
        assert abs(diff - (g[name] * v).sum()) <= 1e-6 * max(1.0, np.sqrt((g[name] ** 2).sum())), k


def test_group_norm_invariants():
    """Unit statistics per group; one group is the layer norm; groups do not see each other."""
    rng = np.random.default_rng(12)
    x = rng.standard_normal((4, 30)) * 3 + 1
    y, mean, rstd = groupnorm.norm(x, np.ones(30), None, 3, 0.0)
    v = y.reshape(4, 3, 10)
    assert np.allclose(v.mean(-1), 0, atol=1e-13) and np.allclose(np.square(v).mean(-1), 1, rtol=1e-12)
    assert np.allclose(mean, x.reshape(4, 3, 10).mean(-1), rtol=1e-13)
    x2 = x.copy()
    x2[:, 10:20] *= 7
    assert np.array_equal(groupnorm.norm(x2, np.ones(30), None, 3, 0.0)[0][:, :10], y[:, :10])
    q = groupnorm.norm(x, np.ones(30), None, 1, 0.0, centre=False)[0]
    assert np.allclose(np.square(q).mean(-1), 1, rtol=1e-12)
