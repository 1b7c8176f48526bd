"""The fp64 oracle of the gated linear recurrence (oracle/gated.py) pinned by closed forms and
differences, so that it can check the GPU kernels.

Tolerances: fp64 sums of at most a few hundred terms of size one, relative error below 1e-12.
Central differences with step 1e-5 have an error of step^2 / 6 times a third derivative of size one
(2e-11) plus rounding 1e-16 * |loss| / step (|loss| < 1e3: 1e-8): bound 1e-6."""
import numpy as np
import pytest

from oracle import gated


def _case(bsz, L, D, seed, gate=True):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)
    return dict(x=n(bsz, L, D), r=n(bsz, L, D), g=n(bsz, L, D), A=-np.exp(n(D) - 1.0),
                z=n(bsz, L, D) if gate else None, h0=n(bsz, D))


def test_constant_gates_closed_form():
    """Constant decay a and input b: h_n = a^n h_0 + b (1 - a^n) / (1 - a)."""
    D, L = 3, 40
    A = np.array([-0.5, -0.01, -2.0])
    r = np.full((1, L, D), 0.3)
    g = np.full((1, L, D), -0.2)
    x = np.full((1, L, D), 1.7)
    h0 = np.array([[0.5, -1.0, 2.0]])
    y, last = gated.scan(x, r, g, A, h0=h0)
    a = np.exp(A / (1.0 + np.exp(-0.3)))
    b = np.sqrt(1.0 - a * a) / (1.0 + np.exp(0.2)) * 1.7
    for n in (1, 7, 40):
        ref = a ** n * h0[0] + b * (1.0 - a ** n) / (1.0 - a)
        assert np.allclose(y[0, n - 1], ref, rtol=1e-12, atol=0)
    assert np.array_equal(last[0], y[0, -1])


def test_variance_is_kept():
    """With independent inputs of variance 1 and an open input gate the state's variance tends to 1."""
    rng = np.random.default_rng(1)
    L, D = 400, 4000
    x = rng.standard_normal((1, L, D))
    y, last = gated.scan(x, np.zeros((1, L, D)), np.full((1, L, D), 40.0), np.full(D, -0.2))
    assert abs(last.var() - 1.0) < 6.0 * np.sqrt(2.0 / D)   # six standard deviations of the estimate


def test_open_and_closed_gates():
    """r -> -inf: the state stays as it is; A = 0 likewise; a huge decay forgets the past."""
    x, g = np.ones((1, 1, 2)), np.zeros((1, 1, 2))
    h0 = np.array([[3.0, -4.0]])
    for r, A in ((np.full((1, 1, 2), -800.0), np.array([-1.0, -2.0])), (np.zeros((1, 1, 2)), np.zeros(2))):
        assert np.array_equal(gated.scan(x, r, g, A, h0=h0)[1], h0)
    y, last = gated.scan(x, np.full((1, 1, 2), 40.0), g, np.array([-1e4, -1e4]), h0=h0)
    assert np.allclose(last, 0.5, rtol=1e-12)


def test_pieces_and_lengths():
    c = _case(3, 20, 4, 2)
    seq = [20, 0, 11]
    y, last = gated.scan(**c, seq_lens=seq)
    for b, n in enumerate(seq):
        one = {k: (v if v is None or k == "A" else v[b:b + 1, :n] if v.ndim == 3 else v[b:b + 1]) for k, v in c.items()}
        yb, lb = gated.scan(**one)
        assert np.array_equal(y[b, :n], yb[0]) and np.array_equal(last[b], lb[0]) and not y[b, n:].any()
    assert np.array_equal(last[1], c["h0"][1])


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("seq", [None, [6, 0, 3]])
def test_gradients_against_differences(gate, seq):
    c = _case(3, 6, 2, 3, gate)
    rng = np.random.default_rng(4)
    dy, dlast = rng.standard_normal(c["x"].shape), rng.standard_normal(c["h0"].shape)
    got = gated.grads(dy, **c, seq_lens=seq, dlast=dlast)

    def loss(cc):
        y, last = gated.scan(**cc, seq_lens=seq)
        return float((y * dy).sum() + (last * dlast).sum())
    for k, name in (("x", "dx"), ("r", "dr"), ("g", "dg"), ("z", "dz"), ("A", "dA"), ("h0", "dinitial_state")):
        if c[k] is None:
            assert name not in got
            continue
        num = np.zeros_like(c[k])
        for at in np.ndindex(*c[k].shape):
            v = []
            for sign in (1.0, -1.0):
                cc = dict(c, **{k: c[k].copy()})
                cc[k][at] += sign * 1e-5
                v.append(loss(cc))
            num[at] = (v[0] - v[1]) / 2e-5
        assert np.abs(num - got[name]).max() < 1e-6, (k, np.abs(num - got[name]).max())


def test_mutants_are_seen():
    """Each term of the gradients matters: a formula without it is far from the oracle's."""
    c = _case(2, 12, 8, 5)
    rng = np.random.default_rng(6)
    dy = rng.standard_normal(c["x"].shape)
    ref = gated.grads(dy, **c)
    no_gate = gated.grads(dy, **dict(c, z=None))
    no_state = gated.grads(dy, **dict(c, h0=None))
    for k in ("dx", "dr", "dg", "dA"):
        assert np.abs(ref[k] - no_gate[k]).max() > 1e-2 * np.abs(ref[k]).max()
    assert np.abs(ref["dr"] - no_state["dr"]).max() > 1e-2 * np.abs(ref["dr"]).max()
