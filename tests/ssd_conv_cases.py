"""Seeded cases of the state space dual layer with its convolution for the GPU tests, and their checks against the fp64
oracle.

Tolerances, relative to the rms of the reference and before the final rounding to bf16:
- What is formed between products of bf16 operands and leaves in bf16 is carried as two bf16 parts, off by at most
  2^-8 * 2^-8 = 2^-16 of its value.  An output is a sum of at most n = 64 + 128 such terms, whose absolute sum is at most
  sqrt(n) times their root of squares, and the largest outputs are about 5 of the root of squares: 2^-16 * 14 * 5 =
  1.1e-3, three such sums in a row at most: BF = 3.3e-3 bounds outputs in bf16.
- fp32 results (states, sums; everything with fp32 I/O): a token adds at most three roundings of 2^-24 to a state
  of at most ~4 rms, so 1000 tokens as a random walk give sqrt(1000) * 3 * 4 * 6e-8 = 2.3e-5, and four times
  that, F32 = 1e-4, is the bound.
- Sums over tokens (gradients of parameters) may cancel: their errors, those of their terms (2^-16 each with bf16
  I/O, hence BF), are held against the root of the sum of squares of the terms."""
import numpy as np
import torch

from gpu_util import to_dev, to_host_f64, y_error
from oracle import ssd_conv
from selective_state_space_32_amd import inputs, ssmscan

BF, F32 = 3.3e-3, 1e-4
SUMS = ("dA", "dD", "ddt_bias", "dconv_b", "dconv_w")


class Case:
    """Device tensors in `t`, the values they hold in fp64 in `v`."""

    def __init__(self, bsz, L, H, P, G, N, io, seed, W=4, state=True, lens=None, parts=True, softplus=True, extra=0, scale=1.0):
        rng = np.random.default_rng(seed)
        n = lambda *s: rng.standard_normal(s, dtype=np.float32)
        self.io, self.dims, self.W, self.lens, self.softplus = io, (bsz, L, H, P, G, N), W, lens, softplus
        self.t, self.v = {}, {}
        hp, row = H * P, H * P + 2 * G * N
        proj = n(bsz, L, hp + row + H + extra)      # a projected row: gate | x B C | step sizes | more
        proj[..., :hp + row] *= scale
        proj[..., hp + row:] *= 0.5
        if not softplus:
            proj[..., hp + row:] = np.abs(proj[..., hp + row:]) * 0.1
        self._add("proj", proj, io)
        for k, lo, hi in (("xbc", hp, hp + row), ("dt", hp + row, hp + row + H)):
            self.v[k] = self.v["proj"][..., lo:hi]
            self.t[k] = self.t["proj"][..., lo:hi]
            if parts is False:
                self.t[k] = self.t[k].contiguous()
        self._add("conv_w", 0.5 * n(row, W), "f32")
        self._add("conv_b", 0.1 * n(row), "f32")
        self._add("A", -np.exp(rng.uniform(0.0, np.log(16.0), H)), "f32")
        self._add("D", n(H), "f32")
        bias = np.log(np.expm1(np.exp(rng.uniform(np.log(1e-3), np.log(0.1), H))))
        self._add("dt_bias", bias if softplus else np.abs(bias) * 0.01, "f32")
        self._add("dy", n(bsz, L, H, P) * scale, io)
        if state:
            self._add("h0", n(bsz, H, P, N), "f32")
            self._add("dlast", n(bsz, H, P, N), "f32")
            self._add("conv_state", n(bsz, W - 1, row) * scale, io)
        self.t["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")

    def _add(self, k, a, io):
        a = np.asarray(a, np.float32)
        if io == "bf16":
            bits = inputs.bf16_bits(a)
            self.t[k], self.v[k] = to_dev(bits, torch), inputs.bf16_to_f32(bits).astype(np.float64)
        else:
            self.t[k], self.v[k] = to_dev(a, torch), a.astype(np.float64)

    def layer(self):
        g = self.t.get
        return (g("xbc"), g("conv_w"), g("conv_b"), g("dt"), g("A"), g("D"), g("dt_bias"), self.softplus)

    def shape(self):
        return dict(dstate=self.dims[5], ngroups=self.dims[4])

    def start(self):
        return dict(conv_state=self.t.get("conv_state"), initial_state=self.t.get("h0"), seq_lens=self.t["lens"])

    def oracle(self):
        g = self.v.get
        rounded = (lambda u: inputs.bf16_to_f32(inputs.bf16_bits(np.asarray(u, np.float32))).astype(np.float64)) if self.io == "bf16" else (lambda u: u)
        return ssd_conv.Layer(g("xbc"), g("conv_w"), g("conv_b"), g("dt"), g("A"), g("D"), g("dt_bias"), self.dims[5], self.dims[4],
                              conv_state=g("conv_state"), h0=g("h0"), seq_lens=self.lens, softplus=self.softplus, rounded=rounded)


def run_fwd(c, **kw):
    out = ssmscan.ssd_conv_fwd(*c.layer(), **c.shape(), **c.start(), **kw)
    torch.cuda.synchronize()
    return out


def run_bwd(c, checkpoints=None, **kw):
    g = ssmscan.ssd_conv_bwd(c.t["dy"], *c.layer(), **c.shape(), **c.start(), dlast_state=c.t.get("dlast"),
                             want_initial_state_grad=True, want_conv_state_grad=True, checkpoints=checkpoints, **kw)
    torch.cuda.synchronize()
    return g


def close(got, ref, io, tol, label):
    got = to_host_f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), label
    if not ref.size:
        return
    e = y_error(got, ref, io) if np.any(ref) else float(np.abs(got).max())
    print(f"{label}: err/rms {e:.2e} (tol {tol:.1e})", flush=True)
    assert e <= tol, (label, e)


def close_sum(got, ref, scale, tol, label):
    got = to_host_f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), label
    e = float(np.max(np.abs(got - ref) / np.maximum(scale, np.sqrt(np.mean(scale ** 2)) + 1e-300))) if ref.size else 0.0
    print(f"{label}: err/terms {e:.2e} (tol {tol:.1e})", flush=True)
    assert e <= tol, (label, e)


def check_fwd(c, label=""):
    print(f"[{label}] {c.dims} {c.io}", flush=True)
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    ry, rlast, rrows = c.oracle().scan()
    close(y, ry, c.io, BF if c.io == "bf16" else F32, "y")
    close(last, rlast, "f32", F32, "last_state")
    assert np.array_equal(to_host_f64(rows), rrows), "conv_state"
    y2, last2, rows2 = run_fwd(c)
    assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(rows, rows2)
    return ck


def check_bwd(c, ck, label=""):
    tol = BF if c.io == "bf16" else F32
    ref, scale = c.oracle().grads(c.v["dy"], c.v.get("dlast"))
    one, two = run_bwd(c, ck), run_bwd(c)
    assert set(one) == set(ref)
    for k, r in ref.items():
        if k in SUMS:
            close_sum(one[k], r, scale[k], tol, k)
        else:
            close(one[k], r, "f32" if k == "dinitial_state" else c.io, F32 if k == "dinitial_state" else tol, k)
        assert torch.equal(one[k], two[k]), f"{k}: other values without the forward's states"


def check(c, label=""):
    check_bwd(c, check_fwd(c, label), label)
