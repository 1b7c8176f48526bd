"""A block's operators together, as they are used: layer norm with the residual sum, projection, the state space dual
layer with its convolution, the gated group norm, projection -- a prompt and then single tokens, and the gradients of a
training step -- against the fp64 oracles in a row.

Tolerances: with fp32 I/O every operator is within 1e-4 of the rms for inputs that are right (their own tests); three
in a row, and projections of 64 terms (their fp32 roundings are smaller), 4e-4.  Parameter sums are held against the
root of the sum of squares of their terms.  With bf16 the values between the operators are rounded, which the oracle
does not follow: 2^-8 each, of which a block has five in a row, random: 5 of the largest of a thousand values are 4
standard deviations (a rounding's is 2^-8 / sqrt(3)) of sqrt(5): 2^-8 / 1.7 * 2.2 * 4 = 2.1e-2 of the rms and of the value."""
import numpy as np
import pytest

from gpu_util import rms, to_host_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import groupnorm, ssd_conv  # noqa: E402
from selective_state_space_32_amd import ssmscan  # noqa: E402

EPS = 1e-5
WIDTH, H, P, G, N = 64, 6, 16, 2, 16
HP, ROW = H * P, H * P + 2 * G * N
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


class Block:
    def __init__(self, io, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=gen, device="cuda")
        self.io = IO[io]
        self.p = dict(nw=1 + 0.1 * n(WIDTH), nb=0.1 * n(WIDTH), conv_w=0.5 * n(ROW, 4), conv_b=0.1 * n(ROW),
                      A=-torch.exp(n(H).clamp(-2, 2)), D=n(H), dt_bias=n(H) - 2.0, gw=1 + 0.1 * n(HP))
        self.W_in = (n(WIDTH, HP + ROW + H) * WIDTH ** -0.5).to(self.io)
        self.W_out = (n(HP, WIDTH) * HP ** -0.5).to(self.io)

    def project(self, v, w):
        return (v.reshape(-1, v.shape[-1]) @ w).view(*v.shape[:-1], -1)

    def cut(self, proj):
        return proj[..., :HP], proj[..., HP:HP + ROW], proj[..., HP + ROW:]

    def layer(self, xbc, dt):
        p = self.p
        return xbc, p["conv_w"], p["conv_b"], dt, p["A"], p["D"], p["dt_bias"]

    def norm(self, y, z):
        return ssmscan.groupnorm_fwd(y.flatten(-2), self.p["gw"], None, EPS, groups=G, centre=False, z=z, gate_first=True)

    def prompt(self, x, lens=None, train=False):
        n, _, mean, rstd = ssmscan.layernorm_fwd(x, self.p["nw"], self.p["nb"], EPS)
        z, xbc, dt = self.cut(self.project(n, self.W_in))
        out = ssmscan.ssd_conv_fwd(*self.layer(xbc, dt), dstate=N, ngroups=G, seq_lens=lens, save_checkpoints=train)
        v, _, grstd = self.norm(out[0], z)
        if train:
            self.kept = (x, n, mean, rstd, z, xbc, dt, out[0], out[3], v, grstd, lens)
        return self.project(v, self.W_out), out[1], out[2]

    def token(self, x, state, rows):
        n = ssmscan.layernorm_fwd(x, self.p["nw"], self.p["nb"], EPS)[0]
        z, xbc, dt = self.cut(self.project(n, self.W_in))
        y = ssmscan.ssd_conv_step(state, rows, *self.layer(xbc, dt), dstate=N, ngroups=G)
        return self.project(self.norm(y, z)[0], self.W_out)

    def backward(self, dout):
        x, n, mean, rstd, z, xbc, dt, y, ck, v, grstd, lens = self.kept
        dv = self.project(dout, self.W_out.T.contiguous())
        g = ssmscan.groupnorm_bwd(dv, y.flatten(-2), self.p["gw"], None, None, grstd, groups=G, z=z, gate_first=True)
        s = ssmscan.ssd_conv_bwd(g["dx"].view(y.shape), *self.layer(xbc, dt), dstate=N, ngroups=G, seq_lens=lens, checkpoints=ck)
        dproj = torch.cat([g["dz"], s["dxbc"], s["ddt"]], -1)
        l = ssmscan.layernorm_bwd(self.project(dproj, self.W_in.T.contiguous()), x, self.p["nw"], mean, rstd)
        return dict(x=l["ds"], gw=g["dweight"], nw=l["dweight"], nb=l["dbias"],
                    **{k: s["d" + k] for k in ("conv_w", "conv_b", "A", "D", "dt_bias")})


def reference(b, x, lens, dout=None):
    """The block in fp64 numpy from the same parameters; (out, states, rows, gradients)."""
    h = lambda t: to_host_f64(t)
    p = {k: h(v) for k, v in b.p.items()}
    W_in, W_out, xv = h(b.W_in), h(b.W_out), h(x)
    bsz, L = xv.shape[:2]
    flat = xv.reshape(-1, WIDTH)
    mean = flat.mean(-1)
    rstd = 1.0 / np.sqrt(flat.var(-1) + EPS)
    nh = (flat - mean[:, None]) * rstd[:, None]
    proj = ((nh * p["nw"] + p["nb"]) @ W_in).reshape(bsz, L, -1)
    z, xbc, dt = proj[..., :HP], proj[..., HP:HP + ROW], proj[..., HP + ROW:]
    lay = ssd_conv.Layer(xbc, p["conv_w"], p["conv_b"], dt, p["A"], p["D"], p["dt_bias"], N, G, seq_lens=lens)
    y, last, rows = lay.scan()
    args = (y.reshape(-1, HP), p["gw"], None, G, EPS, z.reshape(-1, HP), "before", False)
    v = groupnorm.norm(*args)[0]
    out = (v @ W_out).reshape(bsz, L, WIDTH)
    if dout is None:
        return out, last, rows, None
    gn, _ = groupnorm.grads(h(dout).reshape(-1, WIDTH) @ W_out.T, *args)
    s, scale = lay.grads(gn["dx"].reshape(y.shape))
    dproj = np.concatenate([gn["dz"].reshape(z.shape), s["dxbc"], s["ddt"]], -1)
    dn = dproj.reshape(-1, dproj.shape[-1]) @ W_in.T
    w = dn * p["nw"]
    dx = rstd[:, None] * (w - w.mean(-1, keepdims=True) - nh * (w * nh).mean(-1, keepdims=True))
    g = dict(x=dx.reshape(xv.shape), gw=gn["dweight"], nw=(dn * nh).sum(0), nb=dn.sum(0),
             **{k: s["d" + k] for k in ("conv_w", "conv_b", "A", "D", "dt_bias")})
    return out, last, rows, g


def near(got, ref, tol, label):
    got = to_host_f64(got)
    e = float(np.max(np.abs(got - ref) / np.maximum(np.abs(ref), rms(ref))))
    print(f"{label}: {e:.2e} (tol {tol:.1e})", flush=True)
    assert got.shape == ref.shape and e <= tol, (label, e)


@pytest.mark.parametrize("io,tol", [("f32", 4e-4), ("bf16", 2.1e-2 * 2)])
def test_prompt_then_tokens(io, tol):
    """(The states after the prompt carry the roundings too, hence twice the bound with bf16.)"""
    b = Block(io, 1)
    x = torch.randn(3, 75, WIDTH, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(b.io)
    ref, last, rows, _ = reference(b, x, None)
    out, state, conv = b.prompt(x[:, :70].contiguous())
    near(out, ref[:, :70], tol, "prompt")
    for t in range(70, 75):
        near(b.token(x[:, t].contiguous(), state, conv), ref[:, t], tol, f"token {t}")
    near(state, last, tol, "state")


def test_training_step():
    """fp32, a padded batch; every gradient against the oracles' in a row."""
    b = Block("f32", 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(3, 90, WIDTH, device="cuda", generator=gen)
    dout = torch.randn(3, 90, WIDTH, device="cuda", generator=gen)
    lens = [90, 0, 41]
    for k, n in enumerate(lens):
        dout[k, n:] = 0.0
    out, state, _ = b.prompt(x, torch.tensor(lens, dtype=torch.int32, device="cuda"), train=True)
    got = b.backward(dout)
    ref, last, _, g = reference(b, x, lens, dout)
    for k, n in enumerate(lens):
        if n:
            near(out[k, :n], ref[k, :n], 4e-4, f"sequence {k}")
    near(state, last, 4e-4, "state")
    assert set(got) == set(g)
    for k in g:
        near(got[k], g[k], 4e-4, k)


def test_training_step_in_a_graph():
    """The same training step captured: replays give the eager gradients, beside eager ones of the same inputs."""
    b = Block("bf16", 5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, dout = (torch.randn(2, 130, WIDTH, device="cuda", generator=gen).bfloat16() for _ in range(2))
    b.prompt(x, train=True)
    eager = {k: v.clone() for k, v in b.backward(dout).items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.prompt(x, train=True)
        got = b.backward(dout)
    kept = b.kept
    for _ in range(3):
        for v in got.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(eager[k], got[k]) for k in eager)
        b.prompt(x, train=True)
        again = b.backward(dout)
        assert all(torch.equal(eager[k], again[k]) for k in eager)
    del kept
