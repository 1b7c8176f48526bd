"""Slow heads of the state space dual layer with its convolution: memories of tens of thousands of tokens, over sequences
several times as long, as a prompt, token by token and back, against the definition in fp64 (chunks of 64 in torch).

Tolerance of a state, relative to its rms.  A state is rounded where it is multiplied by a decay and where something is
added to it, each time by at most half a step, 2^-24 of itself; these roundings have no mean, and they are forgotten as
the state is, so that a memory of T tokens with n roundings a token holds a walk of n T / 2 steps of 2^-24 / sqrt(3).
T is at most 20,000 here.  One token at a time n = 1 (the sum; what is added is smaller by T): 100 steps' length,
3.5e-6 of a state, five times that at the worst of the elements, which are up to 4 rms: 7e-5.  In chunks of 64 tokens
n = 18 / 64 (the decay and at most 17 sums): 5.3e-1 of that.  STATE = 7e-5 covers both.  A decay that were itself
rounded would be off by up to 2^-25 in every token alike, 6e-4 after T of them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_32_amd import ssmscan  # noqa: E402

STATE = 7e-5
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


class Slow:
    """A layer whose heads remember 1 / `per_token` tokens, with step sizes that vary or not."""

    def __init__(self, bsz, L, H, P, N, io, per_token, vary, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
        self.dims, self.io = (bsz, L, H, P, N), io
        row = H * P + 2 * N
        self.x, self.w, self.cb = n(bsz, L, row).to(IO[io]), 0.5 * n(row, 4), 0.1 * n(row)
        self.raw = (0.3 * n(bsz, L, H) if vary else torch.zeros(bsz, L, H, device="cuda")).to(IO[io])
        self.A = -torch.linspace(1.0, 1.5, H, device="cuda")
        self.bias = torch.full((H,), float(np.log(np.expm1(per_token))), device="cuda")

    def args(self, at=slice(None)):
        return (self.x[:, at], self.w, self.cb, self.raw[:, at], self.A, None, self.bias)

    def definition(self, b):
        """y, the last state and what the chunks start from of sequence b, in fp64."""
        _, L, H, P, N = self.dims
        d = torch.float64
        pre = torch.zeros(L, self.x.shape[2], dtype=d, device="cuda") + self.cb.to(d)
        for k in range(4):
            pre[3 - k:] += self.w[:, k].to(d) * self.x[b, :L - 3 + k].to(d)
        u = pre * torch.sigmoid(pre)
        if self.io == "bf16":
            u = u.float().to(torch.bfloat16).to(d)
        X, B, C = u[:, :H * P].reshape(L, H, P), u[:, H * P:H * P + N], u[:, H * P + N:]
        dt = torch.nn.functional.softplus(self.raw[b].to(d) + self.bias.to(d))
        g = self.A.to(d) * dt
        S, y = torch.zeros(H, P, N, dtype=d, device="cuda"), torch.zeros(L, H, P, dtype=d, device="cuda")
        for t0 in range(0, L, 64):
            s = slice(t0, min(t0 + 64, L))
            c = torch.cumsum(g[s], 0)
            n = c.shape[0]
            low = torch.tril(torch.ones(n, n, dtype=d, device="cuda"))
            M = ((C[s] @ B[s].T.contiguous()) * low)[None] * (c.T[:, :, None] - c.T[:, None, :]).clamp(max=0).exp() * dt[s].T[:, None, :]
            Xh, Ch = X[s].permute(1, 0, 2).contiguous(), C[s][None] * c.T.exp()[:, :, None]
            y[s] = (torch.bmm(M, Xh) + torch.bmm(Ch, S.transpose(1, 2).contiguous())).permute(1, 0, 2)
            w = ((c[-1:] - c).exp() * dt[s]).T[:, :, None]
            S = c[-1].exp()[:, None, None] * S + torch.matmul((Xh * w).transpose(1, 2).contiguous(), B[s])
        return y, S


def close(got, want, tol, label):
    e = float((got.double() - want).abs().max() / want.pow(2).mean().sqrt())
    print(f"{label}: err/rms {e:.2e} (tol {tol:.1e})", flush=True)
    assert e <= tol, (label, e)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("vary", [True, False])
@pytest.mark.parametrize("per_token", [5e-5, 1e-3, 0.3, 3.0])
def test_tokens_one_by_one(io, vary, per_token):
    """(The fast heads: decays of 0.74 to 0.01 a token, on both sides of 1/2.)"""
    L = 60000 if per_token < 1e-4 else 3000
    c = Slow(1, L, 2, 16, 16, io, per_token, vary, seed=1)
    y, want = c.definition(0)
    st, cs = torch.zeros(1, 2, 16, 16, device="cuda"), torch.zeros(1, 3, c.x.shape[2], dtype=IO[io], device="cuda")
    for t in range(L):
        x, w, cb, raw, A, D, bias = c.args(t)
        out = ssmscan.ssd_conv_step(st, cs, x, w, cb, raw, A, D, bias, dstate=16)
    close(st[0], want, STATE, "state")
    # (y: the state's error through sums of 16 terms, and its rounding)
    e = (out[0].double() - y[-1]).abs() - (y[-1].abs() * 2.0 ** -8 if io == "bf16" else 0.0)
    assert float(e.max() / y[-1].pow(2).mean().sqrt()) <= 4 * STATE


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("vary", [True, False])
@pytest.mark.parametrize("bsz,L,H,P,N", [(1, 60000, 2, 16, 16), (256, 20000, 2, 64, 64), (2, 60000, 4, 64, 128)])
def test_prompts(io, vary, bsz, L, H, P, N):
    """Sequences in many segments, in one (there are as many heads as that takes), and with 128 states."""
    c = Slow(bsz, L, H, P, N, io, 5e-5, vary, seed=2)
    y, want = c.definition(bsz - 1)
    got, last, _ = ssmscan.ssd_conv_fwd(*c.args(), dstate=N)
    close(last[-1], want, STATE, "last_state")
    if io == "f32":
        close(got[-1], y, 4 * STATE, "y")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_then_tokens(io):
    """A sequence goes from the one to the other at any token: the state after 20,000 tokens of each."""
    L = 40000
    c = Slow(1, L, 2, 16, 16, io, 5e-5, True, seed=3)
    _, want = c.definition(0)
    x, w, cb, raw, A, D, bias = c.args(slice(0, L // 2))
    _, st, cs = ssmscan.ssd_conv_fwd(x.contiguous(), w, cb, raw.contiguous(), A, D, bias, dstate=16)
    for t in range(L // 2, L):
        x, w, cb, raw, A, D, bias = c.args(t)
        ssmscan.ssd_conv_step(st, cs, x, w, cb, raw, A, D, bias, dstate=16)
    close(st[0], want, STATE, "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_states_that_are_not_finite(io):
    """An infinite or NaN state stays so, beside states that keep their values, in heads that forget slowly, fast, and
    not at all; tokens one by one and as a prompt."""
    H, P, N = 4, 8, 16
    c = Slow(2, 3, H, P, N, io, 0.5, True, seed=5)
    c.A = torch.tensor([-1e-4, -0.5, -4.0, 0.0], device="cuda")
    st = torch.randn(2, H, P, N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    clean = st.clone()
    st[0, :, 2, 3], st[1, :, 5, 7], st[1, :, 0, 0] = float("inf"), -float("inf"), float("nan")
    bad = ~torch.isfinite(st)
    first = st.clone()

    def steps(s):
        cs = torch.zeros(2, 3, c.x.shape[2], dtype=IO[io], device="cuda")
        for t in range(3):
            x, w, cb, raw, A, D, bias = c.args(t)
            ssmscan.ssd_conv_step(s, cs, x, w, cb, raw, A, D, bias, dstate=N)
        return s
    one, without = steps(st), steps(clean.clone())
    assert torch.equal(torch.isnan(one), torch.isnan(first)) and torch.equal(one[torch.isinf(first)], first[torch.isinf(first)])
    assert torch.equal(one[~bad], without[~bad])
    last = ssmscan.ssd_conv_fwd(*c.args(), dstate=N, initial_state=first)[1]
    assert torch.equal(torch.isnan(last), torch.isnan(first)) and torch.equal(last[torch.isinf(first)], first[torch.isinf(first)])
