"""A residual recurrent block from the library's operators: trained for a few steps, then run token by
token.

    total  = residual + x                       layernorm_fwd (the residual stream stays fp32)
    n      = layer norm of total
    c      = silu(conv1d(n Wc))                 conv1d, width 4
    h      = gated linear recurrence of c with the gates n Wr, n Wg, times silu(n Wz)
    x'     = h Wo                               the next block's x

The projections are plain matrix products.  Run it on a GPU:  python examples/recurrent_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from selective_state_space_32_amd import ssmscan  # noqa: E402


class RecurrentBlock:
    """Parameters in fp32; activations in `io`.  forward() keeps what backward() needs."""

    NAMES = ("norm_w", "norm_b", "Wc", "Wr", "Wg", "Wz", "Wo", "conv_w", "conv_b", "A_log")

    def __init__(self, width, inner, io=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=gen, device=device) * scale
        self.io = io
        self.p = {"norm_w": torch.ones(width, device=device), "norm_b": torch.zeros(width, device=device),
                  "conv_w": normal(inner, 4, scale=0.5), "conv_b": torch.zeros(inner, device=device)}
        for k in ("Wc", "Wr", "Wg", "Wz"):
            self.p[k] = normal(width, inner, scale=width ** -0.5)
        self.p["Wo"] = normal(inner, width, scale=inner ** -0.5)
        # A = -exp(A_log): decays of 0.9 to 0.999 where the recurrence gate is open
        rate = torch.rand(inner, generator=gen, device=device) * 0.099 + 0.9
        self.p["A_log"] = torch.log(-torch.log(rate))

    def _project(self, n, k):
        return (n.reshape(-1, n.shape[-1]) @ self.p[k].to(self.io)).view(*n.shape[:-1], -1)

    def forward(self, x, residual=None, seq_lens=None):
        """x (batch, L, width) of `io`, residual fp32 or None; returns (x', total)."""
        n, total, mean, rstd = ssmscan.layernorm_fwd(x, self.p["norm_w"], self.p["norm_b"], residual=residual,
                                                     sum_f32=True)
        pre, r, g, z = (self._project(n, k) for k in ("Wc", "Wr", "Wg", "Wz"))
        c, _ = ssmscan.conv1d(pre, self.p["conv_w"], self.p["conv_b"], return_state=False)
        A = -torch.exp(self.p["A_log"])
        y, _, states = ssmscan.gated_scan_fwd(c, r, g, A, z, seq_lens=seq_lens, return_last_state=False,
                                              save_checkpoints=True)
        self.kept = (n, total, mean, rstd, pre, c, r, g, z, A, y, states, seq_lens)
        return self._project(y, "Wo"), total

    def backward(self, dx, dtotal=None):
        """Gradients given those of x' (and of total, fp32): (gradient of x, of residual, dict)."""
        n, total, mean, rstd, pre, c, r, g, z, A, y, states, seq_lens = self.kept
        flat = lambda v: v.reshape(-1, v.shape[-1])
        grads = {"Wo": flat(y).t().float() @ flat(dx).float()}
        dy = (flat(dx) @ self.p["Wo"].to(self.io).t()).view(y.shape)
        s = ssmscan.gated_scan_bwd(dy, c, r, g, A, z, seq_lens=seq_lens, checkpoints=states)
        conv = ssmscan.conv1d_bwd(s["dx"], pre, self.p["conv_w"], self.p["conv_b"])
        grads["conv_w"], grads["conv_b"] = conv["dw"], conv["dbias"]
        grads["A_log"] = s["dA"] * A
        dn = torch.zeros_like(flat(n), dtype=torch.float32)
        for k, d in (("Wc", conv["dx"]), ("Wr", s["dr"]), ("Wg", s["dg"]), ("Wz", s["dz"])):
            grads[k] = flat(n).t().float() @ flat(d).float()
            dn += (flat(d) @ self.p[k].to(self.io).t()).float()
        norm = ssmscan.layernorm_bwd(dn.to(self.io).view(n.shape), total, self.p["norm_w"], mean, rstd, dresidual=dtotal)
        grads["norm_w"], grads["norm_b"] = norm["dweight"], norm["dbias"]
        return norm.get("dx", norm["ds"]), norm["ds"], grads

    def start(self, sequences):
        """The state of `sequences` empty sequences: the convolution's last inputs, the recurrence's."""
        inner, dev = self.p["Wc"].shape[1], self.p["Wc"].device
        return (torch.zeros((sequences, 3, inner), dtype=self.io, device=dev),
                torch.zeros((sequences, inner), device=dev))

    def step(self, x, state, residual=None):
        """One token of every sequence: x (sequences, width); the state is updated in place."""
        conv, h = state
        n, total, _, _ = ssmscan.layernorm_fwd(x, self.p["norm_w"], self.p["norm_b"], residual=residual, sum_f32=True)
        pre, r, g, z = (self._project(n, k) for k in ("Wc", "Wr", "Wg", "Wz"))
        c, _ = ssmscan.conv1d(pre[:, None], self.p["conv_w"], self.p["conv_b"], state=conv, state_out=conv)
        y = ssmscan.gated_step(h, c[:, 0].contiguous(), r, g, -torch.exp(self.p["A_log"]), z)
        return self._project(y, "Wo"), total


def train(steps=60, batch=8, length=192, width=64, inner=128, keep=0.9, rate=3e-2, seed=0, say=print):
    """Learns the running average h_t = keep h_{t-1} + sqrt(1 - keep^2) x_t of its input, with steps
    scaled by the gradients' running sizes; returns the losses and the block."""
    block = RecurrentBlock(width, inner, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    mean = {k: torch.zeros_like(v) for k, v in block.p.items()}
    square = {k: torch.zeros_like(v) for k, v in block.p.items()}
    losses = []
    for k in range(steps):
        x = torch.randn((batch, length, width), generator=gen, device="cuda")
        want, h = torch.empty_like(x), torch.zeros_like(x[:, 0])
        for t in range(length):
            h = keep * h + (1.0 - keep * keep) ** 0.5 * x[:, t]
            want[:, t] = h
        out, _ = block.forward(x.to(block.io))
        diff = out.float() - want
        losses.append(float((diff * diff).mean()))
        _, _, grads = block.backward((diff * (2.0 / (batch * length))).to(block.io))
        for name, g in grads.items():
            mean[name].lerp_(g, 0.1)
            square[name].lerp_(g * g, 0.01)
            size = (square[name] / (1.0 - 0.99 ** (k + 1))).sqrt() + 1e-8
            block.p[name].sub_(rate / (1.0 - 0.9 ** (k + 1)) * mean[name] / size)
        if say and (k % 10 == 0 or k == steps - 1):
            say(f"step {k}: loss {losses[-1]:.4f}", flush=True)
    return losses, block


def decode_difference(block, batch=4, length=40, seed=3):
    """Largest difference of the token-by-token outputs from the whole sequence's, over their rms."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((batch, length, block.p["Wc"].shape[0]), generator=gen, device="cuda").to(block.io)
    out, _ = block.forward(x)
    state = block.start(batch)
    steps = [block.step(x[:, t].contiguous(), state)[0] for t in range(length)]
    out, tokens = out.float(), torch.stack(steps, 1).float()
    return float((tokens - out).abs().max() / out.pow(2).mean().sqrt())


if __name__ == "__main__":
    _, trained = train()
    print(f"token by token against the whole sequence: {decode_difference(trained):.2e} of the rms")
