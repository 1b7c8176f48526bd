"""The recurrent block of examples/recurrent_block.py: layer norm, convolution, gated recurrence and their
gradients together, against torch's autograd in fp64 on the CPU; the training loop; decoding; and two
streams at once."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import recurrent_block  # noqa: E402
from selective_state_space_32_amd import ssmscan  # noqa: E402


def reference(p, x, residual, lens):
    """x' and total in fp64 with autograd: the block's formulas, token by token."""
    total = x + residual
    c = total - total.mean(-1, keepdim=True)
    n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * p["norm_w"] + p["norm_b"]
    pre, r, g, z = (n @ p[k] for k in ("Wc", "Wr", "Wg", "Wz"))
    pad = torch.cat([torch.zeros_like(pre[:, :3]), pre], 1)
    u = sum(pad[:, k:k + pre.shape[1]] * p["conv_w"][:, k] for k in range(4)) + p["conv_b"]
    u = u * torch.sigmoid(u)
    log_a = -torch.exp(p["A_log"]) * torch.sigmoid(r)
    a, b = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(g) * u
    h, ys = torch.zeros_like(b[:, 0]), []
    for t in range(x.shape[1]):
        h = a[:, t] * h + b[:, t]
        ys.append(h * z[:, t] * torch.sigmoid(z[:, t]) * (t < lens)[:, None])
    return torch.stack(ys, 1) @ p["Wo"], total


def test_block_gradients_against_autograd():
    """fp32 activations: every gradient within 2e-4 of its rms (the products' fp32 sums over 96 to 300
    terms and the recurrence's walk of 70 tokens: a few times 1e-5)."""
    torch.manual_seed(7)
    block = recurrent_block.RecurrentBlock(48, 72, io=torch.float32, seed=5)
    x, res = torch.randn(3, 70, 48, device="cuda"), torch.randn(3, 70, 48, device="cuda")
    dx, dt = torch.randn(3, 70, 48, device="cuda"), torch.randn(3, 70, 48, device="cuda")
    lens = torch.tensor([70, 0, 33], dtype=torch.int32, device="cuda")
    out, total = block.forward(x, res, seq_lens=lens)
    gx, gr, grads = block.backward(dx, dt)
    torch.cuda.synchronize()
    p = {k: v.double().cpu().requires_grad_() for k, v in block.p.items()}
    xr, rr = x.double().cpu().requires_grad_(), res.double().cpu().requires_grad_()
    ro, rt = reference(p, xr, rr, lens.cpu())
    ((ro * dx.double().cpu()).sum() + (rt * dt.double().cpu()).sum()).backward()
    pairs = {"x'": (out, ro.detach()), "total": (total, rt.detach()), "x": (gx, xr.grad), "residual": (gr, rr.grad)}
    pairs.update({k: (grads[k], p[k].grad) for k in block.NAMES})
    for k, (got, ref) in pairs.items():
        e = float((got.double().cpu() - ref).abs().max() / ref.pow(2).mean().sqrt())
        print(f"{k}: {e:.2e}", flush=True)
        assert e <= 2e-4, (k, e)


def test_training_lowers_the_loss():
    losses, block = recurrent_block.train(steps=60, say=None)
    assert losses[0] > 0.9 and losses[-1] < 0.5 * losses[0], losses[::8]
    # bf16 activations: a few roundings of 2^-9 between the two ways
    assert recurrent_block.decode_difference(block) < 0.1


def test_two_streams_at_once():
    """Scans and gradients of two streams, each with its own workspace, overlap in time and give what they
    give alone."""
    A = -torch.rand(640, device="cuda") * 0.1
    xs = [torch.randn(4, 3000, 640, device="cuda").bfloat16() for _ in range(2)]
    alone = []
    for x in xs:
        y, last, ck = ssmscan.gated_scan_fwd(x, x, x, A, x, save_checkpoints=True)
        alone.append((y, last, ssmscan.gated_scan_bwd(x, x, x, x, A, x, checkpoints=ck)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                y, last, ck = ssmscan.gated_scan_fwd(x, x, x, A, x, save_checkpoints=True)
                got.append((y, last, ssmscan.gated_scan_bwd(x, x, x, x, A, x, checkpoints=ck)))
        torch.cuda.synchronize()
        for (y, last, g), (y2, last2, g2) in zip(alone, got):
            assert torch.equal(y, y2) and torch.equal(last, last2) and all(torch.equal(g[k], g2[k]) for k in g)
