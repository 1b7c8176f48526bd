"""Decays near 1 on the GPU: an error with a mean, however small, is added up over a slow channel's whole
memory of 1 / (1 - a) tokens, whatever the type of the inputs: the states are fp32."""
import numpy as np
import pytest

from gpu_util import to_host_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import gated  # noqa: E402
from selective_state_space_32_amd import ssmscan  # noqa: E402
from test_gated_gpu import Case, run_bwd, run_fwd  # noqa: E402

IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(1e-5, 1e-4), (1e-4, 2e-3), (2e-3, 2e-2), (2e-2, 0.1), (0.1, 0.4), (0.4, 1.0)])
def test_decays_have_no_bias(io, lo, hi):
    """The step with a state of 1 and no input leaves the decay itself.  Its rounding to fp32 (at most 3e-8, rms
    1.73e-8) averages to 3.4e-11 over 2^18 channels, five times which is allowed; what it is rounded from may be
    off by 5e-7 of 1 - a, as that is all that the state is then off by."""
    n = 1 << 18
    rng = np.random.default_rng(5000)
    A = torch.tensor(-rng.uniform(lo, hi, n), dtype=torch.float32, device="cuda")
    r = torch.tensor(rng.standard_normal((1, n)), device="cuda").to(IO[io])
    zero, state = torch.zeros_like(r), torch.ones((1, n), device="cuda")
    ssmscan.gated_step(state, zero, r, zero, A)
    torch.cuda.synchronize()
    a = np.exp(to_host_f64(A) * gated.sigmoid(to_host_f64(r)))
    mean, bound = float((to_host_f64(state) - a).mean()), 1.7e-10 + 5e-7 * float((1.0 - a).mean())
    print(f"A {-hi}..{-lo}: mean error {mean:.2e} (bound {bound:.1e})", flush=True)
    assert abs(mean) <= bound


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_slow_channels_of_a_long_sequence(io):
    """Channels that remember 1 / (1 - a) of up to 20,000 tokens, over 30,000.  A token rounds its decay and its
    state, 1.7e-8 each in the mean square: sqrt(20000) * 2.5e-8 = 3.5e-6 of a state as a random walk; four times
    that at a state of three times the rms over the channels is 4.2e-5."""
    c = Case(1, 30000, 64, io, seed=5010, gate=False, state=False)
    c._add("A", -np.geomspace(1e-4, 3e-3, 64).astype(np.float32), "f32")
    _, last = run_fwd(c)
    _, want = gated.scan(*(c.v[k] for k in ("x", "r", "g", "A")))
    e = float(np.abs(to_host_f64(last) - want).max() / np.sqrt(np.mean(want * want)))
    print(f"last_state: err/rms {e:.2e}", flush=True)
    assert e <= 4.2e-5


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_slow_channels_of_many_sequences(io):
    """The same where every chunk waits for the one before it (64 chains), forwards and backwards, from a given
    state and end gradient: sqrt(6000) * 2.5e-8 = 1.9e-6, four times that at three times the rms 2.3e-5."""
    c = Case(64, 6000, 64, io, seed=5020, gate=False)
    c._add("A", -np.geomspace(1e-4, 3e-3, 64).astype(np.float32), "f32")
    _, last, ck = run_fwd(c, save_checkpoints=True)
    grads = run_bwd(c, ck)
    x, r, g, dy, A, h, lam = (c.t[k].double() for k in ("x", "r", "g", "dy", "A", "h0", "dlast"))
    u = A * torch.sigmoid(r)
    a, b = torch.exp(u), torch.sqrt(-torch.expm1(2.0 * u)) * torch.sigmoid(g) * x
    for t in range(c.shape[1]):
        h = a[:, t] * h + b[:, t]
        lam = lam + dy[:, -1 - t]
        lam = lam * a[:, -1 - t]
    for k, got, want in (("last_state", last, h), ("dinitial_state", grads["dinitial_state"], lam)):
        e = float((got.double() - want).abs().max() / want.pow(2).mean().sqrt())
        print(f"{k}: err/rms {e:.2e}", flush=True)
        assert e <= 2.3e-5, k
