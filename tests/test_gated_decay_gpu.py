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
