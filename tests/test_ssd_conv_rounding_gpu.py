"""bf16 outputs of the state space dual layer with its convolution: fp32's error, rounded once.

An output that is off by e before its rounding comes out one step of 2^-8 (up to 2^-7) of itself away from the rounding of
the exact value where a border between two bf16 values lies within e: the difference has a mean square of 2 |e| times the
mean step, which for values of all sizes around their rms is about 3e-3 of it.  Held like fp32 an output is cut or
rounded 13 times (two halves of the states' products and two of the pairs' in three parts each, and the decay between them),
each by 2^-24 / sqrt(3) in the mean square of sums of up to three rms: |e| is 4e-7 of the rms at most in the mean, and the
root of the mean square of the difference 5e-5.  Operands in two bf16 parts would be off by 2^-17, eight times that."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_32_amd import ssmscan  # noqa: E402
from test_ssd_conv_slow_gpu import Slow  # noqa: E402

DIFFERENCE = 5e-5


@pytest.mark.parametrize("bsz,L,H,P,N", [(1, 4096, 8, 64, 64), (64, 1024, 8, 64, 64), (1, 4096, 8, 64, 128), (64, 1024, 8, 64, 128),
                                         (2, 3001, 5, 40, 24), (1, 2000, 3, 128, 96)])
@pytest.mark.parametrize("per_token", [0.002, 0.05])
def test_outputs_are_rounded_once(bsz, L, H, P, N, per_token):
    c = Slow(bsz, L, H, P, N, "bf16", per_token, True, seed=11)
    y = ssmscan.ssd_conv_fwd(*c.args(), dstate=N)[0]
    for b in {0, bsz - 1}:
        want = c.definition(b)[0]
        once = want.float().to(torch.bfloat16).double()
        e = float((y[b].double() - once).pow(2).mean().sqrt() / want.pow(2).mean().sqrt())
        print(f"({bsz}, {L}, {H}, {P}, {N}) sequence {b}: {e:.2e} from the rounding of the exact values", flush=True)
        assert e <= DIFFERENCE
