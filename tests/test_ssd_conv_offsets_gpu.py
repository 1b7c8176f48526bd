"""The backward of the state space dual layer with its convolution where rows, states and gradients hold more than 2^31
elements: the last sequences' gradients equal those of a batch of their own, and the parameters' add up."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_32_amd import ssmscan  # noqa: E402


@pytest.mark.parametrize("kept", [True, False])
def test_backward_beyond_32_bits(kept):
    """3 sequences of 66,000 tokens, 256 heads of 64 channels and 64 states: 3.3e9 elements of rows, 3.2e9 of chunks' states.
    (Two of them run by the same plan: one segment, a group's heads in one part.)"""
    bsz, L, H, P, N = 3, 66000, 256, 64, 64
    row = H * P + 2 * N
    if torch.cuda.mem_get_info()[0] < 180e9:
        pytest.skip("needs 180 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    x, dt, dy = rnd(bsz, L, row), rnd(bsz, L, H), rnd(bsz, L, H, P)
    w = torch.full((row, 4), 0.4, device="cuda")
    A, bias, D = torch.full((H,), -1.0, device="cuda"), torch.full((H,), -3.0, device="cuda"), torch.ones(H, device="cuda")
    cb = torch.zeros(row, device="cuda")

    def grads(s):
        args = (x[s], w, cb, dt[s], A, D, bias)
        ck = ssmscan.ssd_conv_fwd(*args, dstate=N, return_states=False, save_checkpoints=True)[3] if kept else None
        g = ssmscan.ssd_conv_bwd(dy[s], *args, dstate=N, want_initial_state_grad=True, want_conv_state_grad=True, checkpoints=ck)
        torch.cuda.synchronize()
        return g

    whole, two, first = grads(slice(0, 3)), grads(slice(1, 3)), grads(slice(0, 1))
    for k in ("dxbc", "ddt", "dinitial_state", "dconv_state"):
        assert torch.equal(whole[k][1:], two[k]), k
        assert torch.isfinite(whole[k][2, -1].float()).all() and torch.count_nonzero(whole[k][2, -1]), k
    # sums over tokens, in 64 bits of the same terms but for those of B and C (added up over the heads in another order)
    for k in ("dA", "dD", "ddt_bias", "dconv_w", "dconv_b"):
        e = (whole[k].double() - two[k].double() - first[k].double()).abs().max() / whole[k].double().abs().max()
        assert float(e) <= 1e-5, (k, float(e))
