"""The layer norm's row means where they are known exactly: rows of one value, and gradients whose terms are
equal, at widths whose reciprocal is rounded up, down, or not at all."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_32_amd import ssmscan  # noqa: E402
from test_layernorm_gpu import close, tensor  # noqa: E402

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
CONSTANTS = [0.0, 1e-30, 1.9375, -3.5, 100.0, 100.1, 1000.0, 1900.0, -1900.3]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [100, 500, 1000, 1500, 3000, 6000, 8191, 10000, 16383, 20001])
def test_constant_rows_of_any_width(io, D):
    """Widths whose reciprocal rounds either way, and sums that are not exact.  The mean is the constant
    itself: what its first value m lacks is taken from the centred values, which are exact, so that it is
    good to far below half an ulp.  A row's sum runs through at most 140 additions, so m is off by at most
    140 * 6e-8 * 1900 = 1.6e-2 and the correction by 140 * 6e-8 of that, 1.3e-7, which
    rstd = 316 and a weight of up to 1.5 take to 6.4e-5 of y; the variance keeps twice 8.4e-6 of 2.6e-4, 4.4e-9
    beside eps = 1e-5, 2.2e-4 of rstd."""
    rng = np.random.default_rng(3430 + D)
    w, vw = tensor(rng, D, "f32", 0.1, 1.0)
    b, vb = tensor(rng, D, "f32", 0.1)
    x = torch.tensor(CONSTANTS, device="cuda").to(IO[io])[:, None].expand(len(CONSTANTS), D).contiguous()
    y, _, mean, rstd = ssmscan.layernorm_fwd(x, w, b)
    # the same constants as sums of a residual
    half = (x.float() * 0.5).contiguous()
    y2, total, mean2, _ = ssmscan.layernorm_fwd(half.to(IO[io]), w, b, residual=half)
    torch.cuda.synchronize()
    assert torch.equal(mean, x[:, 0].float()) and torch.equal(mean2, total[:, 0])
    assert float((rstd.double() * 1e-5 ** 0.5 - 1.0).abs().max()) <= 2.2e-4
    for got in (y, y2):
        close(got, np.broadcast_to(vb, x.shape), io, 6.5e-5 / np.sqrt(np.mean(vb * vb)), "y")


@pytest.mark.parametrize("io,kept", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("D", [98, 500, 1000, 1498, 3000, 6000, 8190, 10000, 16382, 20002])
def test_gradient_of_equal_terms(io, kept, D):
    """dy w the same in every column and n of alternating ones: every sum is exact, dy w - mean(dy w) is 0 and
    so is mean(dy w n), hence ds is 0 to the bit, whatever the width and rstd."""
    dy = torch.tensor([1.9375, -3.0, 0.65625, 1.3125], device="cuda").to(IO[io])[:, None].expand(4, D).contiguous()
    s = torch.full((4, D), 2.0 ** -8, device="cuda")
    s[:, 1::2] *= -1.0
    rows = torch.full((4,), 2.0 ** 8, device="cuda")
    g = ssmscan.layernorm_bwd(dy, s.to(IO[kept]), torch.full((D,), 1.25, device="cuda"), torch.zeros_like(rows), rows)
    torch.cuda.synchronize()
    assert not torch.count_nonzero(g["ds"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_statistics_of_rows_without_values(io):
    """Rows of width 0: their mean is 0 / 0, so both statistics are NaN, and no row keeps what was there."""
    import ctypes
    mean, rstd = torch.full((9,), 7.0, device="cuda"), torch.full((9,), 7.0, device="cuda")
    dims = ssmscan.ssm_dims(1, 9, 0, 1, 1 if io == "bf16" else 0, 0)

    def call(m, r):
        return ssmscan.lib.ssm_layernorm_fwd(None, None, None, None, 1e-5, 0, None, None, m, r, ctypes.byref(dims),
                                             torch.cuda.current_stream().cuda_stream)
    assert call(mean.data_ptr(), None) == 0 and call(None, None) == 0
    torch.cuda.synchronize()
    assert torch.isnan(mean).all() and torch.equal(rstd, torch.full_like(rstd, 7.0))
    assert call(None, rstd.data_ptr()) == 0
    torch.cuda.synchronize()
    assert torch.isnan(rstd).all()
    x, w = torch.empty((2, 3, 0), dtype=IO[io], device="cuda"), torch.ones(0, device="cuda")
    y, total, m, r = ssmscan.layernorm_fwd(x, w, w, residual=x.clone())
    torch.cuda.synchronize()
    assert y.shape == x.shape and total.shape == x.shape and m.shape == r.shape == (2, 3)
    assert torch.isnan(m).all() and torch.isnan(r).all()
