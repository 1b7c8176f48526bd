"""Convolutions of fewer than four taps reach W - 1 rows back and no further: an infinity or NaN before that is not in
their outputs, nor in the gradients."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from ssd_conv_cases import Case, run_bwd, run_fwd  # noqa: E402


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("parts", [True, False])
def test_reach_of_a_bad_row(io, bad, W, parts):
    """A bad value of C in the last row that tokens of the first chunk of 64 alone reach (C is in no state): every token from
    64 on has the bits it has without it, and so have the gradients of their rows and step sizes."""
    bsz, L, H, P, G, N = 2, 200, 2, 16, 1, 16
    c = Case(bsz, L, H, P, G, N, io, seed=40 + W, W=W, parts=parts)
    at = H * P + N + 3
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    g = run_bwd(c, ck)
    c.t["xbc"][1, 64 - W, at] = float(bad)
    y2, last2, rows2, ck2 = run_fwd(c, save_checkpoints=True)
    # (silu(-inf) = -inf * 0 is NaN here as in its definition by a quotient)
    assert not torch.isfinite(y2[1, 64 - W]).all()
    assert torch.equal(y2[0], y[0]) and torch.equal(y2[1, 64:], y[1, 64:])
    assert torch.equal(last2, last) and torch.equal(rows2, rows)
    for g2 in (run_bwd(c, ck2), run_bwd(c)):
        for k in ("dxbc", "ddt"):
            assert torch.equal(g2[k][0], g[k][0]) and torch.equal(g2[k][1, 64:], g[k][1, 64:]), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
def test_reach_of_a_bad_gradient(io, W):
    """A NaN in dy of the first token of a chunk is in that token's gradient of C and in no earlier token's: dxbc has
    it, in C's columns, in the W - 1 rows before, and the rows before those keep their bits."""
    bsz, L, H, P, G, N = 1, 150, 2, 16, 1, 16
    c = Case(bsz, L, H, P, G, N, io, seed=50 + W, W=W)
    cols = slice(H * P + N, H * P + 2 * N)
    ck = run_fwd(c, save_checkpoints=True)[3]
    g = run_bwd(c, ck)["dxbc"]
    c.t["dy"][0, 128, 0, 5] = float("nan")
    for g2 in (run_bwd(c, ck)["dxbc"], run_bwd(c)["dxbc"]):
        assert torch.isnan(g2[0, 129 - W:129, cols]).all()
        assert torch.equal(g2[0, :129 - W, cols], g[0, :129 - W, cols])
