"""The layer norm on the GPU (ssm_layernorm_fwd / _bwd) against the fp64 oracle on the same inputs.

Tolerances, relative to the rms of the reference and before the final rounding to bf16: a row's sum of D
values runs through at most ~140 successive fp32 additions for D <= 8192, an error below 140 * 6e-8 =
8.4e-6 of the values' size; y and ds carry two such sums: 2e-5.  The parameters' gradients add M <= 5000
random terms, each sum within sqrt(M) * 6e-8 of the terms' size times a few: 5e-5 of their rms."""
import numpy as np
import pytest

from selective_state_space_32_amd import inputs
from gpu_util import raw_error, to_dev, to_host_f64, y_error

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import layernorm  # noqa: E402
from selective_state_space_32_amd import ssmscan  # noqa: E402

TOL, TOL_W = 2e-5, 5e-5


def tensor(rng, shape, io, scale=1.0, offset=0.0):
    """A device tensor and the exact values it holds."""
    a = (rng.standard_normal(shape, dtype=np.float32) * scale + offset).astype(np.float32)
    if io == "bf16":
        a = inputs.bf16_bits(a)
        return to_dev(a, torch), inputs.bf16_to_f32(a).astype(np.float64)
    return to_dev(a, torch), a.astype(np.float64)


def close(got, ref, io, tol, label):
    got = to_host_f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), label
    if ref.size and np.any(ref):
        e = y_error(got, ref, io)
        print(f"{label}: err/rms {e:.2e} (tol {tol:.1e})", flush=True)
        assert e <= tol, (label, e)
    else:
        assert not np.any(got), label


def check(M, D, io, res, seed, bias=True, offset=0.25, tol=TOL, dres=True):
    print(f"[M{M} D{D} {io} residual={res}]", flush=True)
    rng = np.random.default_rng(seed)
    kept = {"none": io, "same": io, "f32": "f32"}[res]
    x, vx = tensor(rng, (M, D), io, offset=offset)
    w, vw = tensor(rng, D, "f32", 0.1, 1.0)
    b, vb = tensor(rng, D, "f32", 0.1) if bias else (None, None)
    r, vr = tensor(rng, (M, D), kept, 2.0) if res != "none" else (None, None)
    y, total, mean, rstd = ssmscan.layernorm_fwd(x, w, b, residual=r)
    torch.cuda.synchronize()
    if r is None:
        assert total is x
        s = vx
    else:
        # one fp32 sum, rounded once to the kept type: bitwise what it has to be
        assert torch.equal(total, (x.float() + r.float()).to(total.dtype))
        s = to_host_f64(total)     # what is kept is what is normalised
    ry, rm, rr = layernorm.forward(s, vw, vb)
    close(y, ry, io, tol, "y")
    close(mean, rm, "f32", tol, "mean")
    close(rstd, rr, "f32", tol, "rstd")
    dy, vdy = tensor(rng, (M, D), io)
    dr, vdr = tensor(rng, (M, D), kept) if dres else (None, None)
    g = ssmscan.layernorm_bwd(dy, total, w, mean, rstd, dresidual=dr)
    torch.cuda.synchronize()
    ref = layernorm.grads(vdy, s, vw, to_host_f64(mean), to_host_f64(rstd), vdr)
    close(g["ds"], ref["ds"], kept, tol, "ds")
    assert ("dx" in g) == (kept != io)
    if "dx" in g:
        assert torch.equal(g["dx"], g["ds"].to(g["dx"].dtype))
    close(g["dweight"], ref["dweight"], "f32", max(TOL_W, tol), "dweight")
    close(g["dbias"], ref["dbias"], "f32", max(TOL_W, tol), "dbias")
    return x, w, b, r, y, total, mean, rstd, dy, dr, g


KINDS = [("f32", "none"), ("f32", "same"), ("bf16", "none"), ("bf16", "same"), ("bf16", "f32")]


@pytest.mark.parametrize("io,res", KINDS)
@pytest.mark.parametrize("D", [2, 3, 8, 63, 64, 65, 127, 256, 500, 512, 513, 1000, 1024, 1536, 2048, 2049, 4096, 5120,
                               8192])
def test_widths(io, res, D):
    check(13, D, io, res, seed=3000 + D)


@pytest.mark.parametrize("io,res", KINDS)
@pytest.mark.parametrize("D", [8193, 10240, 16384, 20001])
def test_wide_rows(io, res, D):
    check(3, D, io, res, seed=3100 + D, tol=2 * TOL)


@pytest.mark.parametrize("io,res", KINDS)
@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 255, 256, 257, 1025, 4999])
def test_rows(io, res, M):
    check(M, 96, io, res, seed=3200 + M)


@pytest.mark.parametrize("io,res", KINDS)
def test_options(io, res):
    check(70, 640, io, res, seed=3300, bias=False, dres=False)
    check(70, 641, io, res, seed=3301, bias=False, dres=True)


def test_many_rows_wide():
    check(4096, 1536, "f32", "none", seed=3310)
    check(1500, 5120, "bf16", "f32", seed=3311)


@pytest.mark.parametrize("io,res", KINDS)
@pytest.mark.parametrize("M,D", [(4999, 200), (2500, 1290), (2500, 1500), (600, 8200), (300, 20001)])
def test_many_rows_per_sum(io, res, M, D):
    """More rows than workgroups, in every split of the sums over rows."""
    check(M, D, io, res, seed=3320 + D, tol=2 * TOL if D > 8192 else TOL)


def test_large_mean():
    """Rows around 1000 with deviations of one: the variance is taken from centred values.  The mean
    itself is good to a few ulps of 1000 (6e-5), which shifts y by as much."""
    rng = np.random.default_rng(3400)
    x, vx = tensor(rng, (9, 3000), "f32", 1.0, 1000.0)
    w, vw = tensor(rng, 3000, "f32", 0.1, 1.0)
    y, _, mean, rstd = ssmscan.layernorm_fwd(x, w)
    torch.cuda.synchronize()
    ry, rm, rr = layernorm.forward(vx, vw)
    close(y, ry, "f32", 1e-3, "y")
    close(rstd, rr, "f32", 1e-5, "rstd")


def test_constant_rows():
    """No deviation: y is the bias, whatever the constant; one column likewise."""
    w, b = torch.randn(100, device="cuda"), torch.randn(100, device="cuda")
    x = torch.tensor([0.0, 1.0, -3.5, 1e30, 1e-30], device="cuda")[:, None].expand(5, 100).contiguous()
    y, _, mean, rstd = ssmscan.layernorm_fwd(x[:3].contiguous(), w, b)
    torch.cuda.synchronize()
    assert torch.allclose(y, b.expand(3, 100), atol=1e-3) and torch.allclose(rstd, torch.full_like(rstd, 1e5 ** 0.5))
    y, _, mean, rstd = ssmscan.layernorm_fwd(torch.randn((6, 1), device="cuda"), w[:1].clone(), b[:1].clone())
    torch.cuda.synchronize()
    assert torch.equal(y, b[:1].expand(6, 1))


def test_bad_rows_stay_alone():
    """A row with NaN or infinity is NaN; the rows beside it are untouched."""
    x, w, b, r, y, total, mean, rstd, dy, dr, g = check(40, 320, "bf16", "f32", seed=3500)
    x2 = x.clone()
    x2[7, 3], x2[20, 5], x2[39, 0] = float("nan"), float("inf"), float("-inf")
    y2, total2, mean2, rstd2 = ssmscan.layernorm_fwd(x2, w, b, residual=r)
    g2 = ssmscan.layernorm_bwd(dy, total2, w, mean2, rstd2, dresidual=dr)
    torch.cuda.synchronize()
    bad = [7, 20, 39]
    ok = [k for k in range(40) if k not in bad]
    assert torch.equal(y2[ok], y[ok]) and torch.equal(g2["ds"][ok], g["ds"][ok])
    assert torch.isnan(y2[bad]).all() and torch.isnan(g2["ds"][bad]).all()


@pytest.mark.parametrize("io,res", KINDS)
def test_unaligned(io, res):
    """Tensors one element into their storage: the same values."""
    x, w, b, r, y, total, mean, rstd, dy, dr, g = check(33, 512, io, res, seed=3600)
    put = lambda v: None if v is None else torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")[1:].view(
        v.shape).copy_(v)
    y2, total2, mean2, rstd2 = ssmscan.layernorm_fwd(put(x), put(w), put(b), residual=put(r))
    g2 = ssmscan.layernorm_bwd(put(dy), put(total), put(w), put(mean), put(rstd), dresidual=put(dr))
    torch.cuda.synchronize()
    assert raw_error(to_host_f64(y2), to_host_f64(y)) <= (1e-5 if io == "f32" else 2e-2)
    assert raw_error(to_host_f64(g2["ds"]), to_host_f64(g["ds"])) <= (1e-5 if g["ds"].dtype == torch.float32 else 2e-2)
    assert raw_error(to_host_f64(g2["dweight"]), to_host_f64(g["dweight"])) <= TOL_W
    assert raw_error(to_host_f64(g2["dbias"]), to_host_f64(g["dbias"])) <= TOL_W


@pytest.mark.parametrize("D", [512, 513, 12000])
def test_in_place(D):
    """The residual stream updated in place, forwards and backwards."""
    x, w, b, r, y, total, mean, rstd, dy, dr, g = check(21, D, "bf16", "f32", seed=3700, tol=2 * TOL)
    y2, t2, _, _ = ssmscan.layernorm_fwd(x, w, b, residual=r, total=r)
    g2 = ssmscan.layernorm_bwd(dy, total, w, mean, rstd, dresidual=dr, ds=dr)
    torch.cuda.synchronize()
    assert t2 is r and torch.equal(y2, y) and torch.equal(r, total)
    assert g2["ds"] is dr and torch.equal(dr, g["ds"]) and torch.equal(g2["dx"], g["dx"])


def test_widened_sum():
    """sum_f32 without a residual: the start of an fp32 residual stream."""
    rng = np.random.default_rng(3800)
    x, vx = tensor(rng, (17, 320), "bf16")
    w, vw = tensor(rng, 320, "f32", 0.1, 1.0)
    y, total, mean, rstd = ssmscan.layernorm_fwd(x, w, sum_f32=True)
    torch.cuda.synchronize()
    assert total.dtype == torch.float32 and torch.equal(total, x.float())
    close(y, layernorm.forward(vx, vw)[0], "bf16", TOL, "y")


def test_same_from_run_to_run():
    x, w, b, r, y, total, mean, rstd, dy, dr, g = check(3001, 520, "bf16", "f32", seed=3900)
    for _ in range(3):
        y2 = ssmscan.layernorm_fwd(x, w, b, residual=r)[0]
        g2 = ssmscan.layernorm_bwd(dy, total, w, mean, rstd, dresidual=dr)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)


def test_without_parameter_gradients():
    x, w, b, r, y, total, mean, rstd, dy, dr, g = check(30, 200, "f32", "same", seed=3910)
    g2 = ssmscan.layernorm_bwd(dy, total, w, mean, rstd, dresidual=dr, want_param_grads=False)
    torch.cuda.synchronize()
    assert set(g2) == {"ds"} and torch.equal(g2["ds"], g["ds"])


def test_leading_shape_and_empty():
    w = torch.ones(8, device="cuda")
    x = torch.randn((2, 3, 8), device="cuda")
    y, total, mean, rstd = ssmscan.layernorm_fwd(x, w)
    assert y.shape == x.shape and mean.shape == (2, 3)
    for M, D in ((0, 8), (5, 0)):
        x, w = torch.empty((M, D), device="cuda"), torch.ones(D, device="cuda")
        y, total, mean, rstd = ssmscan.layernorm_fwd(x, w)
        g = ssmscan.layernorm_bwd(x, total, w, mean, rstd)
        torch.cuda.synchronize()
        assert g["dweight"].shape == (D,) and not torch.count_nonzero(g["dweight"]) and not torch.count_nonzero(
            g["dbias"])


def test_graph_replays():
    x, w, b, r, y, total, mean, rstd, dy, dr, g = check(500, 640, "bf16", "f32", seed=3920)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, t2, m2, r2 = ssmscan.layernorm_fwd(x, w, b, residual=r)
        g2 = ssmscan.layernorm_bwd(dy, t2, w, m2, r2, dresidual=dr)
    for _ in range(4):
        for v in (y2, t2, m2, r2, *g2.values()):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(t2, total) and all(torch.equal(g[k], g2[k]) for k in g)
        ssmscan.layernorm_fwd(x, w, b, residual=r)


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows equal those of a call of their own."""
    M, D = 420000, 5120
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    w = torch.ones(D, device="cuda")
    y, total, mean, rstd = ssmscan.layernorm_fwd(x, w)
    ys, _, ms, rs = ssmscan.layernorm_fwd(x[-64:].contiguous(), w)
    g = ssmscan.layernorm_bwd(x, total, w, mean, rstd, want_param_grads=False)
    gs = ssmscan.layernorm_bwd(x[-64:].contiguous(), x[-64:].contiguous(), w, ms, rs, want_param_grads=False)
    torch.cuda.synchronize()
    assert torch.equal(y[-64:], ys) and torch.equal(mean[-64:], ms) and torch.equal(g["ds"][-64:], gs["ds"])


def test_gradient_against_differences_of_the_kernel():
    """The kernel's loss changes along its gradient as the gradient says (step 1e-2, fp32)."""
    rng = np.random.default_rng(3950)
    s, _ = tensor(rng, (20, 300), "f32", 2.0)
    w, _ = tensor(rng, 300, "f32", 0.1, 1.0)
    b, _ = tensor(rng, 300, "f32", 0.1)
    dy, vdy = tensor(rng, (20, 300), "f32")
    _, total, mean, rstd = ssmscan.layernorm_fwd(s, w, b)
    g = ssmscan.layernorm_bwd(dy, total, w, mean, rstd)
    for k, name in ((0, "ds"), (1, "dweight"), (2, "dbias")):
        args = [s, w, b]
        d = g[name]
        u = d / d.abs().max() * 1e-2
        v = []
        for sign in (1.0, -1.0):
            args[k] = (s, w, b)[k] + sign * u
            y = ssmscan.layernorm_fwd(*args)[0]
            torch.cuda.synchronize()
            v.append(float((to_host_f64(y) * vdy).sum()))
        want = 2.0 * float((to_host_f64(d) * to_host_f64(u)).sum())
        assert abs((v[0] - v[1]) - want) <= 5e-3 * abs(want), (name, v[0] - v[1], want)
