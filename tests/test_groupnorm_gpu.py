"""The group norm with its activation on the GPU (ssm_groupnorm_fwd / _bwd) against the fp64 oracle.

Tolerances, relative to the rms of the reference and before the final rounding to bf16: a value passes some ten
fp32 roundings of 2^-24 and two sums over a group, whose partial sums of D terms add at most (log2 D + 20) / 2 more
to terms of at most ~5 rms: 25 * 5 * 6e-8 = 7.5e-6, twice that is the bound, 1.5e-5.  Sums over rows are held against
the root of the sum of squares of their terms (random walks of at most 4096 rows: the same bound).  dv is what is
left of dn rstd when its parts along n (and 1) are taken off: with one value and no centring, or two and centring, only
eps rstd^2 (1e-5) of it, while the roundings are those of the terms.  So dx and the dz of a gate before are held against
the larger of their own rms and that first term's."""
import numpy as np
import pytest

from gpu_util import rms, to_dev, to_host_f64, y_error

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import groupnorm  # noqa: E402
from selective_state_space_32_amd import inputs, ssmscan  # noqa: E402

TOL = 1.5e-5
EPS = 1e-5
GATES = ["none", "before", "after", "silu"]


class Case:
    def __init__(self, rows, dim, groups, io, gate, centre, seed, bias=True, offset=0.25, part=True, extra=9):
        rng = np.random.default_rng(seed)
        n = lambda *s: rng.standard_normal(s, dtype=np.float32)
        self.groups, self.io, self.gate, self.centre = groups, io, gate, centre
        self.t, self.v = {}, {}
        self._add("x", n(rows, dim) + np.float32(offset), io)
        self._add("dy", n(rows, dim), io)
        self._add("w", 1.0 + 0.1 * n(dim), "f32")
        if bias:
            self._add("b", 0.1 * n(dim), "f32")
        if gate in ("before", "after"):
            self._add("wide", n(rows, dim + extra), io)
            self.t["z"], self.v["z"] = self.t["wide"][:, 5:5 + dim], self.v["wide"][:, 5:5 + dim]
            if not part:
                self.t["z"] = self.t["z"].contiguous()

    def _add(self, k, a, io):
        a = np.asarray(a, np.float32)
        if io == "bf16":
            bits = inputs.bf16_bits(a)
            self.t[k], self.v[k] = to_dev(bits, torch), inputs.bf16_to_f32(bits).astype(np.float64)
        else:
            self.t[k], self.v[k] = to_dev(a, torch), a.astype(np.float64)

    def kw(self):
        return dict(groups=self.groups, z=self.t.get("z"), gate_first=self.gate == "before", silu=self.gate == "silu")

    def fwd(self, **kw):
        out = ssmscan.groupnorm_fwd(self.t["x"], self.t["w"], self.t.get("b"), EPS, centre=self.centre, **self.kw(), **kw)
        torch.cuda.synchronize()
        return out

    def bwd(self, mean, rstd, **kw):
        g = ssmscan.groupnorm_bwd(self.t["dy"], self.t["x"], self.t["w"], self.t.get("b"), mean, rstd, **self.kw(), **kw)
        torch.cuda.synchronize()
        return g

    def reference(self):
        a = (self.v["x"], self.v["w"], self.v.get("b"), self.groups, EPS, self.v.get("z"), self.gate, self.centre)
        return groupnorm.norm(*a), groupnorm.grads(self.v["dy"], *a)


def close(got, ref, io, label, tol=TOL):
    got = to_host_f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), label
    if ref.size:
        e = y_error(got, ref, io)
        print(f"{label}: err/rms {e:.2e} (tol {tol:.1e})", flush=True)
        assert e <= tol, (label, e)


def check(c, tol=TOL):
    print(f"{tuple(c.t['x'].shape)} groups {c.groups} {c.io} {c.gate} centre={c.centre}", flush=True)
    y, mean, rstd = c.fwd()
    (ry, rm, rr), (rg, scale) = c.reference()
    close(y, ry, c.io, "y", tol)
    close(rstd, rr, "f32", "rstd", tol)
    assert (mean is None) == (not c.centre)
    if c.centre:
        assert np.max(np.abs(to_host_f64(mean) - rm)) <= tol * (1.0 + np.max(np.abs(rm)))
    g = c.bwd(mean, rstd)
    assert set(g) == set(rg) - (set() if "b" in c.t else {"dbias"})
    for k in g:
        if k in scale and scale[k].ndim == 1:
            e = np.max(np.abs(to_host_f64(g[k]) - rg[k]) / (scale[k] + 1e-30))
            assert e <= tol, (k, e)
        else:
            more = max(1.0, rms(scale[k]) / rms(rg[k])) if k in scale and np.any(rg[k]) else 1.0
            close(g[k], rg[k], c.io, k, tol * more)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("centre", [True, False])
def test_modes(io, gate, centre):
    for dim, groups in ((96, 3), (640, 1), (2560, 2)):
        check(Case(70, dim, groups, io, gate, centre, seed=dim, bias=centre))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 7, 31, 32, 33, 64, 65, 127, 128, 129, 256, 257, 511, 513, 768, 769, 1023, 1024, 1025, 2048, 2049, 4099,
                               5120, 5121, 8192, 8193, 12000])
def test_group_widths(io, D):
    """Around every change of the lanes that hold a group, and odd widths, whose rows start anywhere."""
    for groups in (1, 3):
        check(Case(9, D * groups, groups, io, "before", True, seed=D + groups))
        check(Case(9, D * groups, groups, io, "after", False, seed=D + groups + 1))


@pytest.mark.parametrize("groups", [1, 2, 5, 15, 16, 17, 24, 31, 64, 100])
def test_group_counts(groups):
    """Groups that fill a workgroup's slots, leave some without one, and several workgroups across a row."""
    for D in (16, 64, 200):
        check(Case(33, D * groups, groups, "bf16", "before", False, seed=groups + D))


@pytest.mark.parametrize("rows", [1, 2, 3, 500, 4096])
def test_rows(rows):
    check(Case(rows, 192, 3, "f32", "after", True, seed=rows))
    check(Case(rows, 1536, 1, "bf16", "before", False, seed=rows + 1))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strides_and_alignment(io):
    """z as a part of wider rows and packed: the same bits."""
    a, b = (Case(40, 320, 5, io, "before", True, seed=3, part=p) for p in (True, False))
    ya, yb = a.fwd(), b.fwd()
    assert all(torch.equal(p, q) for p, q in zip(ya, yb))
    ga, gb = a.bwd(*ya[1:]), b.bwd(*yb[1:])
    assert all(torch.equal(ga[k], gb[k]) for k in ga)


def test_large_means():
    """Groups far from zero that vary little: x = 1900 + noise of fp32; the mean of 200 terms rounds, rstd is about 1 and
    x - mean carries the roundings of x alone."""
    c = Case(50, 500, 1, "f32", "none", True, seed=5, offset=1900.0)
    y, mean, rstd = c.fwd()
    ry, rm, rr = c.reference()[0]
    # n = (x - mean) rstd: the mean is right to 2^-24 of 1900 (1.1e-4) at worst, of n about 1
    assert y_error(to_host_f64(y), ry, "f32") <= 2.5e-4
    assert np.max(np.abs(to_host_f64(rstd) / rr - 1)) <= TOL


def test_constant_groups():
    """A group of one value has no variance: y is the bias, rstd 1 / sqrt(eps); groups of zeros likewise."""
    for value in (0.0, 3.0, -1900.5):
        x = torch.full((5, 300), value, device="cuda")
        w, b = torch.randn(300, device="cuda"), torch.randn(300, device="cuda")
        y, mean, rstd = ssmscan.groupnorm_fwd(x, w, b, EPS, groups=3)
        torch.cuda.synchronize()
        assert torch.equal(y, b.expand(5, 300)) and torch.all(mean == value)
        assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=1e-6)


def test_nan_stays_in_its_group():
    c = Case(8, 96, 3, "f32", "before", True, seed=6)
    ref = c.fwd()[0].clone()
    c.t["x"][2, 40] = float("nan")
    c.t["x"][5, 90] = float("inf")
    y = c.fwd()[0]
    bad = torch.isnan(y)
    assert bad[2, 32:64].all() and bad[5, 64:].all() and int(bad.sum()) == 64
    assert torch.equal(y[~bad], ref[~bad])


def test_extreme_gates():
    """Gates of +-200: silu's limits, no overflow in its derivative."""
    c = Case(6, 64, 2, "f32", "after", True, seed=7, part=False)
    z = np.tile(np.array([-200.0, 200.0, -88.0, 88.0], np.float32), 16)
    c._add("z", np.broadcast_to(z, (6, 64)).copy(), "f32")
    check(c)


def test_same_from_run_to_run_and_workspaces():
    c = Case(700, 1280, 20, "bf16", "before", True, seed=8)
    y, mean, rstd = c.fwd()
    g = c.bwd(mean, rstd)
    for fill in (0, 0xFF, 0x3F):
        ws = torch.full((1 << 24,), fill, dtype=torch.uint8, device="cuda")
        again = c.bwd(mean, rstd, workspace=ws)
        assert all(torch.equal(g[k], again[k]) for k in g)
    assert set(c.bwd(mean, rstd, want_param_grads=False)) == {"dx", "dz"}


def test_leading_axes():
    c = Case(24, 96, 3, "bf16", "before", False, seed=9)
    y, _, rstd = c.fwd()
    wide = c.t["wide"].view(2, 3, 4, -1)
    y2, none, r2 = ssmscan.groupnorm_fwd(c.t["x"].view(2, 3, 4, 96), c.t["w"], c.t["b"], EPS, groups=3, centre=False,
                                         z=wide[..., 5:101], gate_first=True)
    torch.cuda.synchronize()
    assert none is None and torch.equal(y2.view(24, 96), y) and torch.equal(r2.view(24, 3), rstd) and r2.shape == (2, 3, 4, 3)


def test_graph_and_stream():
    c = Case(300, 1024, 4, "bf16", "before", False, seed=10)
    y, mean, rstd = c.fwd()
    g = {k: v.clone() for k, v in c.bwd(mean, rstd).items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, _, r2 = ssmscan.groupnorm_fwd(c.t["x"], c.t["w"], c.t["b"], EPS, centre=False, **c.kw())
        g2 = ssmscan.groupnorm_bwd(c.t["dy"], c.t["x"], c.t["w"], c.t["b"], None, r2, **c.kw())
    for _ in range(4):
        for v in (y2, r2, *g2.values()):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(rstd, r2) and all(torch.equal(g[k], g2[k]) for k in g)
        c.fwd()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        y3, _, r3 = ssmscan.groupnorm_fwd(c.t["x"], c.t["w"], c.t["b"], EPS, centre=False, stream=s, **c.kw())
        outs.append((y3, ssmscan.groupnorm_bwd(c.t["dy"], c.t["x"], c.t["w"], c.t["b"], None, r3, stream=s, **c.kw())))
        torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(0x3F)
    torch.cuda.synchronize()
    for y3, g3 in outs:
        assert torch.equal(y, y3) and all(torch.equal(g[k], g3[k]) for k in g)


def test_empty():
    w = torch.ones(64, device="cuda")
    x = torch.zeros(0, 64, device="cuda")
    y, mean, rstd = ssmscan.groupnorm_fwd(x, w, w, groups=4)
    g = ssmscan.groupnorm_bwd(x, x, w, w, mean, rstd, groups=4)
    torch.cuda.synchronize()
    assert y.shape == (0, 64) and rstd.shape == (0, 4)
    assert not torch.count_nonzero(g["dweight"]) and not torch.count_nonzero(g["dbias"])


def test_gradient_against_differences_of_the_kernel():
    for gate in GATES:
        c = Case(6, 96, 3, "f32", gate, True, seed=11, part=False)
        y, mean, rstd = c.fwd()
        g = c.bwd(mean, rstd)
        loss = lambda: float((to_host_f64(c.fwd()[0]) * c.v["dy"]).sum())
        for k, name in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("z", "dz")):
            if k not in c.t:
                continue
            keep, d = c.t[k].clone(), g[name].float()
            u, v = d / d.abs().max() * 1e-2, []
            for sign in (1.0, -1.0):
                c.t[k] = keep + sign * u
                v.append(loss())
            c.t[k] = keep
            want = 2.0 * float((to_host_f64(d) * to_host_f64(u)).sum())
            # third-order terms of steps of 1e-2 (relative 1e-4 each) and fp32 rounding of the change
            assert abs((v[0] - v[1]) - want) <= 5e-3 * abs(want), (gate, k, v[0] - v[1], want)


def test_offsets_beyond_32_bits():
    rows, dim = 300000, 8192
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.ones(dim, device="cuda")
    y, _, rstd = ssmscan.groupnorm_fwd(x, w, groups=8, centre=False, z=x, gate_first=True)
    g = ssmscan.groupnorm_bwd(x, x, w, None, None, rstd, groups=8, z=x, gate_first=True)
    tail = x[-100:]
    y2, _, r2 = ssmscan.groupnorm_fwd(tail, w, groups=8, centre=False, z=tail, gate_first=True)
    g2 = ssmscan.groupnorm_bwd(tail, tail, w, None, None, r2, groups=8, z=tail, gate_first=True)
    torch.cuda.synchronize()
    assert torch.equal(y[-100:], y2) and torch.equal(g["dx"][-100:], g2["dx"]) and torch.equal(g["dz"][-100:], g2["dz"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", GATES)
def test_group_of_one_channel_is_its_mean(io, gate):
    """n = 0 exactly, so y is the bias (under its gate or activation) and x, z (gate first) and the weight get no gradient."""
    c = Case(50, 37, 37, io, gate, True, seed=77, offset=3.0)
    y, mean, rstd = c.fwd()
    g = c.bwd(mean, rstd)
    assert not torch.any(g["dx"]) and not torch.any(g["dweight"])
    if gate == "before":
        assert not torch.any(g["dz"])
        assert torch.equal(y.float(), c.t["b"].to(y.dtype).float().expand(50, 37))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dim,groups", [(640, 1), (5120, 8), (1536, 24), (2500, 1)])
def test_more_rows_than_workgroups(io, gate, dim, groups):
    """Workgroups that take several rows each, of which the last is short."""
    check(Case(3001, dim, groups, io, gate, groups != 8, seed=80 + groups))
