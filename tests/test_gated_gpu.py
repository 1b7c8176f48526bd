"""The gated linear recurrence on the GPU (ssm_gated_scan_fwd / _bwd, ssm_gated_step) against the fp64
oracle on the same inputs.

Tolerances, relative to the rms of the reference and before the final rounding to bf16: a token adds at
most three fp32 roundings (decay, input, sum) of 2^-24 of a state of at most ~4 rms, so L <= 1000 tokens
give sqrt(L) * 3 * 4 * 6e-8 = 2.3e-5 as a random walk; four times that, 1e-4, is the bound, for outputs
and for the gradients (two such walks and a few products).  A sequence of `long` tokens has states with a
memory of at most 1 / (1 - a) ~ 2000 tokens, hence the same bound times sqrt(2)."""
import numpy as np
import pytest

from selective_state_space_32_amd import inputs
from gpu_util import raw_error, to_dev, to_host_f64, y_error

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import gated  # noqa: E402
from selective_state_space_32_amd import ssmscan  # noqa: E402

TOL = 1e-4
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    """Seeded inputs: device tensors in `t`, the exact values the device holds in fp64 in `v`."""

    def __init__(self, bsz, L, D, io, seed, gate=True, state=True, lens=None, spread=1.0):
        rng = np.random.default_rng(seed)
        self.io, self.shape = io, (bsz, L, D)
        self.t, self.v = {}, {}
        for k in ("x", "r", "g", "dy") + (("z",) if gate else ()):
            self._add(k, rng.standard_normal((bsz, L, D), dtype=np.float32) * (spread if k in ("r", "g") else 1.0), io)
        self._add("A", np.log(rng.uniform(0.9, 0.999, D)).astype(np.float32), "f32")
        if state:
            self._add("h0", rng.standard_normal((bsz, D), dtype=np.float32), "f32")
            self._add("dlast", rng.standard_normal((bsz, D), dtype=np.float32), "f32")
        self.lens = lens
        self.t["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")

    def _add(self, k, a, io):
        a = np.asarray(a, np.float32)
        if io == "bf16":
            bits = inputs.bf16_bits(a)
            self.t[k], self.v[k] = to_dev(bits, torch), inputs.bf16_to_f32(bits).astype(np.float64)
        else:
            self.t[k], self.v[k] = to_dev(a, torch), a.astype(np.float64)

    def fwd_args(self):
        g = self.t.get
        return (g("x"), g("r"), g("g"), g("A"), g("z")), dict(initial_state=g("h0"), seq_lens=g("lens"))

    def reference(self):
        g = self.v.get
        a = (g("x"), g("r"), g("g"), g("A"), g("z"), g("h0"), self.lens)
        y, last = gated.scan(*a)
        return y, last, gated.grads(g("dy"), *a, g("dlast"))


def run_fwd(c, **kw):
    a, k = c.fwd_args()
    out = ssmscan.gated_scan_fwd(*a, **k, **kw)
    torch.cuda.synchronize()
    return out


def run_bwd(c, checkpoints=None):
    a, k = c.fwd_args()
    grads = ssmscan.gated_scan_bwd(c.t["dy"], *a, **k, dlast_state=c.t.get("dlast"),
                                   want_initial_state_grad=True, checkpoints=checkpoints)
    torch.cuda.synchronize()
    return grads


def close(got, ref, io, tol, label):
    got = to_host_f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), label
    if not ref.size:
        return
    e = y_error(got, ref, io) if np.any(ref) else float(np.abs(got).max())
    print(f"{label}: err/rms {e:.2e} (tol {tol:.1e})", flush=True)
    assert e <= tol, (label, e)


def check(c, tol=TOL, label=""):
    print(f"[{label}] {c.shape} {c.io}", flush=True)
    y, last, ck = run_fwd(c, save_checkpoints=True)
    ry, rlast, rg = c.reference()
    close(y, ry, c.io, tol, "y")
    close(last, rlast, "f32", tol, "last_state")
    one, two = run_bwd(c, ck), run_bwd(c)
    assert set(one) == set(rg)
    for k, ref in rg.items():
        close(one[k], ref, "f32" if k in ("dA", "dinitial_state") else c.io, tol, k)
        assert torch.equal(one[k], two[k]), f"{k}: other values without the forward's states"


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 71])          # vector and element-wise access
@pytest.mark.parametrize("L", LENGTHS)
def test_lengths(io, D, L):
    check(Case(2, L, D, io, seed=1000 + L + D), label=f"L{L} D{D}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 8, 66, 127, 128, 129, 130, 256, 260, 520])
def test_widths(io, D):
    check(Case(3, 150, D, io, seed=1100 + D), label=f"D{D}")


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("lens", [None, [200, 0, 77]])
def test_options(gate, state, lens):
    for io in ("f32", "bf16"):
        check(Case(3, 200, 96, io, seed=1200, gate=gate, state=state, lens=lens),
              label=f"gate={gate} state={state} lens={lens}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 130, 700])
def test_ragged(io, L):
    """Lengths from none to all tokens, below zero and above L (clamped), at and around whole chunks."""
    lens = [0, 1, L, L + 5, -3, L // 2, min(64, L), min(65, L), max(L - 1, 0), min(128, L), min(129, L)]
    check(Case(len(lens), L, 40, io, seed=1300 + L, lens=lens), label=f"L{L}")


def test_many_chunks_one_sequence():
    """One sequence of 1000 tokens in few channels: every chunk waits for the one before it."""
    for io in ("f32", "bf16"):
        check(Case(1, 1000, 24, io, seed=1400), label="one sequence")


def test_many_sequences():
    check(Case(37, 190, 130, "bf16", seed=1410), label="37 sequences")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_gates(io):
    """Gates far out on both sides (|r|, |g| up to ~80): decays of exactly 1 (beta = 0) and inputs of
    exactly 0; the gradients stay finite."""
    check(Case(2, 150, 64, io, seed=1500, spread=20.0), label="strong gates")


def test_no_decay_channels():
    """A = 0: the state never changes, beta is 0 and the gradients that divide by it are defined as 0."""
    c = Case(2, 150, 64, "f32", seed=1510)
    c.t["A"][::2] = 0.0
    c.v["A"][::2] = 0.0
    check(c, label="A = 0")
    y, last = run_fwd(c)
    assert torch.equal(last[:, ::2], c.t["h0"][:, ::2])


def test_fast_decay_channels():
    """A down to -200: the state forgets within a token and products of decays underflow to 0."""
    c = Case(2, 300, 64, "f32", seed=1520)
    A = -np.exp(np.linspace(-8, np.log(200.0), 64)).astype(np.float32)
    c._add("A", A, "f32")
    check(c, label="A to -200")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_padding_is_not_read(io):
    """NaN and infinities past the lengths reach nothing; the outputs there are zero."""
    lens = [130, 0, 64, 1]
    c = Case(4, 200, 72, io, seed=1600, lens=lens)
    ry, rlast, rg = c.reference()
    for b, n in enumerate(lens):
        for k in ("x", "r", "g", "z", "dy"):
            c.t[k][b, n:] = float("nan") if k != "r" else float("inf")
    y, last, ck = run_fwd(c, save_checkpoints=True)
    close(y, ry, io, TOL, "y")
    close(last, rlast, "f32", TOL, "last")
    grads = run_bwd(c, ck)
    for k, ref in rg.items():
        close(grads[k], ref, "f32" if k in ("dA", "dinitial_state") else io, TOL, k)
        if ref.ndim == 3:
            for b, n in enumerate(lens):
                assert not to_host_f64(grads[k])[b, n:].any(), k
    for b, n in enumerate(lens):
        assert not to_host_f64(y)[b, n:].any()
        if n == 0:
            assert torch.equal(last[b], c.t["h0"][b]) and torch.equal(grads["dinitial_state"][b], c.t["dlast"][b])


def test_nan_stays_in_its_channel():
    """A NaN input spoils its own channel of its own sequence from its token on, and nothing else."""
    c = Case(2, 300, 64, "f32", seed=1610)
    ref = run_fwd(c)[0].clone()
    c.t["x"][1, 137, 5] = float("nan")
    y = run_fwd(c)[0]
    bad = torch.isnan(y)
    assert bad[1, 137:, 5].all() and int(bad.sum()) == 300 - 137
    assert torch.equal(y[~bad], ref[~bad])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned_tensors(io):
    """Tensors that start one element into their storage take element-wise access; same results."""
    c = Case(2, 140, 64, io, seed=1700)
    y, last, ck = run_fwd(c, save_checkpoints=True)
    grads = run_bwd(c, ck)
    for k in ("x", "r", "g", "z", "dy"):
        buf = torch.empty(c.t[k].numel() + 1, dtype=c.t[k].dtype, device="cuda")[1:]
        c.t[k] = buf.view(c.shape).copy_(c.t[k])
    y2, last2, ck2 = run_fwd(c, save_checkpoints=True)
    assert raw_error(to_host_f64(y2), to_host_f64(y)) <= (1e-5 if io == "f32" else 1e-2)
    check(c, label="one element in")
    assert torch.allclose(run_bwd(c, ck2)["dA"], grads["dA"], rtol=1e-4, atol=1e-4)


def test_state_in_place_and_pieces():
    """A sequence in pieces, each from the state the last one left in the same buffer."""
    c = Case(3, 333, 130, "f32", seed=1800)
    y, last = run_fwd(c)
    (x, r, g, A, z), k = c.fwd_args()
    st = k["initial_state"].clone()
    out, at = [], 0
    for n in (1, 64, 0, 200, 68):
        cut = [v[:, at:at + n].contiguous() for v in (x, r, g, z)]
        out.append(ssmscan.gated_scan_fwd(*cut[:3], A, cut[3], initial_state=st, last_state=st)[0])
        at += n
    torch.cuda.synchronize()
    assert at == 333
    assert raw_error(to_host_f64(torch.cat(out, 1)), to_host_f64(y)) <= 2e-5
    assert raw_error(to_host_f64(st), to_host_f64(last)) <= 2e-5


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("S,D", [(1, 1), (1, 2048), (3, 71), (5, 130), (256, 520)])
def test_step(io, gate, S, D):
    """Tokens one by one: each against the oracle, and the states against the scan's."""
    c = Case(S, 5, D, io, seed=1900 + S + D, gate=gate)
    ry, rlast, _ = c.reference()
    st = c.t["h0"].clone()
    for t in range(5):
        cut = [None if c.t.get(k) is None else c.t[k][:, t].contiguous() for k in ("x", "r", "g", "z")]
        y = ssmscan.gated_step(st, *cut[:3], c.t["A"], cut[3])
        torch.cuda.synchronize()
        close(y, ry[:, t], io, 1e-5, f"token {t}")
    close(st, rlast, "f32", 1e-5, "state")
    _, last = run_fwd(c)
    assert raw_error(to_host_f64(st), to_host_f64(last)) <= 1e-5


def test_step_unaligned():
    c = Case(4, 1, 64, "bf16", seed=1950)
    ry, rlast, _ = c.reference()
    put = lambda v: torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")[1:].view(v.shape).copy_(v)
    st = put(c.t["h0"])
    y = ssmscan.gated_step(st, *(put(c.t[k][:, 0]) for k in ("x", "r", "g")), put(c.t["A"]), put(c.t["z"][:, 0]))
    torch.cuda.synchronize()
    close(y, ry[:, 0], "bf16", 1e-5, "y")
    close(st, rlast, "f32", 1e-5, "state")


def test_step_call_repeats():
    """The marshalled call advances the same state token by token, like gated_step."""
    c = Case(3, 1, 130, "bf16", seed=1960)
    cut = [c.t[k][:, 0].contiguous() for k in ("x", "r", "g", "z")]
    a, b = c.t["h0"].clone(), c.t["h0"].clone()
    y = torch.empty_like(cut[0])
    call = ssmscan.gated_step_call(a, *cut[:3], c.t["A"], cut[3], y=y)
    for _ in range(4):
        call()
        y2 = ssmscan.gated_step(b, *cut[:3], c.t["A"], cut[3])
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(y, y2)


def test_same_from_run_to_run():
    """No result depends on the order in which workgroups run: several calls are bitwise equal."""
    c = Case(4, 900, 300, "bf16", seed=2000, lens=[900, 5, 450, 899])
    y, last, ck = run_fwd(c, save_checkpoints=True)
    grads = run_bwd(c, ck)
    for _ in range(4):
        y2, last2, ck2 = run_fwd(c, save_checkpoints=True)
        again = run_bwd(c, ck2)
        assert torch.equal(y, y2) and torch.equal(last, last2)
        assert all(torch.equal(grads[k], again[k]) for k in grads)


def test_workspace_contents_do_not_matter():
    c = Case(2, 700, 130, "f32", seed=2010)
    y, last, ck = run_fwd(c, save_checkpoints=True)
    grads = run_bwd(c, ck)
    a, k = c.fwd_args()
    ws = ssmscan.gated_scan_fwd(*a, **k, save_checkpoints=True)[2]
    d = ssmscan.make_dims(2, 700, 130, 1, torch.float32)
    import ctypes
    need = int(ssmscan.lib.ssm_gated_scan_bwd_workspace_bytes(ctypes.byref(d)))
    for fill in (0, 0xFF, 0x3F, 0xBF, 0x80):
        ws.fill_(fill)
        y2, last2, ck2 = run_fwd(c, workspace=ws, save_checkpoints=True)
        assert torch.equal(y, y2) and torch.equal(last, last2), fill
        wb = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        g2 = ssmscan.gated_scan_bwd(c.t["dy"], *a, **k, dlast_state=c.t["dlast"], want_initial_state_grad=True,
                                    checkpoints=ck2, workspace=wb)
        torch.cuda.synchronize()
        assert all(torch.equal(grads[n], g2[n]) for n in grads), fill


def test_another_stream():
    """The work goes to the stream given, or to the current one."""
    c = Case(2, 500, 256, "bf16", seed=2020)
    y, last = run_fwd(c)
    a, k = c.fwd_args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2 = torch.empty_like(y)
    ssmscan.gated_scan_fwd(*a, **k, y=y2, stream=s)
    with torch.cuda.stream(s):
        y3, last3 = ssmscan.gated_scan_fwd(*a, **k)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3) and torch.equal(last, last3)


def test_workspace_of_another_stream_is_kept():
    """A call on a stream of the caller's: the workspace it allocated is not handed out again while that
    stream may still use it (nothing is allocated on the caller's stream between the calls)."""
    c = Case(8, 2000, 512, "bf16", seed=2025)
    a, k = c.fwd_args()
    y, last = run_fwd(c)
    s = torch.cuda.Stream()
    outs = [torch.empty_like(y) for _ in range(6)]
    torch.cuda.synchronize()
    for o in outs:
        ssmscan.gated_scan_fwd(*a, **k, y=o, stream=s, return_last_state=False)
        torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(0x3F)   # what the allocator hands out next
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)


def test_graph_replays():
    """Forward and backward captured in a graph: every replay gives the eager results."""
    c = Case(2, 600, 256, "bf16", seed=2030)
    y, last, ck = run_fwd(c, save_checkpoints=True)
    grads = {k: v.clone() for k, v in run_bwd(c, ck).items()}
    a, k = c.fwd_args()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, last2, ck2 = ssmscan.gated_scan_fwd(*a, **k, save_checkpoints=True)
        g2 = ssmscan.gated_scan_bwd(c.t["dy"], *a, **k, dlast_state=c.t["dlast"], want_initial_state_grad=True,
                                    checkpoints=ck2)
    for _ in range(4):
        y2.zero_()
        last2.zero_()
        for v in g2.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(last, last2)
        assert all(torch.equal(grads[n], g2[n]) for n in grads)
        run_fwd(c)


def test_empty():
    for bsz, L, D in ((0, 5, 8), (2, 0, 8), (2, 5, 0)):
        z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
        x, A = z(bsz, L, D), z(D) - 1.0
        h0 = torch.ones((bsz, D), device="cuda")
        y, last, ck = ssmscan.gated_scan_fwd(x, x, x, A, x, initial_state=h0, save_checkpoints=True)
        g = ssmscan.gated_scan_bwd(x, x, x, x, A, x, initial_state=h0, dlast_state=h0, want_initial_state_grad=True,
                                   checkpoints=ck)
        torch.cuda.synchronize()
        assert y.shape == x.shape and not torch.count_nonzero(g["dA"])
        if L == 0:
            assert torch.equal(last, h0) and torch.equal(g["dinitial_state"], h0)
    ssmscan.gated_step(z(0, 8), z(0, 8), z(0, 8), z(0, 8), z(8))


def test_long_sequence():
    """A long sequence in few channels, against the oracle's last tokens."""
    c = Case(1, 20000, 6, "bf16", seed=2100, gate=False, state=False)
    y, last = run_fwd(c)
    ry, rlast = gated.scan(*(c.v[k] for k in ("x", "r", "g", "A")))
    close(y, ry, "bf16", TOL * 1.5, "y")
    close(last, rlast, "f32", TOL * 1.5, "last")


def test_offsets_beyond_32_bits():
    """More than 2^31 elements per tensor: the last sequence's values equal those of a small batch."""
    bsz, L, D = 2, 66000, 16512
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((bsz, L, D), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    A = torch.full((D,), -0.05, device="cuda")
    y, last = ssmscan.gated_scan_fwd(x, x, x, A)
    ys, lasts = ssmscan.gated_scan_fwd(*[x[1:].contiguous()] * 3, A)
    torch.cuda.synchronize()
    assert torch.equal(y[1:], ys) and torch.equal(last[1:], lasts)
    t = slice(L - 50, L)
    ry, _ = gated.scan(*[to_host_f64(x[1:, -20000:, -4:])] * 3, to_host_f64(A[-4:]))
    close(y[1:, t, -4:], ry[:, -50:], "bf16", TOL * 1.5, "the last channels' last tokens")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradient_against_differences_of_the_kernel(io):
    """The directional derivative of the kernel's own loss along its gradient: for fp32 within the
    differences' error (step 1e-2 of inputs of size one: third-order terms 1e-4 and fp32 rounding 1e-5 of
    the loss's change), for bf16 with the loss summed in fp64 (output rounding 2^-9 over 1e4 outputs)."""
    c = Case(2, 100, 50, "f32", seed=2200)
    grads = run_bwd(c)
    w, wl = c.v["dy"], c.v["dlast"]

    def loss():
        y, last = run_fwd(c)
        return float((to_host_f64(y) * w).sum() + (to_host_f64(last) * wl).sum())
    if io == "bf16":   # the same gradients from the bf16 kernel on rounded inputs
        b = Case(2, 100, 50, "bf16", seed=2200)
        gb = run_bwd(b)
        for k in grads:
            assert raw_error(to_host_f64(gb[k]), to_host_f64(grads[k])) <= 0.2, k
        return
    for k, name in (("x", "dx"), ("r", "dr"), ("g", "dg"), ("z", "dz"), ("A", "dA"), ("h0", "dinitial_state")):
        keep, d = c.t[k].clone(), grads[name].float()
        u = d / d.abs().max() * (1e-2 if k != "A" else 1e-4)
        v = []
        for sign in (1.0, -1.0):
            c.t[k] = keep + sign * u
            v.append(loss())
        c.t[k] = keep
        want = 2.0 * float((to_host_f64(d) * to_host_f64(u)).sum())
        assert abs((v[0] - v[1]) - want) <= 5e-3 * abs(want), (k, v[0] - v[1], want)
