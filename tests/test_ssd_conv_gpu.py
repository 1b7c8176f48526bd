"""The state space dual layer with its convolution on the GPU (ssm_ssd_conv_fwd / _bwd / _step) against the fp64
oracle on the same inputs; the tolerances are derived in ssd_conv_cases.py."""
import ctypes

import numpy as np
import pytest

from gpu_util import to_host_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_32_amd import inputs, ssmscan  # noqa: E402
from ssd_conv_cases import BF, F32, Case, check, check_bwd, check_fwd, close, run_bwd, run_fwd  # noqa: E402

IOS = ["f32", "bf16"]


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("L", [1, 2, 3, 4, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200])
def test_lengths(io, L):
    check(Case(2, L, 2, 64, 1, 64, io, seed=100 + L), label=f"L{L}")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("H,P,G,N", [(1, 8, 1, 8), (2, 16, 1, 16), (3, 24, 3, 24), (4, 40, 2, 72), (2, 64, 1, 96), (6, 32, 2, 128),
                                     (4, 64, 4, 128), (2, 72, 1, 64), (2, 128, 2, 40), (1, 192, 1, 128), (5, 8, 1, 128)])
def test_heads_and_states(io, H, P, G, N):
    check(Case(2, 90, H, P, G, N, io, seed=200 + H + P + N), label=f"H{H} P{P} G{G} N{N}")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("state", [True, False])
def test_widths_of_the_convolution(io, W, state):
    check(Case(2, 70, 2, 32, 1, 32, io, seed=300 + W, W=W, state=state), label=f"W{W} state={state}")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("L", [2, 130, 300])
def test_ragged(io, L):
    """Lengths from none to all tokens, below zero and above L (clamped), at and around whole chunks."""
    lens = [0, 1, L, L + 5, -3, L // 2, min(64, L), min(65, L), max(L - 1, 0), min(128, L), min(129, L)]
    check(Case(len(lens), L, 2, 16, 1, 24, io, seed=400 + L, lens=lens), label=f"L{L}")


@pytest.mark.parametrize("io", IOS)
def test_without_softplus(io):
    check(Case(2, 150, 2, 64, 1, 64, io, seed=500, softplus=False), label="dt as it is")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("extra", [0, 1, 3])
def test_strides_and_alignment(io, extra):
    """Parts of wider rows whose rows start at any element; packed rows give the same bits."""
    c = Case(2, 100, 3, 24, 1, 24, io, seed=600 + extra, extra=extra)
    check(c, label=f"rows of {c.t['proj'].shape[-1]}")
    p = Case(2, 100, 3, 24, 1, 24, io, seed=600 + extra, extra=extra, parts=False)
    for a, b in zip(run_fwd(c), run_fwd(p)):
        assert torch.equal(a, b)
    one, two = run_bwd(c), run_bwd(p)
    assert all(torch.equal(one[k], two[k]) for k in one)


@pytest.mark.parametrize("io", IOS)
def test_without_options(io):
    """No bias, no skip, no history, no gradients beyond the inputs'."""
    c = Case(2, 80, 2, 32, 1, 32, io, seed=650, state=False)
    for k in ("conv_b", "D", "dt_bias"):
        c.t[k] = c.v[k] = None
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    lay = c.oracle()
    ry, rl, _ = lay.scan()
    tol = BF if io == "bf16" else F32
    close(y, ry, io, tol, "y")
    close(last, rl, "f32", F32, "last")
    g = ssmscan.ssd_conv_bwd(c.t["dy"], *c.layer(), **c.shape(), checkpoints=ck)
    ref, _ = lay.grads(c.v["dy"])
    assert set(g) == {"dxbc", "ddt", "dconv_w", "dA"}
    close(g["dxbc"], ref["dxbc"], io, tol, "dxbc")
    close(g["ddt"], ref["ddt"], io, tol, "ddt")
    y2, none1, none2 = ssmscan.ssd_conv_fwd(*c.layer(), **c.shape(), return_states=False)
    assert none1 is None and none2 is None and torch.equal(y, y2)


@pytest.mark.parametrize("io", IOS)
def test_padding_is_not_read(io):
    """NaN and infinities past the lengths reach nothing; the outputs there are zero."""
    lens = [130, 0, 64, 1]
    c = Case(4, 200, 2, 24, 1, 24, io, seed=700, lens=lens)
    lay = c.oracle()
    ry, rlast, rrows = lay.scan()
    rg, scale = lay.grads(c.v["dy"], c.v["dlast"])
    y0, l0, _, ck0 = run_fwd(c, save_checkpoints=True)
    g0 = run_bwd(c, ck0)
    for b, n in enumerate(lens):
        c.t["proj"][b, n:] = float("nan")
        c.t["proj"][b, n:, ::3] = float("inf")
        c.t["dy"][b, n:] = float("nan")
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    assert torch.equal(y, y0) and torch.equal(last, l0) and np.array_equal(to_host_f64(rows), rrows)
    close(y, ry, io, BF if io == "bf16" else F32, "y")
    g = run_bwd(c, ck)
    for k in g:
        assert torch.equal(g[k], g0[k]), k
    for b, n in enumerate(lens):
        assert not to_host_f64(y)[b, n:].any() and not to_host_f64(g["dxbc"])[b, n:].any() and not to_host_f64(g["ddt"])[b, n:].any()
        if n == 0:
            assert torch.equal(last[b], c.t["h0"][b]) and torch.equal(g["dinitial_state"][b], c.t["dlast"][b])


def test_nan_stays_near():
    """A NaN input spoils its own sequence from the start of its chunk of 64 on, and nothing else."""
    c = Case(2, 300, 2, 32, 1, 32, "f32", seed=710)
    ref = run_fwd(c)[0].clone()
    c.t["xbc"][1, 150, 5] = float("nan")
    y = run_fwd(c)[0]
    bad = torch.isnan(y)
    assert bad[1, 150, 0, 5] and not bad[0].any() and not bad[1, :128].any() and not bad[1, :, 1].any()
    assert torch.equal(y[~bad], ref[~bad])


@pytest.mark.parametrize("io", IOS)
def test_strong_and_weak_decays(io):
    """A from 0 (the state only adds up) to -2000 (it forgets within a token), step sizes up to ~50."""
    c = Case(2, 200, 4, 16, 1, 16, io, seed=720)
    c._add("A", np.array([0.0, -1e-4, -30.0, -2000.0]), "f32")
    c._add("dt_bias", np.array([0.0, 3.0, 0.0, 50.0]), "f32")
    # (A = 0 at a step size of about 0.7: states of 200 tokens add up, no decay weights their errors down: the
    # walk of F32 has no less memory)
    check(c, label="A from 0 to -2000")


@pytest.mark.parametrize("scale", [1e-6, 1e4])
def test_scales(scale):
    """Inputs and gradients far from one: nothing is held in a type of narrow exponents."""
    check(Case(2, 100, 2, 64, 1, 64, "bf16", seed=730, scale=scale, state=False), label=f"scale {scale}")


@pytest.mark.parametrize("io", IOS)
def test_u_is_the_exact_values_rounding(io):
    """The convolution's output, which every path of the layer starts from: with bf16 the rounding of the exact
    value at every element, with fp32 within 2^-21 of its rms and half that of itself."""
    c = Case(2, 257, 40, 64, 1, 64, io, seed=740, state=False)
    _, _, _, ck = run_fwd(c, save_checkpoints=True)
    n, es = c.t["xbc"].numel(), c.t["xbc"].element_size()
    u = to_host_f64(ck[:n * es].view(c.t["xbc"].dtype)).reshape(c.v["xbc"].shape)
    lay = c.oracle()
    if io == "bf16":
        assert np.array_equal(u, lay.u)
    else:
        assert np.max(np.abs(u - lay.u) / (np.abs(lay.u) * 2.0 ** -21 + 2.0 ** -21)) <= 1.0


def test_u_at_extremes():
    """Pre-activations far out on both sides, infinite and NaN: silu's limits."""
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 60.0, -60.0, -90.0, -200.0, 3e38, float("inf"), float("nan"), 1e-38, 88.0, -88.0, -64.1, 64.1],
                     dtype=torch.bfloat16, device="cuda")
    H, P, N = 2, 8, 8
    x = torch.zeros(1, 1, H * P + 2 * N, dtype=torch.bfloat16, device="cuda")
    x[..., :16] = v
    w = torch.ones(x.shape[-1], 1, device="cuda")
    dt = torch.zeros(1, 1, H, dtype=torch.bfloat16, device="cuda")
    ck = ssmscan.ssd_conv_fwd(x, w, None, dt, -torch.ones(H, device="cuda"), dstate=N, save_checkpoints=True)[3]
    u = ck[:32 * 2].view(torch.bfloat16)[:16].double().cpu()
    want = torch.nn.functional.silu(v.double().cpu()).float().bfloat16().double()
    assert torch.equal(u.isnan(), want.isnan()) and torch.equal(u[~u.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("io", IOS)
def test_state_in_place_and_pieces(io):
    """A sequence in pieces, each from the states the last one left in the same buffers, equals one call."""
    c = Case(3, 333, 2, 40, 1, 24, io, seed=800)
    y, last, rows = run_fwd(c)
    st, cs = c.t["h0"].clone(), c.t["conv_state"].clone()
    out, at = [], 0
    for n in (64, 128, 0, 1, 2, 100, 38):
        a = c.layer()
        cut = (a[0][:, at:at + n].contiguous(),) + a[1:3] + (a[3][:, at:at + n].contiguous(),) + a[4:]
        out.append(ssmscan.ssd_conv_fwd(*cut, **c.shape(), conv_state=cs, initial_state=st, last_state=st, conv_state_out=cs)[0])
        at += n
    torch.cuda.synchronize()
    assert at == 333
    got = torch.cat(out, 1)
    assert torch.equal(cs, rows)
    close(got, to_host_f64(y), io, 2 * BF if io == "bf16" else F32, "pieces")
    close(st, to_host_f64(last), "f32", F32, "state")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("S,H,P,G,N,W", [(1, 2, 64, 1, 64, 4), (3, 4, 40, 2, 24, 4), (2, 3, 8, 1, 8, 2), (5, 2, 128, 1, 128, 3), (2, 2, 24, 1, 96, 1),
                                          (300, 2, 16, 2, 16, 4)])
def test_step(io, S, H, P, G, N, W):
    """Tokens one by one against the oracle, after a prompt, from its states; the states equal the scan's."""
    c = Case(S, 12, H, P, G, N, io, seed=900 + S + N, W=W)
    ry, rlast, rrows = c.oracle().scan()
    a = c.layer()
    first = (a[0][:, :7],) + a[1:3] + (a[3][:, :7],) + a[4:]
    if not all(v.stride(0) == v.shape[1] * v.stride(1) for v in (first[0], first[3])):
        first = (first[0].contiguous(),) + a[1:3] + (first[3].contiguous(),) + a[4:]
    y, st, cs = ssmscan.ssd_conv_fwd(*first, **c.shape(), conv_state=c.t["conv_state"], initial_state=c.t["h0"])
    tol = BF if io == "bf16" else F32
    close(y, ry[:, :7], io, tol, "prompt")
    for t in range(7, 12):
        y = ssmscan.ssd_conv_step(st, cs if W > 1 else None, a[0][:, t], *a[1:3], a[3][:, t], *a[4:], **c.shape())
        torch.cuda.synchronize()
        close(y, ry[:, t], io, F32, f"token {t}")
    close(st, rlast, "f32", F32, "state")
    assert np.array_equal(to_host_f64(cs), rrows)


def test_step_call_repeats():
    c = Case(3, 1, 4, 32, 2, 32, "bf16", seed=950)
    a = c.layer()
    args = (a[0][:, 0], *a[1:3], a[3][:, 0], *a[4:])
    s1, s2, c1, c2 = (c.t[k].clone() for k in ("h0", "h0", "conv_state", "conv_state"))
    y = torch.empty(3, 4, 32, dtype=torch.bfloat16, device="cuda")
    call = ssmscan.ssd_conv_step_call(s1, c1, *args, **c.shape(), y=y)
    for _ in range(5):
        call()
        y2 = ssmscan.ssd_conv_step(s2, c2, *args, **c.shape())
        torch.cuda.synchronize()
        assert torch.equal(s1, s2) and torch.equal(c1, c2) and torch.equal(y, y2)


@pytest.mark.parametrize("io", IOS)
def test_same_from_run_to_run(io):
    c = Case(3, 700, 6, 64, 2, 64, io, seed=1000, lens=[700, 5, 450])
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    g = run_bwd(c, ck)
    for _ in range(3):
        y2, last2, rows2, ck2 = run_fwd(c, save_checkpoints=True)
        g2 = run_bwd(c, ck2)
        assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(rows, rows2)
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_workspace_contents_do_not_matter():
    c = Case(2, 300, 4, 40, 2, 72, "bf16", seed=1010)
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    g = run_bwd(c, ck)
    for fill in (0, 0xFF, 0x3F, 0x80):
        ws = torch.full_like(ck, fill)
        y2, last2, _, ck2 = run_fwd(c, workspace=ws, save_checkpoints=True)
        assert torch.equal(y, y2) and torch.equal(last, last2), fill
        bsz, L, H, P, G, N = c.dims
        for kept in (ck2, None):
            d = ssmscan.ssm_ssd_conv_dims(bsz, L, H, P, G, N, 0, 0, 1, 4)
            need = int(ssmscan.lib.ssm_ssd_conv_bwd_workspace_bytes(ctypes.byref(d), 4 if kept is not None else 0))
            g2 = run_bwd(c, kept, workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
            assert all(torch.equal(g[k], g2[k]) for k in g), fill


def test_another_stream():
    """The work goes to the stream given, or to the current one; what a call allocated for another stream is kept
    while that stream may use it."""
    c = Case(4, 900, 8, 64, 1, 64, "bf16", seed=1020)
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    g = run_bwd(c, ck)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        y2, last2, _, ck2 = ssmscan.ssd_conv_fwd(*c.layer(), **c.shape(), **c.start(), save_checkpoints=True, stream=s)
        g2 = ssmscan.ssd_conv_bwd(c.t["dy"], *c.layer(), **c.shape(), **c.start(), dlast_state=c.t["dlast"],
                                  want_initial_state_grad=True, checkpoints=ck2, stream=s)
        outs.append((y2, last2, g2))
        torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(0x3F)   # what the allocator hands out next
    with torch.cuda.stream(s):
        y3 = ssmscan.ssd_conv_fwd(*c.layer(), **c.shape(), **c.start())[0]
    torch.cuda.synchronize()
    assert torch.equal(y, y3)
    for y2, last2, g2 in outs:
        assert torch.equal(y, y2) and torch.equal(last, last2) and all(torch.equal(g[k], g2[k]) for k in g2)


def test_graph_replays():
    """Forward, backward and steps captured in a graph: every replay gives the eager results."""
    c = Case(2, 200, 4, 64, 2, 64, "bf16", seed=1030)
    a = c.layer()
    tok = (a[0][:, 0], *a[1:3], a[3][:, 0], *a[4:])
    y, last, rows, ck = run_fwd(c, save_checkpoints=True)
    g = {k: v.clone() for k, v in run_bwd(c, ck).items()}
    st, cs = last.clone(), rows.clone()
    ys = [ssmscan.ssd_conv_step(st, cs, *tok, **c.shape()) for _ in range(3)]
    torch.cuda.synchronize()
    s2, c2 = torch.empty_like(last), torch.empty_like(rows)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, last2, rows2, ck2 = ssmscan.ssd_conv_fwd(*a, **c.shape(), **c.start(), save_checkpoints=True)
        g2 = ssmscan.ssd_conv_bwd(c.t["dy"], *a, **c.shape(), **c.start(), dlast_state=c.t["dlast"], want_initial_state_grad=True,
                                  checkpoints=ck2)
        s2.copy_(last2)
        c2.copy_(rows2)
        yt = [ssmscan.ssd_conv_step(s2, c2, *tok, **c.shape()) for _ in range(3)]
    for _ in range(4):
        for v in (y2, last2, rows2, *g2.values(), *yt):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(last, last2) and torch.equal(rows, rows2)
        assert all(torch.equal(g[k], g2[k]) for k in g2)
        assert torch.equal(st, s2) and torch.equal(cs, c2) and all(torch.equal(p, q) for p, q in zip(ys, yt))
        run_fwd(c)


def test_empty():
    f = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
    for bsz, L in ((0, 5), (2, 0)):
        H, P, N = 2, 8, 8
        row = H * P + 2 * N
        h0 = torch.ones(bsz, H, P, N, device="cuda")
        cs = torch.ones(bsz, 3, row, device="cuda")
        args = (f(bsz, L, row), f(row, 4), f(row), f(bsz, L, H), f(H) - 1.0, f(H), f(H))
        y, last, rows, ck = ssmscan.ssd_conv_fwd(*args, dstate=N, conv_state=cs, initial_state=h0, save_checkpoints=True)
        g = ssmscan.ssd_conv_bwd(y, *args, dstate=N, conv_state=cs, initial_state=h0, dlast_state=h0,
                                 want_initial_state_grad=True, checkpoints=ck)
        torch.cuda.synchronize()
        assert y.shape == (bsz, L, H, P) and torch.equal(last, h0) and torch.equal(rows, cs)
        assert torch.equal(g["dinitial_state"], h0) and not torch.count_nonzero(g["dconv_state"])
        for k in ("dA", "dD", "ddt_bias", "dconv_w", "dconv_b"):
            assert not torch.count_nonzero(g[k]), k
    ssmscan.ssd_conv_step(f(0, 2, 8, 8), f(0, 3, 32), f(0, 32), f(32, 4), None, f(0, 2), f(2), dstate=8)


@pytest.mark.parametrize("io", IOS)
def test_long_sequence(io):
    check_fwd(Case(1, 9000, 2, 16, 1, 16, io, seed=1100), label="9000 tokens")


def test_gradient_against_differences_of_the_kernel():
    """The directional derivative of the kernel's own loss along its gradient, fp32: the differences' third-order
    terms (steps of 1e-2, relative 1e-4 of the change) and fp32 rounding of the loss's change (1e-5): 5e-3."""
    c = Case(2, 100, 2, 24, 1, 24, "f32", seed=1200, parts=False)
    g = run_bwd(c)
    w, wl = c.v["dy"], c.v["dlast"]

    def loss():
        y, last, _ = run_fwd(c)
        return float((to_host_f64(y) * w).sum() + (to_host_f64(last) * wl).sum())
    for k, name in (("xbc", "dxbc"), ("dt", "ddt"), ("conv_w", "dconv_w"), ("conv_b", "dconv_b"), ("A", "dA"), ("D", "dD"),
                    ("dt_bias", "ddt_bias"), ("h0", "dinitial_state"), ("conv_state", "dconv_state")):
        keep, d = c.t[k].clone(), g[name].float()
        u = d / d.abs().max() * 1e-2
        v = []
        for sign in (1.0, -1.0):
            c.t[k] = keep + sign * u
            v.append(loss())
        c.t[k] = keep
        want = 2.0 * float((to_host_f64(d) * to_host_f64(u)).sum())
        assert abs((v[0] - v[1]) - want) <= 5e-3 * abs(want), (k, v[0] - v[1], want)


def test_many_sequences_and_heads():
    check(Case(9, 70, 24, 16, 4, 16, "bf16", seed=1300), label="216 heads")


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in a row tensor: the last sequence's values equal those of a batch of its own."""
    bsz, L, H, P, N = 2, 66000, 256, 64, 64
    row = H * P + 2 * N
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((bsz, L, row), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dt = torch.empty((bsz, L, H), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.full((row, 4), 0.4, device="cuda")
    A, bias = torch.full((H,), -1.0, device="cuda"), torch.full((H,), -3.0, device="cuda")
    y, last, rows = ssmscan.ssd_conv_fwd(x, w, None, dt, A, None, bias, dstate=N)
    ys, lasts, rowss = ssmscan.ssd_conv_fwd(x[1:], w, None, dt[1:], A, None, bias, dstate=N)
    torch.cuda.synchronize()
    assert torch.equal(y[1:], ys) and torch.equal(last[1:], lasts) and torch.equal(rows[1:], rowss)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("S,H,P,G,N", [(1, 1, 1000, 1, 8), (1, 2, 264, 2, 128), (1050, 2, 40, 1, 64), (1, 3, 72, 1, 104)])
def test_step_in_parts(io, S, H, P, G, N):
    """A head's channels in several workgroups, with a last part of few or none, and in turns of one workgroup."""
    c = Case(S, 2, H, P, G, N, io, seed=1400 + P)
    ry, rlast, rrows = c.oracle().scan()
    a, st, cs = c.layer(), c.t["h0"].clone(), c.t["conv_state"].clone()
    for t in range(2):
        y = ssmscan.ssd_conv_step(st, cs, a[0][:, t], *a[1:3], a[3][:, t], *a[4:], **c.shape())
        torch.cuda.synchronize()
        close(y, ry[:, t], io, F32, f"token {t}")
    close(st, rlast, "f32", F32, "state")
    assert np.array_equal(to_host_f64(cs), rrows)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("H,P,G,N", [(4, 192, 2, 128), (2, 200, 1, 72), (3, 128, 1, 64), (1, 320, 1, 8)])
def test_heads_of_several_tiles(io, H, P, G, N):
    """What the backward adds up over a head's tiles of 64 channels, over more than one chunk."""
    check(Case(2, 150, H, P, G, N, io, seed=1500 + P, lens=[150, 97]), label=f"{P} channels")


def test_two_streams_at_once():
    """Calls in flight together, each with a workspace of its own, give what they give alone."""
    cases = [Case(2, 700, 6, 64, 2, 64, "bf16", seed=1600 + i) for i in range(2)]
    alone = [run_fwd(c) + tuple(run_bwd(c).values()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        out = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                fwd = ssmscan.ssd_conv_fwd(*c.layer(), **c.shape(), **c.start())
                g = ssmscan.ssd_conv_bwd(c.t["dy"], *c.layer(), **c.shape(), **c.start(), dlast_state=c.t.get("dlast"),
                                         want_initial_state_grad=True, want_conv_state_grad=True)
                out.append(tuple(fwd) + tuple(g.values()))
        torch.cuda.synchronize()
        for got, ref in zip(out, alone):
            assert all(torch.equal(x, y) for x, y in zip(got, ref))
