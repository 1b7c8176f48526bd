"""The gated recurrence's schedules, each at sizes that select it: two bf16 channels per lane (more than 256
work items), groups of one (64 chains or more), long groups in one chain, items of two chunks (few chains,
many chunks), rows on and off the memory's lines, every number of queues.  Tolerances as in
test_gated_gpu.py: 1e-4 of the rms for up to 1000 tokens, times sqrt(2) for long sequences, whose states
remember at most ~2000 tokens."""
import numpy as np
import pytest

from gpu_util import raw_error, to_host_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_32_amd import ssmscan  # noqa: E402
from test_gated_gpu import TOL, Case, check, close, run_bwd, run_fwd  # noqa: E402


def lengths(bsz, L, seed):
    """Lengths from none to all tokens, with the ends of chunks and their neighbours among them."""
    rng = np.random.default_rng(seed)
    some = [0, 1, L, L, 63, 64, 65, 127, 128, 129]
    return [int(min(v, L)) for v in some + list(rng.integers(0, L + 1, max(0, bsz - len(some))))][:bsz]


@pytest.mark.parametrize("D", [2, 3, 66, 127, 128, 129, 260])
def test_two_channels_per_lane(D):
    """90 sequences of three chunks: every lane has two channels, the last of an odd width shared."""
    check(Case(90, 130, D, "bf16", seed=4000 + D, gate=D % 2 == 0, lens=lengths(90, 130, D)), label=f"D{D}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
def test_groups_of_one(io, gate):
    """70 chains and more: every chunk waits for the one before it."""
    check(Case(35, 330, 129, io, seed=4100, gate=gate), label="groups of one")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bsz,D", [(1, 40), (2, 70), (3, 100), (5, 64), (9, 30), (11, 20), (17, 33)])
def test_few_chains(io, bsz, D):
    """Every number of queues and group sizes from 64 down, in sequences of 11 chunks."""
    check(Case(bsz, 700, D, io, seed=4200 + bsz), label=f"{bsz} sequences")


def test_long_groups():
    """One chain of 94 chunks: groups of 64, whose maps the waves compose in runs."""
    for io in ("f32", "bf16"):
        check(Case(1, 6001, 24, io, seed=4300), tol=TOL * 1.5, label="one chain")


@pytest.mark.parametrize("io,D", [("bf16", 1024), ("f32", 512)])
def test_items_of_two_chunks(io, D):
    """32 chains of 129 chunks (the last of 8 tokens): the forward takes two chunks per item and leaves the
    states inside its items too.

    dA has a bound of its own here.  A decay near 1 is rounded by up to 6e-8, which is 1.2e-4 of 1 - a in
    the slowest channels (1 - a ~ |A| / 2 = 5e-4); over their memory of 2000 tokens that averages to
    2.7e-6 of the state and of the adjoint, and dA, a product of both over such spans, is good to a few
    times that, 1.6e-5 of its own size -- which in those channels is up to 30 times the rms over all
    channels: 5e-4 of the rms."""
    c = Case(4, 8200, D, io, seed=4400, gate=False, lens=[8200, 8129, 4000, 65])
    y, last, ck = run_fwd(c, save_checkpoints=True)
    ry, rlast, rg = c.reference()
    close(y, ry, io, TOL * 1.5, "y")
    close(last, rlast, "f32", TOL * 1.5, "last_state")
    one, two = run_bwd(c, ck), run_bwd(c)
    for k, ref in rg.items():
        close(one[k], ref, "f32" if k in ("dA", "dinitial_state") else io, 5e-4 if k == "dA" else TOL * 1.5, k)
        assert torch.equal(one[k], two[k]), f"{k}: other values without the forward's states"


@pytest.mark.parametrize("io,D", [("bf16", 1023), ("f32", 500)])
def test_items_of_two_chunks_in_groups_of_one(io, D):
    """72 chains of 65 chunks: every item of two chunks waits for the one before it; tolerances as above."""
    c = Case(9, 4100, D, io, seed=4450, lens=[4100, 4097, 4096, 4095, 4033, 4032, 3000, 64, 0])
    y, last, ck = run_fwd(c, save_checkpoints=True)
    ry, rlast, rg = c.reference()
    close(y, ry, io, TOL * 1.5, "y")
    close(last, rlast, "f32", TOL * 1.5, "last_state")
    one, two = run_bwd(c, ck), run_bwd(c)
    for k, ref in rg.items():
        close(one[k], ref, "f32" if k in ("dA", "dinitial_state") else io, 5e-4 if k == "dA" else TOL * 1.5, k)
        assert torch.equal(one[k], two[k]), f"{k}: other values without the forward's states"


@pytest.mark.parametrize("io,D", [("bf16", 130), ("f32", 67)])
def test_nan_in_groups_of_one(io, D):
    """A NaN state is handed on as one (and not taken for a missing one); nothing else changes."""
    c = Case(70, 300, D, io, seed=4500, gate=False)
    ref = run_fwd(c)[0].clone()
    c.t["x"][33, 100, 5] = float("nan")
    c.t["h0"][60, 9] = float("nan")
    y, last, ck = run_fwd(c, save_checkpoints=True)
    bad = torch.isnan(y)
    assert bad[33, 100:, 5].all() and bad[60, :, 9].all() and int(bad.sum()) == 200 + 300
    assert torch.equal(y[~bad], ref[~bad])
    assert torch.isnan(last[33, 5]) and torch.isnan(last[60, 9]) and int(torch.isnan(last).sum()) == 2
    grads = run_bwd(c, ck)
    bad = torch.isnan(grads["dr"])
    assert bad[33, 100:, 5].all() and bad[60, :, 9].all() and int(bad.sum()) == 200 + 300
    assert not torch.isnan(grads["dx"]).any(), "dx does not depend on the states"


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bsz,L,D", [(90, 130, 129), (2, 700, 129), (3, 64, 40)])
def test_state_in_place(io, bsz, L, D):
    """last_state over initial_state, in every schedule: the chain's first chunk alone reads it."""
    c = Case(bsz, L, D, io, seed=4600, lens=lengths(bsz, L, 1))
    y, last = run_fwd(c)
    for _ in range(3):
        (x, r, g, A, z), k = c.fwd_args()
        st = k["initial_state"].clone()
        y2, last2 = ssmscan.gated_scan_fwd(x, r, g, A, z, initial_state=st, last_state=st, seq_lens=k["seq_lens"])
        torch.cuda.synchronize()
        assert last2 is st and torch.equal(y, y2) and torch.equal(st, last)


@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("bsz,L,D", [(3000, 40, 129), (1200, 130, 129), (1500, 40, 385), (3000, 40, 131)])
def test_state_in_place_where_lanes_share_a_channel(bsz, L, D, ragged):
    """Many sequences of an odd width, so that the tiles of a sequence run far apart in time: the state
    advanced in place is the one written elsewhere, to the bit."""
    c = Case(bsz, L, D, "bf16", gate=True, state=True, seed=7 * bsz + D, lens=lengths(bsz, L, 5) if ragged else None)
    y, last = run_fwd(c)
    state = c.t["h0"].clone()
    a, k = c.fwd_args()
    y2, last2 = ssmscan.gated_scan_fwd(*a, **dict(k, initial_state=state), last_state=state)
    torch.cuda.synchronize()
    assert last2 is state and torch.equal(y, y2) and torch.equal(last, state)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_schedules_agree(io):
    """The same sequence alone, among others, and in a batch that selects other schedules."""
    one = Case(1, 520, 64, io, seed=4700)
    y, last = run_fwd(one)
    many = Case(80, 520, 64, io, seed=4701)
    for k in ("x", "r", "g", "z", "h0"):
        many.t[k][17] = one.t[k][0]
    many.t["A"].copy_(one.t["A"])
    y2, last2 = run_fwd(many)
    assert raw_error(to_host_f64(last2[17]), to_host_f64(last[0])) <= 2e-5
    assert raw_error(to_host_f64(y2[17]), to_host_f64(y[0])) <= (2e-5 if io == "f32" else 1e-2)


def test_outputs_of_another_stream_wait_for_nothing():
    """A call on a stream of the caller's: what it allocates is not memory that the current stream has
    yet to write, though that memory has been given back."""
    c = Case(4, 1000, 256, "bf16", seed=4900)
    y, last, _ = run_fwd(c, save_checkpoints=True)
    grads = {n: t.clone() for n, t in run_bwd(c).items()}
    a, k = c.fwd_args()
    s = torch.cuda.Stream()
    m = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    busy = [torch.empty_like(y) for _ in range(8)]
    for _ in range(8):
        m = m @ m * 1e-3
    for b in busy:
        b.fill_(3.0)
    del busy, b
    y2, last2, ck = ssmscan.gated_scan_fwd(*a, **k, stream=s, save_checkpoints=True)
    g2 = ssmscan.gated_scan_bwd(c.t["dy"], *a, **k, dlast_state=c.t["dlast"], want_initial_state_grad=True,
                                checkpoints=ck, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, last2)
    assert all(torch.equal(grads[n], g2[n]) for n in grads)


def test_workspace_refusals():
    """A workspace is on the tensors' GPU and in one piece."""
    c = Case(2, 200, 64, "f32", seed=4910)
    a, k = c.fwd_args()
    dy = c.t["dy"]
    for bad in (torch.empty(1 << 22, dtype=torch.uint8), torch.empty(1 << 23, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            ssmscan.gated_scan_fwd(*a, **k, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            ssmscan.gated_scan_bwd(dy, *a, **k, workspace=bad)
        n = torch.ones(64, device="cuda")
        rows = torch.ones(200, device="cuda")
        with pytest.raises(ValueError, match="workspace"):
            ssmscan.layernorm_bwd(dy[0], dy[0], n, rows, rows, workspace=bad)
