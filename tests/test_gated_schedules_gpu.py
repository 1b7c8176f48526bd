"""The gated recurrence under every kind of schedule that its rules can choose, each case with the schedule it
is there for asserted from the library's own plan, so that a change of a rule cannot leave one untested:
queues that do not share the chains evenly (one of them without any), seven queues, few chains with eight draws
in a row and shared hand-overs, in items of one chunk and of two, and many chains with eight draws in a row.

The oracle is the definition in fp64 on the same inputs, token by token.  Tolerances as in test_gated_gpu.py and
test_gated_paths_gpu.py: 1e-4 of the rms, times 1.5 for long sequences, whose states remember at most ~2000
tokens; 5e-4 for dA there, a product of states and adjoints over such spans."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_32_amd import ssmscan  # noqa: E402

IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(bsz, L, D, io, lens, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    v = {k: normal(bsz, L, D).to(IO[io]) for k in ("x", "r", "g", "z", "dy")}
    v["A"] = torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda"))
    v["h0"], v["dlast"] = normal(bsz, D), normal(bsz, D)
    v["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return v


def run(v):
    kw = dict(initial_state=v["h0"], seq_lens=v["lens"])
    y, last, ck = ssmscan.gated_scan_fwd(v["x"], v["r"], v["g"], v["A"], v["z"], save_checkpoints=True, **kw)
    out = ssmscan.gated_scan_bwd(v["dy"], v["x"], v["r"], v["g"], v["A"], v["z"], dlast_state=v["dlast"],
                                 want_initial_state_grad=True, checkpoints=ck, **kw)
    torch.cuda.synchronize()
    return dict(out, y=y, last_state=last)


def oracle(v):
    """The recurrence and its gradients in fp64; tokens past a length have a = 1 and no input."""
    x, r, g, z, dy, A = (v[k].double() for k in ("x", "r", "g", "z", "dy", "A"))
    bsz, L, _ = x.shape
    live = torch.ones((bsz, L, 1), dtype=torch.bool, device="cuda")
    if v["lens"] is not None:
        live = (torch.arange(L, device="cuda") < v["lens"][:, None])[:, :, None]
    s, i, sz = torch.sigmoid(r), torch.sigmoid(g), torch.sigmoid(z)
    u = A * s
    a, beta = torch.exp(u).where(live, torch.ones_like(u)), torch.sqrt(-torch.expm1(2.0 * u))
    b = (beta * i * x).where(live, torch.zeros_like(x))
    h, out = v["h0"].double(), {}
    before, after = torch.empty_like(x), torch.empty_like(x)
    for t in range(L):
        before[:, t] = h
        h = torch.addcmul(b[:, t], a[:, t], h)
        after[:, t] = h
    out["last_state"], out["y"] = h, after * z * sz * live
    dh = dy * z * sz * live
    lam, carry = torch.empty_like(x), v["dlast"].double()
    for t in range(L - 1, -1, -1):
        now = dh[:, t] + carry
        lam[:, t] = now
        carry = a[:, t] * now
    lam *= live
    out["dinitial_state"] = carry
    out["dz"] = dy * after * sz * (1.0 + z * (1.0 - sz)) * live
    out["dx"] = lam * beta * i
    out["dg"] = lam * beta * x * i * (1.0 - i)
    du = lam * (a * before - i * x * a * a / beta)
    out["dr"] = du * A * s * (1.0 - s)
    out["dA"] = (du * s).sum((0, 1))
    return out


def error(got, ref):
    """Largest error over the reference's rms, for bf16 beyond the last rounding's half spacing."""
    d = (got.double() - ref).abs()
    if got.dtype == torch.bfloat16:
        m = got.double().abs()
        d = d - torch.where(m > 0, 0.5 * torch.exp2(torch.floor(torch.log2(m.clamp_min(1e-300))) - 7.0), m)
    return float(d.max() / ref.pow(2).mean().sqrt())


def check(v, tol, tol_dA):
    got, ref = run(v), oracle(v)
    assert set(got) == set(ref)
    for k in ref:
        e = error(got[k], ref[k])
        print(f"{k}: err/rms {e:.2e}", flush=True)
        assert e <= (tol_dA if k == "dA" else tol), (k, e)
    again = run(v)
    assert all(torch.equal(got[k], again[k]) for k in got), "other values on a second run"


# (batch, L, D, io, the forward's plan, the backward's where it differs)
SCHEDULES = [
    # seven chains: dealt to eight queues where they are short (one queue has none), to seven where long
    (1, 700, 448, "f32", dict(chains=7, queues=8, group=16, run=1), {}),
    (1, 2100, 448, "f32", dict(chains=7, queues=7, group=16, run=1), {}),
    (1, 2400, 896, "bf16", dict(chains=7, queues=7, group=16, run=1, lane_channels=2), {}),
    # 21 chains, groups of eight; and 42 in items of two chunks forwards
    (3, 2100, 448, "f32", dict(chains=21, queues=7, group=8, run=1, item_chunks=1), {}),
    (3, 2400, 893, "bf16", dict(chains=21, queues=7, group=8, run=1, lane_channels=2), {}),
    (2, 4200, 1300, "f32", dict(chains=42, queues=7, group=4, run=1, item_chunks=2), dict(item_chunks=1)),
    # one to six queues, two of them with chains of unequal numbers
    (1, 2100, 64, "f32", dict(chains=1, queues=1, group=64), {}),
    (2, 2100, 64, "f32", dict(chains=2, queues=2, group=64), {}),
    (1, 2100, 150, "f32", dict(chains=3, queues=3, group=32), {}),
    (2, 2100, 100, "f32", dict(chains=4, queues=4, group=32), {}),
    (5, 2100, 50, "f32", dict(chains=5, queues=5, group=32), {}),
    (2, 2100, 160, "f32", dict(chains=6, queues=6, group=16), {}),
    (11, 700, 128, "f32", dict(chains=22, queues=8, group=8), {}),
    # many chunks in few chains: eight draws in a row, hand-overs shared, items of two chunks forwards
    (1, 32808, 2048, "bf16", dict(chains=16, group=8, run=8, queues=8, item_chunks=2, lane_channels=2),
     dict(item_chunks=1)),
    (2, 32808, 1024, "bf16", dict(chains=16, group=8, run=8, queues=8, item_chunks=2), dict(item_chunks=1)),
    (1, 32808, 2047, "bf16", dict(chains=16, group=8, run=8, queues=8, item_chunks=2), dict(item_chunks=1)),
    # and of one chunk, where a lane has one channel; five queues
    (5, 19200, 129, "bf16", dict(chains=15, group=8, run=8, queues=5, item_chunks=1, lane_channels=1), {}),
    # many chains of whole lines: eight draws in a row, every chunk waits for the one before it
    (8, 2048, 1024, "f32", dict(chains=128, group=1, run=8, queues=8, item_chunks=1), {}),
    (8, 2048, 2048, "bf16", dict(chains=128, group=1, run=8, queues=8, item_chunks=1, lane_channels=2), {}),
    # and where rows start inside a line, one draw in a row
    (8, 2048, 1027, "f32", dict(chains=136, group=1, run=1, queues=8, item_chunks=1), {}),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("bsz,L,D,io,forward,backward", SCHEDULES)
def test_schedule(bsz, L, D, io, forward, backward, ragged):
    for back, want in ((False, forward), (True, dict(forward, **backward))):
        plan = ssmscan.gated_plan(bsz, L, D, IO[io], backward=back)
        assert {k: plan[k] for k in want} == want, plan
    lens = None
    if ragged:   # the whole length, none, the ends of chunks and their neighbours
        some = [L, 0, L // 2, 64, L - 1, 129, L // 3 // 64 * 64, 1]
        lens = [some[(b + 1) % len(some)] if bsz > 1 else L - 70 for b in range(bsz)]
    print(f"[{bsz} x {L} x {D} {io} lens={lens}]", flush=True)
    long = L > 1000
    check(make(bsz, L, D, io, lens, seed=6000 + L + D), 1.5e-4 if long else 1e-4, 5e-4 if long else 1e-4)


def test_every_schedule_is_there():
    """Between them the cases take every number of queues, both numbers of draws, and each way to hand over."""
    plans = [ssmscan.gated_plan(b, L, D, IO[io], backward=back) for b, L, D, io, _, _ in SCHEDULES
             for back in (False, True)]
    assert {p["queues"] for p in plans} == set(range(1, 9))
    assert {(p["run"], p["group"] > 1, p["item_chunks"]) for p in plans} >= {
        (1, False, 1), (1, True, 1), (1, True, 2), (8, False, 1), (8, True, 1), (8, True, 2)}
    assert any(p["chains"] < p["queues"] for p in plans)
