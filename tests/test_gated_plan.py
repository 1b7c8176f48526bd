"""The gated recurrence's plan query (host logic, no GPU): refusals, and what a launch needs of every plan so
that no work item is left out and no wait is without end."""
import ctypes
import random

import pytest


@pytest.fixture(scope="module")
def b():
    from selective_state_space_32_amd import ssmscan
    return ssmscan


def test_refusals(b):
    out = b.ssm_gated_plan()
    good = b.ssm_dims(2, 700, 128, 3, 1, -7)
    assert b.lib.ssm_gated_scan_plan(None, 0, ctypes.byref(out)) == -1
    assert b.lib.ssm_gated_scan_plan(ctypes.byref(good), 0, None) == -1
    for kw, status in ((dict(batch=-1), -2), (dict(dim=-1), -2), (dict(seqlen=(1 << 30) + 1), -2),
                       (dict(batch=1 << 20, seqlen=1 << 20, dim=1 << 10), -2), (dict(io_dtype=5), -3)):
        d = b.ssm_dims(2, 700, 128, 3, 1, -7)
        for k, v in kw.items():
            setattr(d, k, v)
        out.chains = 99
        assert b.lib.ssm_gated_scan_plan(ctypes.byref(d), 1, ctypes.byref(out)) == status, kw
        assert out.chains == 0
    assert b.gated_plan(0, 5, 8, 0)["workgroups"] == 0 and b.gated_plan(5, 5, 0, 1)["workgroups"] == 0
    with pytest.raises(b.SSMError):
        b.gated_plan(2, -1, 8, 0)


def draws(p):
    """Workgroups that draw from each queue, as the kernel deals them: `run` in a row, queue by queue."""
    n = [0] * p["queues"]
    for turn in range(p["workgroups"] // p["run"]):
        n[turn % p["queues"]] += p["run"]
    return n


def test_every_item_is_drawn(b):
    rng = random.Random(7)
    seen = set()
    for _ in range(3000):
        bsz, L = int(2 ** rng.uniform(0, 7)), int(2 ** rng.uniform(0, 15))
        D = int(2 ** rng.uniform(0, 12))
        io, back = rng.randrange(2), rng.randrange(2)
        p = b.gated_plan(bsz, L, D, io, bool(back))
        V, q, run = p["lane_channels"], p["queues"], p["run"]
        chunks = max(1, -(-L // 64))
        assert V in ((1,) if io == 0 else (1, 2)) and p["chains"] == bsz * -(-D // (64 * V))
        assert p["item_chunks"] in ((1,) if back else (1, 2)) and p["items"] == -(-chunks // p["item_chunks"])
        assert 1 <= q <= 8 and run in (1, 8) and p["group"] in (1, 2, 4, 8, 16, 32, 64)
        assert p["workgroups"] % (q * run) == 0
        # (a lane that shares a channel with its neighbour has that neighbour in its wave)
        assert V == 1 or D % 128 != 1
        share = [p["chains"] * (k + 1) // q - p["chains"] * k // q for k in range(q)]
        assert sum(share) == p["chains"]
        if p["workgroups"] <= 20000:
            assert all(n >= s * p["items"] for n, s in zip(draws(p), share)), (bsz, L, D, io, back, p)
        seen.add((q, run, p["group"]))
    assert len({s[0] for s in seen}) == 8 and {s[1] for s in seen} == {1, 8}
