"""Refusals of the entry points of the state space dual layer with its convolution and of the group norm: every
call here fails (or is empty) on the host, before anything is launched; no pointer is dereferenced and no GPU
is needed."""
import ctypes
import math
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def b():
    from selective_state_space_32_amd import ssmscan
    return ssmscan


def ptr(v):
    return P(v) if v else None


def dims(b, batch=2, seqlen=130, nheads=4, headdim=64, ngroups=2, dstate=64, xs=0, ds=0, io=1, width=4):
    return b.ssm_ssd_conv_dims(batch, seqlen, nheads, headdim, ngroups, dstate, xs, ds, io, width)


FWD = ("x", "w", "cb", "cs", "dt", "A", "D", "bias", "h0", "lens")


def fwd(b, d, flags=1, ws_bytes=None, **kw):
    v = dict(x=FAKE, w=FAKE, cb=0, cs=0, dt=FAKE, A=FAKE, D=0, bias=0, h0=0, lens=0, y=FAKE, last=0, co=0, ws=FAKE)
    v.update(kw)
    ref = None if d is None else ctypes.byref(d)
    if ws_bytes is None:
        ws_bytes = 0 if d is None else b.lib.ssm_ssd_conv_workspace_bytes(ref, flags)
    return b.lib.ssm_ssd_conv_fwd(*(ptr(v[k]) for k in FWD), flags, *(ptr(v[k]) for k in ("y", "last", "co")), ref,
                                  ptr(v["ws"]), ws_bytes, None)


BWD_OUT = ("dx", "dw", "dcb", "dcs", "ddt", "dA", "dD", "dbias", "dh0")


def bwd(b, d, flags=1, ws_bytes=None, ck_bytes=None, **kw):
    v = dict(x=FAKE, w=FAKE, cb=0, cs=0, dt=FAKE, A=FAKE, D=0, bias=0, h0=0, lens=0, dy=FAKE, dlast=0, ck=0, dx=FAKE,
             dw=FAKE, dcb=0, dcs=0, ddt=FAKE, dA=FAKE, dD=0, dbias=0, dh0=0, ws=FAKE)
    v.update(kw)
    ref = None if d is None else ctypes.byref(d)
    if ws_bytes is None:
        ws_bytes = 0 if d is None else b.lib.ssm_ssd_conv_bwd_workspace_bytes(ref, flags)
    if ck_bytes is None:
        ck_bytes = 0 if d is None else b.lib.ssm_ssd_conv_workspace_bytes(ref, 4)
    return b.lib.ssm_ssd_conv_bwd(*(ptr(v[k]) for k in FWD), flags, ptr(v["dy"]), ptr(v["dlast"]), ptr(v["ck"]), ck_bytes,
                                  *(ptr(v[k]) for k in BWD_OUT), ref, ptr(v["ws"]), ws_bytes, None)


def step(b, d, flags=1, ws_bytes=None, **kw):
    v = dict(st=FAKE, cs=FAKE, x=FAKE, w=FAKE, cb=0, dt=FAKE, A=FAKE, D=0, bias=0, y=FAKE, ws=FAKE)
    v.update(kw)
    ref = None if d is None else ctypes.byref(d)
    if ws_bytes is None:
        ws_bytes = 0 if d is None else b.lib.ssm_ssd_conv_step_workspace_bytes(ref)
    return b.lib.ssm_ssd_conv_step(*(ptr(v[k]) for k in ("st", "cs", "x", "w", "cb", "dt", "A", "D", "bias")), flags,
                                   ptr(v["y"]), ref, ptr(v["ws"]), ws_bytes, None)


BAD_SHAPES = [dict(batch=-1), dict(seqlen=-5), dict(nheads=-2), dict(headdim=0), dict(headdim=12), dict(headdim=-8),
              dict(headdim=65544), dict(dstate=0), dict(dstate=20), dict(dstate=136), dict(ngroups=0), dict(ngroups=3),
              dict(width=0), dict(width=5), dict(nheads=1 << 20), dict(ngroups=1 << 18, nheads=1 << 18),
              dict(seqlen=(1 << 30) + 1), dict(batch=(1 << 30) + 1), dict(batch=1 << 29, seqlen=1 << 20),
              dict(xs=511), dict(xs=-1), dict(xs=(1 << 30) + 1), dict(ds=3), dict(ds=-4)]


def test_fwd_refusals(b):
    d = dims(b)
    assert fwd(b, None) == -1
    for k in ("x", "w", "dt", "A", "y"):
        assert fwd(b, d, **{k: 0}) == -1, k
    for kw in BAD_SHAPES:
        assert fwd(b, dims(b, **kw)) == -2, kw
        assert b.lib.ssm_ssd_conv_workspace_bytes(ctypes.byref(dims(b, **kw)), 4) == 0
        assert b.lib.ssm_ssd_conv_bwd_workspace_bytes(ctypes.byref(dims(b, **kw)), 0) == 0
        assert b.lib.ssm_ssd_conv_step_workspace_bytes(ctypes.byref(dims(b, **kw))) == 0
    for io in (2, -1):
        assert fwd(b, dims(b, io=io)) == -3
    for k, off in (("x", 1), ("dt", 1), ("w", 2), ("cb", 2), ("A", 2), ("D", 2), ("bias", 2), ("lens", 2), ("y", 8), ("h0", 8),
                   ("last", 8), ("cs", 8), ("co", 8)):
        assert fwd(b, d, **{k: FAKE + off}) == -4, k
    for flags in (2, 8, 1 | 64):
        assert fwd(b, d, flags=flags, ws_bytes=1 << 40) == -8
    need, more = (b.lib.ssm_ssd_conv_workspace_bytes(ctypes.byref(d), f) for f in (1, 5))
    assert 0 < need < more
    assert fwd(b, d, ws_bytes=need - 1) == -6 and "workspace" in b.last_error()
    assert fwd(b, d, flags=5, ws_bytes=more - 1) == -6
    assert fwd(b, d, ws=0) == -6
    assert fwd(b, d, ws=FAKE + 8) == -4


def test_bwd_refusals(b):
    d = dims(b)
    assert bwd(b, None) == -1
    for k in ("x", "w", "dt", "A", "dy", "dx", "dw", "ddt", "dA"):
        assert bwd(b, d, **{k: 0}) == -1, k
    for kw in BAD_SHAPES:
        assert bwd(b, dims(b, **kw)) == -2, kw
    assert bwd(b, dims(b, io=7)) == -3
    for k, off in (("x", 1), ("dt", 1), ("ddt", 1), ("w", 2), ("cb", 2), ("A", 2), ("D", 2), ("bias", 2), ("lens", 2),
                   ("dw", 2), ("dcb", 2), ("dA", 2), ("dD", 2), ("dbias", 2), ("dy", 8), ("dx", 8), ("h0", 8), ("dlast", 8),
                   ("dh0", 8), ("cs", 8), ("dcs", 8), ("ck", 8)):
        assert bwd(b, d, **{k: FAKE + off}) == -4, k
    assert bwd(b, d, flags=2, ws_bytes=1 << 40) == -8
    assert bwd(b, d, flags=5) == -1 and "checkpoints" in b.last_error()
    ck = b.lib.ssm_ssd_conv_workspace_bytes(ctypes.byref(d), 5)
    assert bwd(b, d, flags=5, ck=FAKE, ck_bytes=ck - 1) == -6
    for flags in (1, 5):
        need = b.lib.ssm_ssd_conv_bwd_workspace_bytes(ctypes.byref(d), flags)
        assert need > 0
        assert bwd(b, d, flags=flags, ck=FAKE, ws_bytes=need - 1) == -6
        assert bwd(b, d, flags=flags, ck=FAKE, ws=0) == -6
        assert bwd(b, d, flags=flags, ck=FAKE, ws=FAKE + 8) == -4


def test_step_refusals(b):
    d = dims(b)
    assert step(b, None) == -1
    for k in ("st", "cs", "x", "w", "dt", "A", "y"):
        assert step(b, d, **{k: 0}) == -1, k
    for kw in BAD_SHAPES:
        assert step(b, dims(b, **kw)) == -2, kw
    for k, off in (("x", 1), ("dt", 1), ("y", 1), ("w", 2), ("cb", 2), ("A", 2), ("D", 2), ("bias", 2), ("st", 8), ("cs", 8)):
        assert step(b, d, **{k: FAKE + off}) == -4, k
    assert step(b, d, flags=4) == -8


def test_empty_calls_launch_nothing(b):
    for kw in (dict(batch=0), dict(nheads=0)):
        d = dims(b, **kw)
        assert fwd(b, d, x=0, w=0, dt=0, A=0, y=0, ws=0) == 0
        assert step(b, d, st=0, cs=0, x=0, w=0, dt=0, A=0, y=0, ws=0) == 0
    assert bwd(b, dims(b, nheads=0), x=0, w=0, dt=0, A=0, dy=0, dx=0, dw=0, ddt=0, dA=0, ws=0) == 0


# ---- the group norm ----

def gdims(b, batch=2, seqlen=7, dim=96, io=1):
    return b.ssm_dims(batch, seqlen, dim, 5, io, -3)   # dstate and chunk_len do not apply


def gfwd(b, d, groups=4, flags=0, eps=1e-5, zs=0, **kw):
    v = dict(x=FAKE, z=0, w=FAKE, bi=0, y=FAKE, m=0, r=0)
    v.update(kw)
    return b.lib.ssm_groupnorm_fwd(ptr(v["x"]), ptr(v["z"]), zs, ptr(v["w"]), ptr(v["bi"]), groups, eps, flags, ptr(v["y"]),
                                   ptr(v["m"]), ptr(v["r"]), None if d is None else ctypes.byref(d), None)


def gbwd(b, d, groups=4, flags=0, zs=0, ws_bytes=None, **kw):
    v = dict(dy=FAKE, x=FAKE, z=0, w=FAKE, bi=0, m=FAKE, r=FAKE, dx=FAKE, dz=0, dw=FAKE, db=0, ws=FAKE)
    v.update(kw)
    ref = None if d is None else ctypes.byref(d)
    if ws_bytes is None:
        ws_bytes = 0 if d is None else b.lib.ssm_groupnorm_bwd_workspace_bytes(ref, groups)
    return b.lib.ssm_groupnorm_bwd(ptr(v["dy"]), ptr(v["x"]), ptr(v["z"]), zs, ptr(v["w"]), ptr(v["bi"]), ptr(v["m"]), ptr(v["r"]),
                                   groups, flags, *(ptr(v[k]) for k in ("dx", "dz", "dw", "db")), ref, ptr(v["ws"]), ws_bytes, None)


def test_groupnorm_refusals(b):
    d = gdims(b)
    for call in (gfwd, gbwd):
        assert call(b, None) == -1
        for kw in (dict(batch=-1), dict(seqlen=-1), dict(dim=-4), dict(batch=1 << 20, seqlen=1 << 12), dict(dim=1 << 27)):
            assert call(b, gdims(b, **kw)) == -2, kw
        for groups in (0, -1, 5, 97):
            assert call(b, d, groups=groups) == -2, groups
        assert call(b, gdims(b, io=9)) == -3
        assert call(b, d, flags=8) == -8
        assert call(b, d, flags=2) == -1 and "GATE_FIRST" in b.last_error()
        assert call(b, d, flags=4, z=FAKE, dz=FAKE) == -8
        assert call(b, d, z=FAKE, zs=95, dz=FAKE) == -2
        assert call(b, d, z=FAKE, zs=(1 << 30) + 1, dz=FAKE) == -2
    for k in ("x", "w", "y"):
        assert gfwd(b, d, **{k: 0}) == -1, k
    for k in ("dy", "x", "w", "m", "r", "dx"):
        assert gbwd(b, d, **{k: 0}) == -1, k
    assert gbwd(b, d, z=FAKE) == -1   # dz
    for k, off in (("x", 1), ("z", 1), ("y", 1), ("w", 2), ("bi", 2), ("m", 2), ("r", 2)):
        assert gfwd(b, d, **{k: FAKE + off}) == -4, k
    for k, off in (("x", 1), ("dy", 1), ("dx", 1), ("dz", 1), ("w", 2), ("m", 2), ("r", 2), ("dw", 2), ("db", 2)):
        assert gbwd(b, d, **{k: FAKE + off}) == -4, k
    for eps in (-1e-3, math.inf, math.nan):
        assert gfwd(b, d, eps=eps) == -9
    need = b.lib.ssm_groupnorm_bwd_workspace_bytes(ctypes.byref(d), 4)
    assert need > 0
    assert gbwd(b, d, ws_bytes=need - 1) == -6
    assert gbwd(b, d, ws=0) == -6
    assert gbwd(b, d, ws=FAKE + 4) == -4
    assert gfwd(b, gdims(b, batch=0), x=0, w=0, y=0) == 0 and gfwd(b, gdims(b, dim=0), groups=1, x=0, w=0, y=0) == 0


# ---- the binding ----

def test_binding_refusals(b):
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    f = lambda *s: z(*s, dt=torch.float32)
    row = 4 * 8 + 2 * 2 * 8
    ok = dict(xbc=z(2, 5, row), conv_w=f(row, 4), conv_b=f(row), dt=z(2, 5, 4), A=f(4), D=f(4), dt_bias=f(4))
    call = lambda **kw: b.ssd_conv_fwd(**dict(ok, **kw), dstate=8, ngroups=2)
    for kw in (dict(xbc=z(2, 5, row + 1)), dict(xbc=z(5, row)), dict(conv_w=f(row, 4, 1)), dict(conv_w=f(row - 1, 4)),
               dict(conv_b=f(row + 1)), dict(dt=z(2, 5, 3)), dict(dt=z(2, 4, 4)), dict(A=f(4, 1)), dict(A=f(5)), dict(D=f(3)),
               dict(dt_bias=f(8)), dict(xbc=z(2, row, 5).transpose(1, 2)), dict(dt=z(2, 5, 4, 2)[..., 0]),
               dict(xbc=z(2, 6, row)[:, :5]), dict(xbc=z(1, 1, row).expand(2, 5, row))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(xbc=z(2, 5, row, dt=torch.float16)), dict(dt=f(2, 5, 4)), dict(A=z(4)), dict(conv_w=z(row, 4))):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(ValueError, match="GPU"):   # host tensors
        call()
    with pytest.raises(ValueError):
        b.ssd_conv_fwd(**ok, dstate=8, ngroups=2, initial_state=f(2, 4, 8, 9))
    with pytest.raises(ValueError):
        b.ssd_conv_fwd(**ok, dstate=8, ngroups=2, conv_state=z(2, 4, row))
    with pytest.raises(ValueError):
        b.ssd_conv_fwd(**ok, dstate=8, ngroups=2, seq_lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.ssd_conv_bwd(z(2, 5, 4, 9), **ok, dstate=8, ngroups=2)
    x, w = z(3, 24), f(24)
    for kw in (dict(groups=5), dict(groups=0), dict(silu=True, z=x), dict(gate_first=True), dict(z=z(3, 23)), dict(z=z(24, 3).T),
               dict(bias=f(23))):
        with pytest.raises(ValueError):
            b.groupnorm_fwd(x, w, **dict(dict(groups=3), **kw))
    with pytest.raises(TypeError):
        b.groupnorm_fwd(x, w, z=f(3, 24))
    with pytest.raises(ValueError):
        b.groupnorm_bwd(x, x, w, None, None, f(3, 2), groups=3)


def test_rows_of_a_wider_tensor(b):
    """The distance between rows that the binding passes on: packed, parts of wider rows, single rows."""
    import torch
    f32, cpu = torch.float32, torch.device("cpu")
    t = torch.zeros(3, 7, 50)
    rows = lambda v, lead, w: b._rows(v, "v", torch.Size(lead), w, f32, cpu)
    assert rows(t, (3, 7), 50) == 50
    assert rows(t[..., 10:30], (3, 7), 20) == 50
    assert rows(t[:, :1, 10:30], (3, 1), 20) == 350
    assert rows(t[:1, :, 10:30], (1, 7), 20) == 50
    assert rows(t[:1, :1, 10:30], (1, 1), 20) == 20
    assert rows(t[:0, :, 10:30], (0, 7), 20) >= 20
    assert rows(t[..., 5:6], (3, 7), 1) == 50
    for bad, lead, w in ((t[:, ::2, :20], (3, 4), 20), (t[:, :5, :20], (3, 5), 20), (t[..., ::2], (3, 7), 25)):
        with pytest.raises(ValueError):
            rows(bad, lead, w)
