"""Refusals of the gated recurrence's and the layer norm's entry points: every call here fails (or is
empty) on the host, before anything is launched; no pointer is dereferenced and no GPU is needed."""
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


def dims(b, batch=2, seqlen=700, dim=128, io=1, dstate=3, chunk_len=-7):
    return b.ssm_dims(batch, seqlen, dim, dstate, io, chunk_len)   # dstate and chunk_len do not apply


def ptr(v):
    return P(v) if v else None


def fwd(b, d, ws_bytes=None, **kw):
    v = dict(x=FAKE, r=FAKE, g=FAKE, A=FAKE, z=0, h0=0, lens=0, y=FAKE, last=0, ws=FAKE)
    v.update(kw)
    ref = None if d is None else ctypes.byref(d)
    if ws_bytes is None:
        ws_bytes = 0 if d is None else b.lib.ssm_gated_scan_workspace_bytes(ref)
    return b.lib.ssm_gated_scan_fwd(*(ptr(v[k]) for k in ("x", "r", "g", "A", "z", "h0", "lens", "y", "last")), ref,
                                    ptr(v["ws"]), ws_bytes, None)


def bwd(b, d, ws_bytes=None, ck_bytes=None, **kw):
    v = dict(x=FAKE, r=FAKE, g=FAKE, A=FAKE, z=0, h0=0, lens=0, dy=FAKE, dlast=0, ck=0, dx=FAKE, dr=FAKE, dg=FAKE,
             dA=FAKE, dz=0, dh0=0, ws=FAKE)
    v.update(kw)
    ref = None if d is None else ctypes.byref(d)
    if ws_bytes is None:
        ws_bytes = 0 if d is None else b.lib.ssm_gated_scan_bwd_workspace_bytes(ref)
    if ck_bytes is None:
        ck_bytes = 0 if d is None else b.lib.ssm_gated_scan_workspace_bytes(ref)
    return b.lib.ssm_gated_scan_bwd(*(ptr(v[k]) for k in ("x", "r", "g", "A", "z", "h0", "lens", "dy", "dlast", "ck")),
                                    ck_bytes, *(ptr(v[k]) for k in ("dx", "dr", "dg", "dA", "dz", "dh0")), ref,
                                    ptr(v["ws"]), ws_bytes, None)


BAD_SHAPES = [dict(batch=-1), dict(seqlen=-5), dict(dim=-2), dict(dim=(1 << 30) + 1), dict(batch=(1 << 30) + 1),
              dict(seqlen=(1 << 30) + 1), dict(batch=1 << 20, dim=1 << 20),
              dict(batch=1 << 10, seqlen=1 << 20, dim=1 << 20)]


def test_gated_fwd_refusals(b):
    d = dims(b)
    assert fwd(b, None) == -1
    for k in ("x", "r", "g", "A", "y"):
        assert fwd(b, d, **{k: 0}) == -1, k
    for kw in BAD_SHAPES:
        assert fwd(b, dims(b, **kw)) == -2, kw
        assert b.lib.ssm_gated_scan_workspace_bytes(ctypes.byref(dims(b, **kw))) == 0
        assert b.lib.ssm_gated_scan_bwd_workspace_bytes(ctypes.byref(dims(b, **kw))) == 0
    assert fwd(b, dims(b, io=7)) == -3
    for k, off in (("x", 1), ("r", 1), ("g", 1), ("z", 1), ("y", 1), ("A", 2), ("h0", 2), ("lens", 2), ("last", 2)):
        assert fwd(b, d, **{k: FAKE + off}) == -4, k
    for k in ("x", "r", "g", "z", "y"):
        assert fwd(b, dims(b, io=0), **{k: FAKE + 2}) == -4, k
    need = b.lib.ssm_gated_scan_workspace_bytes(ctypes.byref(d))
    assert need > 0
    assert fwd(b, d, ws_bytes=need - 1) == -6 and "workspace" in b.last_error()
    assert fwd(b, d, ws=0) == -6
    assert fwd(b, d, ws=FAKE + 8) == -4


def test_gated_bwd_refusals(b):
    d = dims(b)
    assert bwd(b, None) == -1
    for k in ("x", "r", "g", "A", "dy", "dx", "dr", "dg", "dA"):
        assert bwd(b, d, **{k: 0}) == -1, k
    assert bwd(b, d, z=FAKE) == -1 and "dz" in b.last_error()
    for kw in BAD_SHAPES:
        assert bwd(b, dims(b, **kw)) == -2, kw
    assert bwd(b, dims(b, io=-1)) == -3
    for k, off in (("x", 1), ("r", 1), ("g", 1), ("z", 1), ("dy", 1), ("dx", 1), ("dr", 1), ("dg", 1), ("dz", 1),
                   ("A", 2), ("dA", 2), ("h0", 2), ("lens", 2), ("dlast", 2), ("dh0", 2)):
        assert bwd(b, d, **{k: FAKE + off}) == -4, k
    need = b.lib.ssm_gated_scan_bwd_workspace_bytes(ctypes.byref(d))
    ck = b.lib.ssm_gated_scan_workspace_bytes(ctypes.byref(d))
    assert need > ck > 0
    assert bwd(b, d, ws_bytes=need - 1) == -6
    assert bwd(b, d, ws=0) == -6
    assert bwd(b, d, ws=FAKE + 8) == -4
    assert bwd(b, d, ck=FAKE, ck_bytes=ck - 1) == -6 and "checkpoints" in b.last_error()
    assert bwd(b, d, ck=FAKE + 8) == -4


def test_gated_step_refusals(b):
    def step(d, **kw):
        v = dict(state=FAKE, x=FAKE, r=FAKE, g=FAKE, A=FAKE, z=0, y=FAKE)
        v.update(kw)
        return b.lib.ssm_gated_step(*(ptr(v[k]) for k in ("state", "x", "r", "g", "A", "z", "y")),
                                    None if d is None else ctypes.byref(d), None)
    d = dims(b, seqlen=-9)     # seqlen does not apply either
    assert step(None) == -1
    for k in ("state", "x", "r", "g", "A", "y"):
        assert step(d, **{k: 0}) == -1, k
    assert step(dims(b, batch=-1)) == -2 and step(dims(b, batch=1 << 20, dim=1 << 20)) == -2
    assert step(dims(b, io=2)) == -3
    for k, off in (("state", 2), ("x", 1), ("r", 1), ("g", 1), ("z", 1), ("y", 1), ("A", 2)):
        assert step(d, **{k: FAKE + off}) == -4, k
    assert step(dims(b, batch=0), state=0, x=0, r=0, g=0, A=0, y=0) == 0


def test_gated_empty_is_a_noop(b):
    for kw in (dict(batch=0), dict(dim=0)):
        d = dims(b, **kw)
        assert b.lib.ssm_gated_scan_workspace_bytes(ctypes.byref(d)) == 0
        assert fwd(b, d, x=0, r=0, g=0, A=0, y=0, ws=0) == 0
    assert bwd(b, dims(b, dim=0), x=0, r=0, g=0, A=0, dy=0, dx=0, dr=0, dg=0, dA=0, ws=0) == 0


def norm(b, d, eps=1e-5, flags=0, **kw):
    v = dict(x=FAKE, res=0, w=FAKE, bias=0, y=FAKE, sum=0, mean=0, rstd=0)
    v.update(kw)
    return b.lib.ssm_layernorm_fwd(*(ptr(v[k]) for k in ("x", "res", "w", "bias")), eps, flags,
                                   *(ptr(v[k]) for k in ("y", "sum", "mean", "rstd")),
                                   None if d is None else ctypes.byref(d), None)


def norm_bwd(b, d, flags=0, ws_bytes=None, **kw):
    v = dict(dy=FAKE, s=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dres=0, ds=FAKE, dx=0, dw=FAKE, db=FAKE, ws=FAKE)
    v.update(kw)
    ref = None if d is None else ctypes.byref(d)
    if ws_bytes is None:
        ws_bytes = 0 if d is None else b.lib.ssm_layernorm_bwd_workspace_bytes(ref)
    return b.lib.ssm_layernorm_bwd(*(ptr(v[k]) for k in ("dy", "s", "w", "mean", "rstd", "dres")), flags,
                                   *(ptr(v[k]) for k in ("ds", "dx", "dw", "db")), ref, ptr(v["ws"]), ws_bytes, None)


NORM_SHAPES = [dict(batch=-1), dict(seqlen=-1), dict(dim=-1), dict(batch=1 << 16, seqlen=1 << 16),
               dict(dim=(1 << 30) + 1), dict(batch=1, seqlen=1 << 30, dim=1 << 20)]


def test_layernorm_refusals(b):
    d = dims(b)
    assert norm(b, None) == -1
    for k in ("x", "w", "y"):
        assert norm(b, d, **{k: 0}) == -1, k
    for kw in NORM_SHAPES:
        assert norm(b, dims(b, **kw)) == -2, kw
    assert norm(b, dims(b, io=3)) == -3
    for k, off in (("x", 1), ("y", 1), ("res", 1), ("sum", 1), ("w", 2), ("bias", 2), ("mean", 2), ("rstd", 2)):
        assert norm(b, d, **{k: FAKE + off}) == -4, k
    assert norm(b, d, flags=1, res=FAKE + 2) == -4 and norm(b, d, flags=1, sum=FAKE + 2) == -4
    assert norm(b, d, flags=2) == -8 and norm(b, d, flags=-1) == -8
    for eps in (-1e-6, math.nan, math.inf):
        assert norm(b, d, eps=eps) == -9 and "eps" in b.last_error()
    assert norm(b, dims(b, batch=0), x=0, w=0, y=0) == 0 and norm(b, dims(b, dim=0), x=0, w=0, y=0) == 0


def test_layernorm_bwd_refusals(b):
    d = dims(b)
    assert norm_bwd(b, None) == -1
    for k in ("dy", "s", "w", "mean", "rstd", "ds"):
        assert norm_bwd(b, d, **{k: 0}) == -1, k
    for kw in NORM_SHAPES:
        assert norm_bwd(b, dims(b, **kw)) == -2, kw
        assert b.lib.ssm_layernorm_bwd_workspace_bytes(ctypes.byref(dims(b, **kw))) == 0
    assert norm_bwd(b, dims(b, io=3)) == -3
    for k, off in (("dy", 1), ("s", 1), ("dres", 1), ("ds", 1), ("dx", 1), ("w", 2), ("mean", 2), ("rstd", 2),
                   ("dw", 2), ("db", 2)):
        assert norm_bwd(b, d, **{k: FAKE + off}) == -4, k
    assert norm_bwd(b, d, flags=1, s=FAKE + 2) == -4 and norm_bwd(b, d, flags=4) == -8
    need = b.lib.ssm_layernorm_bwd_workspace_bytes(ctypes.byref(d))
    assert need > 0
    assert norm_bwd(b, d, ws_bytes=need - 1) == -6 and norm_bwd(b, d, ws=0) == -6
    assert norm_bwd(b, d, dw=0, ws_bytes=need - 1) == -6      # dbias alone needs it too
    assert norm_bwd(b, d, ws=FAKE + 8) == -4
    assert norm_bwd(b, dims(b, dim=0), dy=0, s=0, w=0, mean=0, rstd=0, ds=0, dw=0, db=0, ws=0) == 0


def test_binding_refusals(b):
    """The Python binding's own checks (host tensors; nothing is called)."""
    import torch
    x, A = torch.zeros(2, 5, 8), torch.zeros(8)
    for bad in (dict(r=torch.zeros(2, 5, 4)), dict(g=torch.zeros(2, 5, 8, dtype=torch.bfloat16)), dict(A=torch.zeros(9)),
                dict(z=torch.zeros(2, 8, 5).transpose(1, 2)), dict(initial_state=torch.zeros(2, 9)),
                dict(seq_lens=torch.zeros(2)), dict(seq_lens=torch.zeros(3, dtype=torch.int32)),
                dict(x=torch.zeros(2, 5, 8, dtype=torch.float16)), dict(x=torch.zeros(5, 8)), dict(y=torch.zeros(2, 5, 9)),
                dict(last_state=torch.zeros(2, 8, dtype=torch.bfloat16)),
                dict(seq_lens=torch.zeros(4, dtype=torch.int32)[::2])):
        kw = dict(dict(x=x, r=x, g=x, A=A), **bad)
        with pytest.raises((ValueError, TypeError)):
            b.gated_scan_fwd(kw.pop("x"), kw.pop("r"), kw.pop("g"), kw.pop("A"), **kw)
    with pytest.raises((ValueError, TypeError)):
        b.gated_scan_bwd(torch.zeros(2, 5, 9), x, x, x, A)
    with pytest.raises((ValueError, TypeError)):
        b.gated_step(torch.zeros(2, 8, dtype=torch.bfloat16), x[:, 0].clone(), x[:, 0].clone(), x[:, 0].clone(), A)
    with pytest.raises((ValueError, TypeError)):
        b.gated_step(torch.zeros(2, 8), x, x, x, A)
    v, w = torch.zeros(4, 8), torch.zeros(8)
    for bad in (dict(weight=torch.zeros(9)), dict(bias=torch.zeros(8, dtype=torch.bfloat16)),
                dict(residual=torch.zeros(4, 9)), dict(residual=torch.zeros(4, 8, dtype=torch.float16)),
                dict(x=torch.zeros(8, 4).t()), dict(x=torch.zeros(4, 8, dtype=torch.int32))):
        kw = dict(dict(x=v, weight=w), **bad)
        with pytest.raises((ValueError, TypeError)):
            b.layernorm_fwd(kw.pop("x"), kw.pop("weight"), kw.pop("bias", None), **kw)
    with pytest.raises((ValueError, TypeError)):
        b.layernorm_bwd(v, torch.zeros(4, 8, dtype=torch.bfloat16), w, torch.zeros(4), torch.zeros(4))
    with pytest.raises((ValueError, TypeError)):
        b.layernorm_bwd(v, v, w, torch.zeros(4, 1), torch.zeros(4))


def test_host_tensors_are_refused(b):
    """Tensors in host memory, everything else right: refused by name, before the library is called."""
    import torch
    x, A, v, w = torch.zeros(2, 5, 8), torch.zeros(8), torch.zeros(4, 8), torch.zeros(8)
    for call in (lambda: b.gated_scan_fwd(x, x, x, A), lambda: b.gated_scan_bwd(x, x, x, x, A),
                 lambda: b.gated_step(v, v, v, v, A), lambda: b.layernorm_fwd(v, w),
                 lambda: b.layernorm_bwd(v, v, w, torch.zeros(4), torch.zeros(4))):
        with pytest.raises((ValueError, RuntimeError, AssertionError), match="cpu|CUDA|NVIDIA|HIP|GPU"):
            call()
