"""Sizes at which a launch of the state space dual layer with its convolution would hold 2^32 threads or more, which HIP
refuses: every entry point refuses them before its first launch.  On the host: what is taken is told by the workspace's
size, and by the refusal of a workspace that is too small for it, so no call here launches anything."""
import ctypes

import pytest

import test_ssd_conv_abi as abi
from test_ssd_conv_abi import b, dims  # noqa: F401  (the fixture)

WG256, WG1024 = (2 ** 32 - 1) // 256, (2 ** 32 - 1) // 1024
SMALL = dict(headdim=8, ngroups=1, dstate=8)


def needs(b, d, flags=1):
    r = ctypes.byref(d)
    return (b.lib.ssm_ssd_conv_workspace_bytes(r, flags), b.lib.ssm_ssd_conv_bwd_workspace_bytes(r, flags),
            b.lib.ssm_ssd_conv_step_workspace_bytes(r))


def taken(call, b, d):
    return call(b, d, ws_bytes=1) == -6


def refused(call, b, d):
    return call(b, d, ws_bytes=1 << 62) == -2 and "launch" in b.last_error()


@pytest.mark.parametrize("nheads,batch", [(64, 1 << 18), (1, WG256 + 1), (WG256 // 1024 + 1, 1024)])
def test_heads_of_many_sequences(b, nheads, batch):
    """A workgroup of 256 threads per (sequence, head)."""
    d = dims(b, batch=batch, seqlen=1, nheads=nheads, **SMALL)
    assert needs(b, d) == (0, 0, 0)
    for call in (abi.fwd, abi.bwd, abi.step):
        assert refused(call, b, d)
    d = dims(b, batch=batch - batch // 64, seqlen=1, nheads=nheads, **SMALL)
    assert needs(b, d)[2] > 0 and taken(abi.step, b, d)
    # (the convolution's launch: a workgroup per sequence's token, and one per four heads for the decays)
    if (batch - batch // 64) * (1 + (nheads + 3) // 4) <= WG256:
        assert needs(b, d)[0] > 0 and taken(abi.fwd, b, d)
    else:
        assert needs(b, d)[0] == 0 and refused(abi.fwd, b, d)


def test_tiles_of_a_head(b):
    """The scan takes a head's channels 64 at a time, the step all of them together."""
    d = dims(b, batch=1 << 21, seqlen=0, nheads=1, headdim=512, ngroups=1, dstate=8)
    assert needs(b, d)[:2] == (0, 0) and needs(b, d)[2] > 0
    assert refused(abi.fwd, b, d) and refused(abi.bwd, b, d) and taken(abi.step, b, d)


def test_rows_of_the_convolution(b):
    """A workgroup of the convolution per 1024 channels of a sequence's token, at least."""
    d = dims(b, batch=1 << 22, seqlen=1, nheads=1, headdim=4096, ngroups=1, dstate=8)     # rows of 4112: five
    assert needs(b, d) == (0, 0, 0)
    for call in (abi.fwd, abi.bwd, abi.step):
        assert refused(call, b, d)


def test_tokens_of_the_convolution(b):
    """Its workgroups take at most 32 tokens; those behind them a chunk of four heads."""
    for seqlen, ok in ((32 * (1 << 14), True), (32 * (1 << 14) + 32 * 768, False)):
        d = dims(b, batch=682, seqlen=seqlen, nheads=1, **SMALL)
        blocks = 682 * (seqlen // 32 + seqlen // 64)
        assert (blocks <= WG256) == ok, blocks
        assert (needs(b, d)[0] > 0) == ok
        assert taken(abi.fwd, b, d) if ok else refused(abi.fwd, b, d)


@pytest.mark.parametrize("batch,seqlen,groups", [(8192, 4096, 8), (WG1024 + 1, 1, 1), (1 << 19, 64, 8)])
def test_chunks_of_the_backward(b, batch, seqlen, groups):
    """A workgroup of 1024 threads per chunk and group: the forward runs such a batch, the backward does not."""
    kw = dict(seqlen=seqlen, nheads=groups, headdim=8, ngroups=groups, dstate=8)
    d = dims(b, batch=batch, **kw)
    for flags in (1, 5):
        assert needs(b, d, flags)[0] > 0 and needs(b, d, flags)[1] == 0
    assert taken(abi.fwd, b, d) and refused(abi.bwd, b, d)
    d = dims(b, batch=batch - max(batch // 4096, 1), **kw)
    assert needs(b, d)[1] > 0 and taken(abi.bwd, b, d)
