"""The group norm's entry points on problems without values, with any number of groups: a status, on the host."""
import ctypes

import pytest

from test_ssd_conv_abi import b, gbwd, gdims, gfwd  # noqa: F401  (the fixture)



@pytest.mark.parametrize("groups", [1, 7, 1 << 26, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, 1 << 32, (1 << 32) + 1, 1 << 62])
@pytest.mark.parametrize("kw", [dict(), dict(batch=0), dict(seqlen=0)])
def test_rows_without_values(b, groups, kw):
    """(2^32 groups of nothing ended the process: their number was cut to 32 bits and divided by.)"""
    d = gdims(b, dim=0, **kw)
    assert gfwd(b, d, groups=groups, x=0, w=0, y=0) == 0
    assert gbwd(b, d, groups=groups, ws_bytes=0, ws=0) == 0
    assert b.lib.ssm_groupnorm_bwd_workspace_bytes(ctypes.byref(d), groups) == 0


def test_values_without_rows(b):
    for kw in (dict(batch=0), dict(seqlen=0)):
        d = gdims(b, **kw)
        assert gfwd(b, d, groups=96, x=0, w=0, y=0) == 0 and gfwd(b, d, groups=5, x=0, w=0, y=0) == -2
