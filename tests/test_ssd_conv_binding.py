"""The binding's checks of the state space dual layer with its convolution and of the group norm, on host tensors: what
it takes, what it refuses, and for which argument."""
import pytest

torch = pytest.importorskip("torch")

CPU, F32, BF16 = torch.device("cpu"), torch.float32, torch.bfloat16
ROW = 4 * 8 + 2 * 2 * 8      # 4 heads of 8 channels, 2 groups of 8 states


@pytest.fixture(scope="module")
def b():
    from selective_state_space_32_amd import ssmscan
    return ssmscan


def rows(b, t, lead, width):
    return b._rows(t, "v", torch.Size(lead), width, F32, CPU)


@pytest.mark.parametrize("lead,source", [((2, 5), (1, 1)), ((2, 5), (2, 1)), ((2, 5), (1, 5)), ((3,), (1,)), ((1, 5), (1, 1)),
                                         ((2, 1), (1, 1)), ((2, 3, 5), (2, 1, 5)), ((2, 3, 5), (1, 1, 1))])
@pytest.mark.parametrize("width", [1, 2, 24])
def test_broadcast_rows_are_refused(b, lead, source, width):
    """One row for several tokens or sequences is not a row of each: a kernel that took it for packed ones would
    read past the tensor."""
    t = torch.zeros(*source, width).expand(*lead, width)
    with pytest.raises(ValueError, match="rows must be contiguous and evenly spaced"):
        rows(b, t, lead, width)


@pytest.mark.parametrize("strides", [(10, 1), (19, 1), (0, 1), (20, 2), (20, 0)])
def test_rows_that_overlap_are_refused(b, strides):
    with pytest.raises(ValueError, match="evenly spaced"):
        rows(b, torch.zeros(200).as_strided((3, 20), strides), (3,), 20)


def test_axes_of_one_have_any_stride(b):
    t = torch.zeros(500)
    assert rows(b, t.as_strided((1, 20), (3, 1)), (1,), 20) == 20
    assert rows(b, t.as_strided((1, 1, 20), (0, 0, 1)), (1, 1), 20) == 20
    assert rows(b, t.as_strided((4, 1, 20), (30, 0, 1)), (4, 1), 20) == 30
    assert rows(b, t.as_strided((1, 4, 20), (7, 30, 1)), (1, 4), 20) == 30
    assert rows(b, t.as_strided((2, 4, 1), (24, 6, 9)), (2, 4), 1) == 6


def layer(**kw):
    z = lambda *s: torch.zeros(*s, dtype=BF16)
    f = lambda *s: torch.zeros(*s)
    v = dict(xbc=z(2, 5, ROW), conv_w=f(ROW, 4), conv_b=f(ROW), dt=z(2, 5, 4), A=f(4), D=f(4), dt_bias=f(4))
    v.update(kw)
    return v


def test_broadcast_inputs_reach_no_entry_point(b):
    z = lambda *s: torch.zeros(*s, dtype=BF16)
    shape = dict(dstate=8, ngroups=2)
    for k, t in (("xbc", z(1, 1, ROW).expand(2, 5, ROW)), ("xbc", z(2, 1, ROW).expand(2, 5, ROW)), ("dt", z(4).expand(2, 5, 4)),
                 ("dt", z(2, 1, 4).expand(2, 5, 4))):
        v = layer(**{k: t})
        for call in (lambda: b.ssd_conv_fwd(**v, **shape), lambda: b.ssd_conv_bwd(z(2, 5, 4, 8), **v, **shape)):
            with pytest.raises(ValueError, match=f"{k}: rows"):
                call()
    for k, t in (("xbc", z(ROW).expand(2, ROW)), ("dt", z(1, 4).expand(2, 4))):
        v = layer(xbc=z(2, ROW), dt=z(2, 4))
        v[k] = t
        for call in (b.ssd_conv_step, b.ssd_conv_step_call):
            with pytest.raises(ValueError, match=f"{k}: rows"):
                call(torch.zeros(2, 4, 8, 8), z(2, 3, ROW), **v, **shape)
    x, w = z(2, 3, 24), torch.zeros(24)
    for gate in (z(24).expand(2, 3, 24), z(2, 1, 24).expand(2, 3, 24), z(1, 3, 24).expand(2, 3, 24)):
        with pytest.raises(ValueError, match="z: rows"):
            b.groupnorm_fwd(x, w, groups=3, z=gate)
        with pytest.raises(ValueError, match="z: rows"):
            b.groupnorm_bwd(x, x, w, None, None, torch.zeros(2, 3, 3), groups=3, z=gate)
