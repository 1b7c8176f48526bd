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


def test_refusals_name_the_argument(b):
    """(Host tensors that pass every check end in a refusal of the host: each case has to be refused before that,
    for the argument that is wrong.)"""
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt)
    f = lambda *s: torch.zeros(*s)
    shape = dict(dstate=8, ngroups=2)
    refused = [("xbc", z(2, 5, ROW + 1), "rows of 65 values are not 4 heads"), ("xbc", z(5, ROW), r"xbc must be \(batch, L, row\)"),
               ("conv_w", f(ROW, 4, 1), r"conv_w must be \(row, width\)"), ("conv_w", f(ROW - 1, 4), "conv_w: shape"),
               ("conv_b", f(ROW + 1), "conv_b: shape"), ("dt", z(2, 5, 3), "dt: shape"), ("dt", z(2, 4, 4), "dt: shape"),
               ("A", f(4, 1), r"A must be \(heads,\)"), ("A", f(5), "are not 5 heads"), ("D", f(3), "D: shape"),
               ("dt_bias", f(8), "dt_bias: shape"), ("xbc", z(2, ROW, 5).transpose(1, 2), "xbc: rows"),
               ("dt", z(2, 5, 4, 2)[..., 0], "dt: rows"), ("xbc", z(2, 6, ROW)[:, :5], "xbc: rows")]
    for k, t, why in refused:
        for call in (lambda v: b.ssd_conv_fwd(**v, **shape), lambda v: b.ssd_conv_bwd(z(2, 5, 4, 8), **v, **shape)):
            with pytest.raises(ValueError, match=why):
                call(layer(**{k: t}))
    for k, t in (("dt", f(2, 5, 4)), ("A", z(4)), ("conv_w", z(ROW, 4)), ("D", z(4))):
        with pytest.raises(TypeError, match=f"{k}: dtype"):
            b.ssd_conv_fwd(**layer(**{k: t}), **shape)
    with pytest.raises(TypeError, match="must be float32 or bfloat16"):
        b.ssd_conv_fwd(**layer(xbc=z(2, 5, ROW, dt=torch.float16), dt=z(2, 5, 4, dt=torch.float16)), **shape)
    for k, t, why in (("initial_state", f(2, 4, 8, 9), "initial_state: shape"), ("conv_state", z(2, 4, ROW), "conv_state: shape"),
                      ("seq_lens", torch.zeros(3, dtype=torch.int32), "seq_lens must be"),
                      ("seq_lens", torch.zeros(2), "seq_lens must be"), ("y", z(2, 5, 4, 9), "y: shape"),
                      ("last_state", f(2, 4, 8), "last_state: shape"), ("conv_state_out", z(2, 4, ROW), "conv_state_out: shape")):
        with pytest.raises(ValueError, match=why):
            b.ssd_conv_fwd(**layer(), **shape, **{k: t})
    for kw, why in ((dict(dy=z(2, 5, 4, 9)), "dy: shape"), (dict(dlast_state=f(2, 4, 8, 4)), "dlast_state: shape"),
                    (dict(checkpoints=f(8, 8).T[:4]), "checkpoints: must be contiguous")):
        with pytest.raises(ValueError, match=why):
            b.ssd_conv_bwd(**dict(dict(dy=z(2, 5, 4, 8)), **kw), **layer(), **shape)
    step = dict(layer(xbc=z(2, ROW), dt=z(2, 4)), state=f(2, 4, 8, 8), conv_state=z(2, 3, ROW))
    for kw, why in ((dict(xbc=z(2, 1, ROW)), r"xbc must be \(sequences, row\)"), (dict(state=f(2, 4, 8, 7)), "state: shape"),
                    (dict(conv_state=z(2, 2, ROW)), "conv_state: shape"), (dict(dt=z(3, 4)), "dt: shape"),
                    (dict(state=f(2, 4, 8, 16)[..., ::2]), "state: must be contiguous"), (dict(y=z(2, 4, 9)), "y: shape")):
        for call in (b.ssd_conv_step, b.ssd_conv_step_call):
            with pytest.raises(ValueError, match=why):
                call(**dict(step, **kw), **shape)


def test_groupnorm_refusals_name_the_argument(b):
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt)
    f = lambda *s: torch.zeros(*s)
    x, w = z(3, 24), f(24)
    for kw, why in ((dict(groups=5), "not 5 equal groups"), (dict(groups=0), "not 0 equal groups"), (dict(silu=True, z=x), "silu is"),
                    (dict(gate_first=True), "gate_first needs"), (dict(z=z(3, 23)), "z: shape"), (dict(z=z(24, 3).T), "z: rows"),
                    (dict(bias=f(23)), "bias: shape"), (dict(y=z(3, 23)), "y: shape")):
        with pytest.raises(ValueError, match=why):
            b.groupnorm_fwd(x, w, **dict(dict(groups=3), **kw))
    with pytest.raises(TypeError, match="z: dtype"):
        b.groupnorm_fwd(x, w, z=f(3, 24))
    with pytest.raises(ValueError, match="rstd: shape"):
        b.groupnorm_bwd(x, x, w, None, None, f(3, 2), groups=3)
    with pytest.raises(ValueError, match="mean: shape"):
        b.groupnorm_bwd(x, x, w, None, f(3, 2), f(3, 3), groups=3)
    with pytest.raises(ValueError, match="dy: shape"):
        b.groupnorm_bwd(z(3, 25), x, w, None, None, f(3, 3), groups=3)


def test_what_passes_ends_at_the_host(b):
    z = lambda *s: torch.zeros(*s, dtype=BF16)
    with pytest.raises(ValueError, match="not the current GPU"):
        b.ssd_conv_fwd(**layer(), dstate=8, ngroups=2)
    with pytest.raises(ValueError, match="not the current GPU"):
        b.groupnorm_fwd(z(3, 24), torch.zeros(24), groups=3, z=z(3, 40)[:, 3:27])
