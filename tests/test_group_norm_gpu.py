"""GPU parity of the group normalisation and its backward pass with the float64
oracle, element by element."""
import numpy as np
import pytest

from mamba_ssd_scan_chunked_b200 import inputs as I
from mamba_ssd_scan_chunked_b200 import ssd
from oracle import layer as O
from tests.gpu_util import to_dev, torch
from tests.layer_util import check, check_dict, dev, draw, f64, rows_of, t_dtype

pytestmark = pytest.mark.gpu
F, B = I.F32, I.BF16

CASES = [
    # rows, group size, groups, x, io, y, center, act, weight, bias, extra
    (5, 24, 3, F, F, F, True, "after", True, True, 0),
    (33, 8, 7, F, F, F, False, "before", True, False, 8),            # one lane a group
    (9, 64, 64, F, B, B, False, "before", True, False, 24),          # a head a group
    (7, 256, 5, B, B, B, True, "silu", True, True, 0),
    (6, 264, 3, F, F, F, True, "none", False, True, 0),              # past one vector a lane
    (3, 1024, 2, F, B, F, False, "after", True, True, 8),
    (4, 1032, 3, B, F, B, True, "before", True, True, 0),            # past a warp
    (300, 4096, 1, F, B, B, False, "before", True, False, 40),
    (2, 8192, 2, F, F, F, True, "after", True, True, 0),
    (3, 16384, 1, F, F, F, True, "silu", True, True, 0),             # the largest group
    (2, 12296, 1, B, B, F, False, "none", True, False, 0),
    (1, 4096, 8, F, F, B, True, "none", False, False, 0),
    (700, 40, 11, F, F, F, True, "before", True, True, 0),           # many rows a slot
    (0, 16, 2, F, F, F, False, "none", True, True, 0),
]


def inputs(rows, C, x, io, act, weight, bias, seed):
    return {"x": draw([seed, 0], (rows, C), x, 2.0, 0.5), "weight": draw([seed, 1], (C,), F, 0.3, 1.0) if weight else None,
            "bias": draw([seed, 2], (C,), F, 0.3) if bias else None,
            "z": draw([seed, 3], (rows, C), io) if act in ("after", "before") else None}


def kw(act, G, center):
    return dict(ngroups=G, eps=1e-5, center=center, gate_first=act == "before", activation="silu" if act == "silu" else None)


@pytest.mark.parametrize("rows,gs,G,x,io,y,center,act,weight,bias,extra", CASES)
def test_group_norm_fwd(rows, gs, G, x, io, y, center, act, weight, bias, extra):
    c = inputs(rows, gs * G, x, io, act, weight, bias, 700 + gs)
    z = None if c["z"] is None else rows_of(c["z"], extra)
    got = ssd.group_norm_fwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), z, y_dtype=t_dtype(y), **kw(act, G, center))
    check("y", got, O.group_norm(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["z"]), G, 1e-5, center, act))


@pytest.mark.parametrize("rows,gs,G,x,io,g,center,act,weight,bias,extra", CASES)
def test_group_norm_bwd(rows, gs, G, x, io, g, center, act, weight, bias, extra):
    c = inputs(rows, gs * G, x, io, act, weight, bias, 800 + gs)
    dy = draw([9, gs], (rows, gs * G), io)
    z = None if c["z"] is None else rows_of(c["z"], extra)
    got = ssd.group_norm_bwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), to_dev(dy), z, grad_dtype=t_dtype(g),
                             **kw(act, G, center))
    ref = O.group_norm_bwd(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["z"]), f64(dy), G, 1e-5, center, act)
    ref["dweight"] = ref["dweight"] if weight else None
    ref["dbias"] = ref["dbias"] if bias else None
    check_dict(got, ref)


def test_a_mean_far_above_the_spread():
    """Values of 1000 +- 1: the squares' expanded form would lose them."""
    c = inputs(6, 512, F, F, "none", True, True, 3)
    c["x"] = (c["x"] / 2 + 1000).astype(np.float32)
    got = ssd.group_norm_fwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), ngroups=2, center=True)
    ref = O.group_norm(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), None, 2, 1e-5, True, "none")
    # the mean of 256 values near 1000 is off by a few 2^-24 * 1000 = 6e-5, which moves every
    # difference of the row alike: 4 roundings on its path give 2.4e-4 of the spread
    assert np.abs(got.double().cpu().numpy() - ref).max() <= 4e-4 * 1.5


def test_leading_dimensions_and_zero_rows_of_input():
    t = torch()
    x = t.zeros(2, 3, 64, device="cuda")
    y = ssd.group_norm_fwd(x, None, None, ngroups=2)
    assert y.shape == x.shape and not y.any()          # 0 / sqrt(eps)
    z = t.randn(2, 3, 96, device="cuda")[..., 32:]
    assert ssd.group_norm_fwd(x, None, None, z, ngroups=2).shape == x.shape


def test_a_row_with_infinity_or_nan_leaves_the_others():
    t = torch()
    x = t.randn(9, 96, device="cuda")
    ref = ssd.group_norm_fwd(x, None, None, ngroups=3)
    bad = x.clone()
    bad[4, 40], bad[7, 2] = float("inf"), float("nan")
    got = ssd.group_norm_fwd(bad, None, None, ngroups=3)
    keep = t.ones(9, 3, dtype=t.bool, device="cuda")
    keep[4, 1] = keep[7, 0] = False
    assert t.equal(got.view(9, 3, 32)[keep], ref.view(9, 3, 32)[keep])
    assert got[4, 40].isnan() and got[7, :32].isnan().all()


def test_group_norm_bwd_repeats_bit_for_bit():
    t = torch()
    c = inputs(500, 512, F, B, "before", True, True, 5)
    dy, z = to_dev(draw(6, (500, 512), B)), to_dev(c["z"])
    outs = [ssd.group_norm_bwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), dy, z, ngroups=4) for _ in range(2)]
    for k in outs[0]:
        assert t.equal(outs[0][k], outs[1][k]), k


@pytest.mark.parametrize("rows,gs,G,center,act", [(1, 8, 2047, False, "before"), (3, 16, 4099, True, "after"),
                                                  (2, 8, 7, False, "none"), (5, 264, 601, False, "before")])
def test_few_rows_of_many_groups(rows, gs, G, center, act):
    """An item a slot, slots of the last block without one, and as many groups as share no factor with a block's
    slots; the workspace is of the size asked for and nothing behind it is written."""
    t = torch()
    c = inputs(rows, gs * G, F, F, act, True, True, 900 + G)
    dy, z = draw([9, G], (rows, gs * G), F), dev(c["z"])
    got = ssd.group_norm_fwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), z, **kw(act, G, center))
    check("y", got, O.group_norm(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["z"]), G, 1e-5, center, act))
    need = 2 * 4 * rows * gs * G
    ws = t.full((need + 4096,), 77, dtype=t.uint8, device="cuda")
    got = ssd.group_norm_bwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), to_dev(dy), z, workspace=ws,
                             **kw(act, G, center))
    check_dict(got, O.group_norm_bwd(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["z"]), f64(dy), G, 1e-5, center,
                                     act))
    assert (ws[need:] == 77).all()


@pytest.mark.parametrize("rows,gs,G,x,io,y,center,act,bias,extra", [
    (12001, 64, 3, F, B, B, False, "before", True, 8),                  # 32 slots a block
    (40001, 8, 5, F, F, F, True, "after", True, 0),                     # 256 slots a block
    (2003, 256, 5, B, B, F, True, "silu", True, 0),                     # a warp a slot
    (2001, 264, 3, F, F, F, False, "before", False, 24),                # several slots of two warps
    (701, 1032, 3, B, F, B, True, "after", True, 8),
    (1501, 4096, 1, F, B, B, False, "before", True, 40),                # a slot a block
    (503, 8192, 1, F, F, F, True, "after", True, 16),                   # two vectors a lane backward
    (499, 8192, 2, B, B, B, False, "before", True, 8),
    (501, 16384, 1, F, F, F, False, "before", True, 8),
])
def test_slots_of_several_rows(rows, gs, G, x, io, y, center, act, bias, extra):
    """A slot walks over rows: the steps of x and of the gate's wider rows, the exchange's two halves in turn and
    the sums of dw and db over a slot's rows.  The backward's partial sums tell the slots; the forward has twice
    as many at most."""
    C = gs * G
    parts = ssd.ssd_group_norm_bwd_workspace_size(ssd.GroupNormDesc(rows, C, G, C + extra, 1e-5, 0, 0, 0, 0, 3)) // (8 * C)
    assert 2 * parts < rows and rows % parts
    c = inputs(rows, C, x, io, act, True, bias, 720 + gs)
    z, dy = None if c["z"] is None else rows_of(c["z"], extra), draw([19, gs], (rows, C), io)
    f = {k: f64(v) for k, v in c.items()}
    got = ssd.group_norm_fwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), z, y_dtype=t_dtype(y), **kw(act, G, center))
    check("y", got, O.group_norm(f["x"], f["weight"], f["bias"], f["z"], G, 1e-5, center, act))
    got = ssd.group_norm_bwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), to_dev(dy), z, grad_dtype=t_dtype(y),
                             **kw(act, G, center))
    ref = O.group_norm_bwd(f["x"], f["weight"], f["bias"], f["z"], f64(dy), G, 1e-5, center, act)
    ref["dbias"] = ref["dbias"] if bias else None
    check_dict(got, ref)
