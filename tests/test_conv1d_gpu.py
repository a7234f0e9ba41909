"""GPU parity of the short causal convolution, its token step and its backward
pass with the float64 oracle, element by element."""
import numpy as np
import pytest

from mamba_ssd_scan_chunked_b200 import inputs as I
from mamba_ssd_scan_chunked_b200 import ssd
from oracle import layer as O
from tests.gpu_util import to_dev, torch
from tests.layer_util import check, check_dict, dev, draw, f64, rows_of, t_dtype

pytestmark = pytest.mark.gpu
F, B = I.F32, I.BF16


def case(b, L, D, W, io, state, init, bias, seed):
    return {"x": draw([seed, 0], (b, L, D), io), "weight": draw([seed, 1], (D, W), F, 0.5),
            "bias": draw([seed, 2], (D,), F, 0.5) if bias else None,
            "init": draw([seed, 3], (b, W - 1, D), state) if init else None}


def pieces(a, split):
    return np.split(a, np.cumsum(split)[:-1], -1)


@pytest.mark.parametrize("b,L,split,W,io,y,state,init,bias,act,pad,extra", [
    (2, 37, (24,), 4, F, F, F, True, True, True, None, 0),
    (3, 33, (64, 8, 16), 4, B, B, F, False, True, True, None, 24),       # x, B, C out of wider rows
    (2, 129, (1032, 128, 128), 4, B, F, B, True, True, True, None, 8),   # channels past one block, bf16 state
    (1, 16, (40, 8), 3, B, B, F, True, False, False, None, 0),           # one run of tokens, two outputs
    (2, 17, (16,), 2, F, B, F, True, True, True, None, 16),              # one token into the next run
    (5, 50, (72,), 3, F, F, F, True, True, True, [0, 1, 16, 49, 50], 0),  # padding to the last token and beyond
    (4, 21, (8, 8, 8), 4, B, B, B, False, True, True, [21, 20, 19, -3], 0),
    (3, 300, (520,), 4, F, F, F, True, True, True, [99, 300, 0], 8),
    (2, 1, (16,), 4, B, B, B, True, True, True, None, 0),                # fewer tokens than taps
    (2, 2, (16,), 4, F, F, F, True, True, False, [1, 0], 0),
    (2, 0, (16,), 4, F, F, F, True, True, True, None, 0),                # no tokens: the state goes through
    (0, 5, (16,), 4, F, F, F, False, True, True, None, 0),
])
def test_conv1d_fwd(b, L, split, W, io, y, state, init, bias, act, pad, extra):
    t = torch()
    D = sum(split)
    c = case(b, L, D, W, io, state, init, bias, 100 + L + D)
    x = rows_of(c["x"], extra)
    if pad is not None:                       # what the padding holds is nobody's business
        for i, p in enumerate(pad):
            x[i, :max(p, 0)] = float("nan") if i % 2 else float("inf")
    got, final = ssd.conv1d_fwd(x, dev(c["weight"]), dev(c["bias"]), dev(c["init"]), split=split,
                                activation="silu" if act else None, y_dtype=t_dtype(y), state_dtype=t_dtype(state),
                                pad_left=None if pad is None else t.tensor(pad, dtype=t.int32, device="cuda"))
    ref, fref = O.conv1d(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["init"]), pad, act)
    assert len(got) == len(split)
    for i, (g, r) in enumerate(zip(got, pieces(ref, split))):
        check(f"y{i}", g, r)
    check("final", final, fref)
    if pad is not None:
        for i, p in enumerate(pad):
            assert not got[0][i, :max(p, 0)].any()


@pytest.mark.parametrize("b,split,W,io,y,state,bias,act,extra", [
    (3, (24,), 4, F, F, F, True, True, 0),
    (7, (1032, 64, 64), 4, B, B, B, True, True, 40),
    (2, (16, 8), 3, B, F, F, False, False, 8),
    (1, (8,), 2, F, B, F, True, True, 0),
    (801, (1032, 64, 64), 4, B, B, B, True, True, 8),                   # four sequences a thread, one left over
    (650, (1160,), 3, F, F, F, True, True, 0),
])
def test_conv1d_update_is_the_forward_token_by_token(b, split, W, io, y, state, bias, act, extra):
    D, L = sum(split), 6
    c = case(b, L, D, W, io, state, True, bias, 200 + D)
    ref, fref = O.conv1d(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["init"]), None, act)
    if state == B and io == F:
        pytest.skip("the kept inputs would be rounded")
    st, x = to_dev(c["init"]), rows_of(c["x"], extra)
    for i in range(L):
        got = ssd.conv1d_update(st, x[:, i], dev(c["weight"]), dev(c["bias"]), split=split,
                                activation="silu" if act else None, y_dtype=t_dtype(y))
        for j, (g, r) in enumerate(zip(got, pieces(ref[:, i], split))):
            check(f"y{j} of token {i}", g, r)
    check("state", st, fref)


@pytest.mark.parametrize("b,L,split,W,io,g,state,init,bias,act,dfinal,extra", [
    (2, 37, (24,), 4, F, F, F, True, True, True, True, 0),
    (3, 133, (136, 8, 16), 4, B, B, F, False, True, True, False, 24),
    (2, 300, (264,), 4, F, F, F, True, True, True, True, 8),             # several blocks of tokens
    (1, 16, (40, 8), 3, B, F, B, True, False, False, True, 0),
    (2, 129, (16,), 2, F, B, F, True, True, True, True, 16),             # one token into the next block
    (2, 1, (16,), 4, B, B, B, True, True, True, True, 0),
    (2, 2, (16,), 4, F, F, F, True, True, False, True, 0),
    (2, 0, (16,), 4, F, F, F, True, True, True, True, 0),                # dinit = dfinal
    (0, 5, (16,), 4, F, F, F, False, True, True, False, 0),
])
def test_conv1d_bwd(b, L, split, W, io, g, state, init, bias, act, dfinal, extra):
    t = torch()
    D = sum(split)
    c = case(b, L, D, W, io, state, init, bias, 300 + L + D)
    dy = draw([7, L], (b, L, D), io)
    df = draw([8, L], (b, W - 1, D), state) if dfinal else None
    dx = t.full((b, L, D + extra), 7.0, dtype=t_dtype(g), device="cuda")
    dys = tuple(to_dev(np.ascontiguousarray(p)) for p in pieces(dy, split))
    got = ssd.conv1d_bwd(rows_of(c["x"], extra), dev(c["weight"]), dev(c["bias"]), dys if len(dys) > 1 else dys[0],
                         dev(c["init"]), dev(df), activation="silu" if act else None, dx=dx[..., extra:],
                         state_dtype=t_dtype(state))
    ref = O.conv1d_bwd(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["init"]), f64(dy), f64(df), act)
    if not bias:
        ref["dbias"] = None
    check_dict(got, ref)
    assert (dx[..., :extra] == 7.0).all()      # the other columns of the rows are left alone


def test_conv1d_bwd_repeats_bit_for_bit():
    t = torch()
    c = case(3, 500, 264, 4, B, F, True, True, 9)
    dy = to_dev(draw(10, (3, 500, 264), B))
    outs = [ssd.conv1d_bwd(dev(c["x"]), dev(c["weight"]), dev(c["bias"]), dy, dev(c["init"])) for _ in range(2)]
    for k in outs[0]:
        assert t.equal(outs[0][k], outs[1][k]), k


@pytest.mark.parametrize("b,L,split,W,io,y,state,init,pad,extra", [
    (4, 613, (4104,), 4, F, F, F, True, [1, 31, 33, 613], 0),          # padding beside a run's border, and all of it
    (4, 613, (4104,), 3, F, F, F, True, [64, 612, 0, 611], 8),
    (3, 805, (4096, 128, 128), 4, B, B, F, False, None, 24),            # x, B, C out of wider rows
    (2, 1281, (4104,), 2, B, F, B, True, None, 0),                      # one token into the last run
])
def test_conv1d_fwd_in_runs_of_32_tokens(b, L, split, W, io, y, state, init, pad, extra):
    """As many channels and tokens as take the long runs (75776 threads with runs of 32)."""
    t = torch()
    D = sum(split)
    assert b * -(-L // 32) * (D // 4) >= 148 * 512
    c = case(b, L, D, W, io, state, init, True, 110 + L + W)
    x = rows_of(c["x"], extra)
    if pad is not None:
        for i, p in enumerate(pad):
            x[i, :p] = float("nan") if i % 2 else float("inf")
    got, final = ssd.conv1d_fwd(x, dev(c["weight"]), dev(c["bias"]), dev(c["init"]), split=split, y_dtype=t_dtype(y),
                                state_dtype=t_dtype(state),
                                pad_left=None if pad is None else t.tensor(pad, dtype=t.int32, device="cuda"))
    ref, fref = O.conv1d(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["init"]), pad, True)
    for i, (g, r) in enumerate(zip(got, pieces(ref, split))):
        check(f"y{i}", g, r)
    check("final", final, fref)
    if pad is not None:
        for i, p in enumerate(pad):
            assert not got[0][i, :p].any()


@pytest.mark.parametrize("run,b,L,split,W,io,g,extra", [
    (32, 4, 287, (8200,), 4, F, F, 0),                                  # one token short of the last warp's run
    (32, 3, 353, (8064, 64, 72), 3, B, B, 8),                           # one into it
    (64, 4, 449, (8200,), 4, B, F, 0),
    (64, 4, 511, (8064, 64, 72), 2, F, F, 16),
    (128, 4, 895, (8200,), 4, F, F, 0),
    (128, 4, 897, (8064, 64, 72), 4, B, B, 24),
])
def test_conv1d_bwd_in_runs_of_more_tokens(run, b, L, split, W, io, g, extra):
    """The runs of 32, 64 and 128 tokens a warp, with kept inputs and their gradients; which one a size takes shows
    in the workspace, a row of sums for each four runs."""
    t = torch()
    D = sum(split)
    c = case(b, L, D, W, io, F, True, True, 310 + L)
    need = ssd.ssd_conv1d_bwd_workspace_size(ssd.Conv1dDesc(b, L, D, W, D + extra, D + extra, 0, 0, 0, 0, 0, 1))
    assert need == 4 * D * (W + 1) * b * -(-L // (4 * run))
    dy, df = draw([17, L], (b, L, D), io), draw([18, L], (b, W - 1, D), F)
    dx = t.full((b, L, D + extra), 7.0, dtype=t_dtype(g), device="cuda")
    dys = tuple(to_dev(np.ascontiguousarray(p)) for p in pieces(dy, split))
    call = lambda: ssd.conv1d_bwd(rows_of(c["x"], extra), dev(c["weight"]), dev(c["bias"]), dys, dev(c["init"]), dev(df),
                                  dx=dx[..., extra:])
    got = call()
    check_dict(got, O.conv1d_bwd(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["init"]), f64(dy), f64(df)))
    assert (dx[..., :extra] == 7.0).all()
    first = {k: v.clone() for k, v in got.items()}
    again = call()
    assert all(t.equal(again[k], first[k]) for k in first)


@pytest.mark.parametrize("b,D,W", [(3, 72, 4), (650, 1160, 3), (5, 16, 2)])
def test_conv1d_update_of_a_bf16_state_and_fp32_inputs(b, D, W):
    """y reads the token as it is; the state keeps it rounded once."""
    c = case(b, 1, D, W, F, B, True, True, 210 + D)
    ref, fref = O.conv1d(f64(c["x"]), f64(c["weight"]), f64(c["bias"]), f64(c["init"]))
    st = to_dev(c["init"])
    check("y", ssd.conv1d_update(st, dev(c["x"])[:, 0], dev(c["weight"]), dev(c["bias"])), ref[:, 0])
    check("state", st, fref)
