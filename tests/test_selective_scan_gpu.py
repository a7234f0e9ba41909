"""GPU parity of the selective scan, its token step and its backward pass with
the float64 oracle, element by element."""
import numpy as np
import pytest

from mamba_ssd_scan_chunked_b200 import inputs as I
from mamba_ssd_scan_chunked_b200 import ssd
from oracle import layer as O
from tests.gpu_util import to_dev, torch
from tests.layer_util import check, check_dict, dev, draw, f64, rows_of, t_dtype

pytestmark = pytest.mark.gpu
F, B = I.F32, I.BF16


def case(b, L, D, N, G, io, state, init, gate, skip, seed):
    rng = np.random.default_rng([seed, 9])
    lead = (b, L) if L is not None else (b,)
    return {"x": draw([seed, 0], lead + (D,), io), "dt_raw": draw([seed, 1], lead + (D,), io),
            "dt_bias": I.to_storage(np.log(np.expm1(rng.uniform(1e-3, 1e-1, D))), F) if skip else None,
            "A": I.to_storage(-np.arange(1, N + 1) * rng.uniform(0.8, 1.2, (D, N)), F),
            "B": draw([seed, 2], lead + (G, N), io), "C": draw([seed, 3], lead + (G, N), io),
            "D": draw([seed, 4], (D,), F) if skip else None,
            "z": draw([seed, 5], lead + (D,), io) if gate else None,
            "init": draw([seed, 6], (b, D, N), state, 0.5) if init else None}


def on_gpu(c, extra=0):
    d = {k: dev(v) for k, v in c.items()}
    if c["z"] is not None:
        d["z"] = rows_of(c["z"], extra)
    return d


def args(d):
    return [d[k] for k in ("x", "dt_raw", "dt_bias", "A", "B", "C", "D")]


@pytest.mark.parametrize("b,L,D,N,G,io,y,state,init,gate,skip,pad,extra", [
    (2, 37, 24, 16, 1, F, F, F, True, True, True, None, 0),
    (2, 70, 72, 16, 1, B, B, F, False, True, True, None, 24),
    (1, 300, 136, 8, 1, F, F, F, True, False, True, None, 0),
    (2, 33, 48, 24, 2, B, F, B, True, True, True, None, 8),              # padded states, two groups
    (1, 65, 16, 64, 2, F, F, F, True, True, True, None, 0),
    (2, 40, 24, 128, 1, B, B, F, True, False, False, None, 0),           # a warp of states a channel
    (1, 20, 16, 136, 1, F, F, F, True, True, True, None, 0),             # more states than one round of lanes
    (1, 19, 8, 256, 1, F, F, F, False, True, True, None, 0),
    (1, 1500, 8, 16, 1, F, F, F, True, True, True, None, 0),             # long: few channels, many tokens
    (1, 2100, 40, 40, 1, B, F, F, True, True, True, None, 0),
    (4, 50, 40, 16, 1, F, F, F, True, True, True, [0, 1, 49, 50], 0),
    (3, 700, 24, 16, 1, F, B, F, False, True, True, [699, 64, -1], 8),
    (75, 20, 264, 16, 1, B, B, F, True, True, True, None, 8),            # more blocks than two for every SM
    (80, 9, 136, 24, 1, F, F, F, True, False, True, None, 0),
    (2, 1, 16, 16, 1, B, B, B, True, True, True, None, 0),
    (2, 0, 16, 16, 1, F, F, F, True, True, True, None, 0),
    (0, 4, 16, 16, 1, F, F, F, False, False, True, None, 0),
])
def test_selective_scan_fwd(b, L, D, N, G, io, y, state, init, gate, skip, pad, extra):
    t = torch()
    c = case(b, L, D, N, G, io, state, init, gate, skip, 400 + L + N)
    d = on_gpu(c, extra)
    if pad is not None:
        for i, p in enumerate(pad):
            for k in ("x", "dt_raw", "B", "C", "z"):
                if d[k] is not None:
                    d[k][i, :max(p, 0)] = float("nan") if i % 2 else float("inf")
    got, final = ssd.selective_scan_fwd(*args(d), d["z"], d["init"], y_dtype=t_dtype(y), state_dtype=t_dtype(state),
                                        pad_left=None if pad is None else t.tensor(pad, dtype=t.int32, device="cuda"))
    f = {k: f64(v) for k, v in c.items()}
    ref, fref = O.selective_scan(*args(f), f["z"], f["init"], pad)
    check("y", got, ref)
    check("final", final, fref)


def test_strong_and_vanishing_decays():
    """dt up to 30 (decays that underflow), dt that vanishes, A = 0 and positive A of a few states."""
    c = case(2, 90, 24, 16, 1, F, F, True, False, True, 5)
    rng = np.random.default_rng(6)
    c["dt_raw"][rng.random(c["dt_raw"].shape) < 0.2] = 30.0
    c["dt_raw"][rng.random(c["dt_raw"].shape) < 0.2] = -1e4
    c["A"][:, 3] = 0.0
    c["A"][::2, 5] = 0.01
    d, f = on_gpu(c), {k: f64(v) for k, v in c.items()}
    got, final = ssd.selective_scan_fwd(*args(d), None, d["init"])
    ref, fref = O.selective_scan(*args(f), None, f["init"])
    check("y", got, ref)
    check("final", final, fref)


@pytest.mark.parametrize("b,D,N,G,io,y,state,gate,skip,extra", [
    (3, 24, 16, 1, F, F, F, True, True, 0),
    (5, 272, 16, 2, B, B, F, True, True, 40),
    (2, 16, 24, 1, B, F, F, False, False, 0),
    (2, 24, 128, 1, F, F, F, True, True, 8),
    (1, 8, 200, 1, F, F, F, True, True, 0),
    (9, 40, 8, 1, B, B, F, True, True, 0),
    (531, 264, 16, 1, B, B, F, True, True, 8),                          # four sequences a thread, three left over
    (302, 272, 64, 2, F, F, F, True, True, 0),
])
def test_selective_state_update_is_the_scan_token_by_token(b, D, N, G, io, y, state, gate, skip, extra):
    L = 5
    c = case(b, L, D, N, G, io, state, True, gate, skip, 500 + D)
    f = {k: f64(v) for k, v in c.items()}
    ref, fref = O.selective_scan(*args(f), f["z"], f["init"])
    d = on_gpu(c, extra)
    st = d["init"].clone()
    for i in range(L):
        tok = {k: v[:, i].contiguous() if k in ("x", "dt_raw", "B", "C") else v for k, v in d.items()}
        got = ssd.selective_state_update(st, *args(tok), None if d["z"] is None else d["z"][:, i], y_dtype=t_dtype(y))
        check(f"y of token {i}", got, ref[:, i])
    check("state", st, fref)


@pytest.mark.parametrize("b,D,N", [(4, 40, 16), (3, 24, 256), (600, 264, 8)])
def test_selective_state_update_bf16_state_rounds_once(b, D, N):
    c = case(b, None, D, N, 1, B, B, True, True, True, 11)
    f = {k: f64(v) for k, v in c.items()}
    d = on_gpu(c)
    h, y = O.selective_step(f["init"], f["x"], f["dt_raw"], f["dt_bias"], f["A"], f["B"], f["C"], f["D"], f["z"])
    st = d["init"]
    got = ssd.selective_state_update(st, *args(d), d["z"], y_dtype=torch().float32)
    check("y", got, y)                         # y reads the state before its rounding
    check("state", st, h)


@pytest.mark.parametrize("b,L,D,N,G,io,g,state,init,gate,skip,dfinal,extra", [
    (2, 37, 24, 16, 1, F, F, F, True, True, True, True, 0),
    (2, 70, 72, 16, 1, B, B, F, False, True, True, False, 24),
    (1, 300, 136, 8, 1, F, F, F, True, False, True, True, 0),
    (2, 33, 48, 24, 2, B, F, B, True, True, True, True, 8),
    (1, 65, 16, 64, 2, F, F, F, True, True, True, True, 0),
    (2, 40, 24, 128, 1, B, B, F, True, False, False, True, 0),
    (1, 20, 16, 136, 1, F, F, F, True, True, True, True, 0),
    (1, 19, 8, 256, 1, F, F, F, False, True, True, True, 0),
    (1, 1100, 8, 16, 1, F, F, F, True, True, True, True, 0),
    (2, 16, 200, 16, 1, F, F, F, True, True, True, True, 0),             # one chunk exactly
    (2, 1, 16, 16, 1, B, B, B, True, True, True, True, 0),
    (2, 0, 16, 16, 1, F, F, F, True, True, True, True, 0),
    (0, 4, 16, 16, 1, F, F, F, False, False, True, False, 0),
    (8, 7190, 136, 8, 1, B, B, F, True, True, True, True, 8),            # so many chunks that a block takes two tiles
    (4, 130, 272, 16, 2, F, F, F, True, True, True, True, 0),            # several tiles of channels in two groups
])
def test_selective_scan_bwd(b, L, D, N, G, io, g, state, init, gate, skip, dfinal, extra):
    c = case(b, L, D, N, G, io, state, init, gate, skip, 600 + L + N)
    dy = draw([13, L], (b, L, D), io)
    df = draw([14, L], (b, D, N), state, 0.5) if dfinal else None
    d, f = on_gpu(c, extra), {k: f64(v) for k, v in c.items()}
    got = ssd.selective_scan_bwd(*args(d), to_dev(dy), d["z"], d["init"], dev(df), grad_dtype=t_dtype(g),
                                 state_dtype=t_dtype(state))
    ref = O.selective_scan_bwd(*args(f), f["z"], f["init"], f64(dy), f64(df))
    if not skip:
        ref["ddt_bias"] = ref["dD"] = None
    check_dict(got, ref)


def test_selective_scan_bwd_repeats_bit_for_bit():
    t = torch()
    c = case(2, 100, 136, 16, 1, B, F, True, True, True, 15)
    d, dy = on_gpu(c), to_dev(draw(16, (2, 100, 136), B))
    outs = [ssd.selective_scan_bwd(*args(d), dy, d["z"], d["init"]) for _ in range(2)]
    for k in outs[0]:
        assert t.equal(outs[0][k], outs[1][k]), k


def test_gradients_against_differences_of_the_forward_kernel():
    """Directional differences of the fp32 forward kernel's own outputs, weighted in 64 bits: with a step
    of 2^-6 the second-order term cancels, the third is below 2^-12 of the scale and the outputs' rounding
    (2^-22 of the sum of |y dy|, over 2^-5) below 2^-17: 2^-9 of the scale holds both."""
    t = torch()
    c = case(1, 40, 16, 16, 1, F, F, True, True, True, 21)
    dy, df = draw(22, (1, 40, 16), F), draw(23, (1, 16, 16), F)
    d = on_gpu(c)
    g = ssd.selective_scan_bwd(*args(d), to_dev(dy), d["z"], d["init"], to_dev(df))
    names = ("x", "dt_raw", "dt_bias", "A", "B", "C", "D", "z", "init")
    grads = dict(zip(names, (g[k] for k in ("dx", "ddt_raw", "ddt_bias", "dA", "dB", "dC", "dD", "dz", "dinit_state"))))
    wy, wf = to_dev(dy).double(), to_dev(df).double()

    def loss(e):
        y, f = ssd.selective_scan_fwd(*args(e), e["z"].contiguous(), e["init"])
        return float((y.double() * wy).sum() + (f.double() * wf).sum()), float((y.double() * wy).abs().sum())

    h = 2.0 ** -6
    for i, k in enumerate(names):
        step = t.randn(d[k].shape, generator=t.Generator("cuda").manual_seed(i), device="cuda")
        up, size = loss({**d, k: d[k] + h * step})
        down, _ = loss({**d, k: d[k] - h * step})
        num, ana = (up - down) / (2 * h), float((grads[k].double() * step).sum())
        assert abs(num - ana) <= 2.0 ** -9 * (size + abs(ana)), (k, num, ana, size)


@pytest.mark.parametrize("L,N,pad", [(13, 16, None), (13, 16, [5, 13]), (70, 24, [0, 33]), (900, 16, [0, 450])])
def test_a_state_that_forgets_at_once(L, N, pad):
    """A = -inf, which -exp(a) of a large a is: the state holds its own token's term alone.  Tokens that are
    absent, before the sequence or behind its end in a tile, leave it as it was (dt = 0, decay 1, not 0 x inf);
    so does the sum of dt of a chunk without tokens.  d dt takes A itself, which gives no number there."""
    t = torch()
    c = case(2, L, 24, N, 1, F, F, True, True, True, 31 + L)
    c["A"][:, 2] = -np.inf
    c["A"][::3, 5] = -3e38                                    # finite, and infinite times log2 e
    d, f = on_gpu(c), {k: f64(v) for k, v in c.items()}
    pads = None if pad is None else t.tensor(pad, dtype=t.int32, device="cuda")
    got, final = ssd.selective_scan_fwd(*args(d), d["z"], d["init"], pad_left=pads)
    ref, fref = O.selective_scan(*args(f), f["z"], f["init"], pad)
    check("y", got, ref)
    check("final", final, fref)
    if pad is None:
        dy = draw([33, L], (2, L, 24), F)
        g = ssd.selective_scan_bwd(*args(d), to_dev(dy), d["z"], d["init"])
        with np.errstate(invalid="ignore"):
            ref = O.selective_scan_bwd(*args(f), f["z"], f["init"], f64(dy))
        for k in ("dx", "dz", "dB", "dC", "dA", "dD", "dinit_state"):
            check(k, g[k], ref[k])


def test_a_token_step_of_a_state_that_forgets_at_once():
    c = case(3, None, 24, 16, 1, F, F, True, True, True, 32)
    c["A"][:, 2] = -np.inf
    d, f = on_gpu(c), {k: f64(v) for k, v in c.items()}
    h, y = O.selective_step(f["init"], f["x"], f["dt_raw"], f["dt_bias"], f["A"], f["B"], f["C"], f["D"], f["z"])
    check("y", ssd.selective_state_update(d["init"], *args(d), d["z"]), y)
    check("state", d["init"], h)


@pytest.mark.parametrize("b,D,N,G,io,gate", [
    (475, 264, 8, 1, F, True),                                          # two lanes a channel
    (301, 264, 16, 1, B, True),                                         # four, too few sequences for four a thread
    (91, 528, 24, 2, F, False),
])
def test_token_steps_of_two_sequences_a_thread(b, D, N, G, io, gate):
    """The token step's middle form: fp32 states whose two sequences a thread fill the machine (1184 blocks) and
    whose four do not, or whose lanes are two."""
    K = 1 << (N // 4 - 1).bit_length()
    blocks = lambda n: -(-b // n) * -(-D // (128 // K))
    assert blocks(2) >= 148 * 8 and (K < 4 or blocks(4) < 148 * 8)
    c = case(b, None, D, N, G, io, F, True, gate, True, 510 + D + N)
    d, f = on_gpu(c, 8), {k: f64(v) for k, v in c.items()}
    h, y = O.selective_step(f["init"], f["x"], f["dt_raw"], f["dt_bias"], f["A"], f["B"], f["C"], f["D"], f["z"])
    check("y", ssd.selective_state_update(d["init"], *args(d), d["z"]), y)
    check("state", d["init"], h)


@pytest.mark.parametrize("b,L,D,N,G,io,pad", [
    (1, 700, 24, 128, 1, F, None),
    (2, 697, 16, 128, 2, F, [0, 333]),
    (1, 500, 24, 200, 1, F, None),                                      # tiles of 16 tokens
    (2, 333, 16, 256, 1, F, [332, 17]),
    (1, 701, 40, 72, 1, B, [129]),
])
def test_cut_sequences_of_many_states(b, L, D, N, G, io, pad):
    """More than 64 states in chunks: the summaries of a warp of states a channel."""
    t = torch()
    assert ssd.ssd_selective_scan_workspace_size(ssd.SelectiveDesc(b, L, D, N, G, D, 0, 0, 0)) > 0
    c = case(b, L, D, N, G, io, F, True, True, True, 410 + L + N)
    c["A"] /= 16                                                        # decays that carry from chunk to chunk
    d, f = on_gpu(c, 8), {k: f64(v) for k, v in c.items()}
    if pad is not None:
        for i, p in enumerate(pad):
            for k in ("x", "dt_raw", "B", "C", "z"):
                d[k][i, :p] = float("nan") if i % 2 else float("inf")
    y, final = ssd.selective_scan_fwd(*args(d), d["z"], d["init"], y_dtype=t.float32,
                                      pad_left=None if pad is None else t.tensor(pad, dtype=t.int32, device="cuda"))
    ref, fref = O.selective_scan(*args(f), f["z"], f["init"], pad)
    check("y", y, ref)
    check("final", final, fref)


def test_dt_keeps_its_relative_precision():
    """y = dt where A = 0, x = B = C = 1 of one state: softplus over five decades of dt below 1, around 0 and above.
    The exponential is off by 2^-22 of itself, the polynomial by 2^-23 with its roundings, the sum by 2^-24 and
    dt_raw + dt_bias, exact here, by nothing: 2^-22 + 2^-23 + 2^-24 < 4.2e-7 of dt."""
    t = torch()
    raw = np.concatenate([np.linspace(-80, 30, 4000), np.linspace(-2, 2, 4000), [0.0, -1e-8, 1e-8]]).astype(np.float32)
    raw = np.pad(raw, (0, -len(raw) % 8))
    n = len(raw)
    one, B = t.ones(1, 1, n, device="cuda"), t.zeros(1, 1, 1, 8, device="cuda")
    B[..., 0] = 1.0
    A = t.zeros(n, 8, device="cuda")
    want = O.softplus(raw.astype(np.float64))
    y, _ = ssd.selective_scan_fwd(one, to_dev(raw)[None, None], None, A, B, B, None)
    step = ssd.selective_state_update(t.zeros(1, n, 8, device="cuda"), one[:, 0], to_dev(raw)[None], None, A, B[:, 0],
                                      B[:, 0], None)
    for got in (y[0, 0], step[0]):
        assert (np.abs(got.double().cpu().numpy() - want) <= 4.2e-7 * want).all()
