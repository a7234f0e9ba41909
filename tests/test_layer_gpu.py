"""The operators around the scan in a run, as a layer makes them: the prompt,
then tokens, then the backward pass; on streams, in graphs, on two workspaces."""
import numpy as np
import pytest

import oracle
from mamba_ssd_scan_chunked_b200 import inputs as I
from mamba_ssd_scan_chunked_b200 import ssd
from oracle import layer as O
from tests.gpu_util import TOL_BF16, TOL_F32, metric, to_dev, to_host64, torch
from tests.layer_util import draw, f64

pytestmark = pytest.mark.gpu
F = I.F32


def mamba2(seed, b=2, L=70, H=4, P=64, G=2, N=64, W=4, io=F):
    """The projection's rows z, x, B, C, dt of a layer, and its parameters."""
    DI, BC = H * P, G * N
    c = {"row": draw([seed, 0], (b, L, 2 * DI + 2 * BC + 8), io), "w": draw([seed, 1], (DI + 2 * BC, W), F, 0.5),
         "bias": draw([seed, 2], (DI + 2 * BC,), F, 0.1), "nw": draw([seed, 3], (DI,), F, 0.1, 1.0),
         **I.draw_head_params(H, seed)}
    return c, (DI, BC, BC), (b, L, H, P, G, N, W)


def test_mamba2_layer_prompt_then_tokens():
    t = torch()
    c, split, (b, L, H, P, G, N, W) = mamba2(1)
    T = 4                                      # the last T tokens come one at a time
    DI, D = split[0], sum(split)
    row, par = to_dev(c["row"]), {k: to_dev(v) for k, v in c.items() if k != "row"}
    cut = lambda r: (r[..., :DI], r[..., DI:DI + D], r[..., DI + D:DI + D + H].contiguous())
    z, xbc, dt = cut(row[:, :L - T].contiguous())

    (x, B, C), conv = ssd.conv1d_fwd(xbc, par["w"], par["bias"], split=split)
    y, state = ssd.chunk_scan_fwd(x.view(b, L - T, H, P), dt, par["dt_bias"], par["A"],
                                  B.view(b, L - T, G, N), C.view(b, L - T, G, N), par["D"], 64)
    outs = [ssd.group_norm_fwd(y.view(b, L - T, DI), par["nw"], None, z, ngroups=G)]
    for i in range(L - T, L):
        z, xbc, dt = cut(row[:, i])
        x, B, C = ssd.conv1d_update(conv, xbc, par["w"], par["bias"], split=split)
        y = ssd.state_update(state, x.view(b, H, P), dt, par["dt_bias"], par["A"], B.view(b, G, N),
                             C.view(b, G, N), par["D"])
        outs.append(ssd.group_norm_fwd(y.view(b, DI), par["nw"], None, z, ngroups=G)[:, None])
    f = {k: f64(v) for k, v in c.items()}
    v, _ = O.conv1d(f["row"][..., DI:DI + D], f["w"], f["bias"])
    xr, Br, Cr = v[..., :DI], v[..., DI:DI + split[1]], v[..., DI + split[1]:]
    yr, sr = oracle.recurrent(xr.reshape(b, L, H, P), f["row"][..., DI + D:DI + D + H], f["dt_bias"], f["A"],
                              Br.reshape(b, L, G, N), Cr.reshape(b, L, G, N), f["D"])
    ref = O.group_norm(yr.reshape(b * L, DI), f["nw"], None, f["row"][..., :DI].reshape(b * L, DI), G, 1e-5, False,
                       "before").reshape(b, L, DI)
    assert metric(to_host64(t.cat(outs, 1)), ref) <= TOL_F32
    assert metric(to_host64(state), sr) <= TOL_F32


def mamba2_backward(row, par, split, dims, dout, ws=None):
    """Forward and backward of the layer's core; the projection's row gets its whole gradient."""
    t = torch()
    b, L, H, P, G, N, W = dims
    DI, D = split[0], sum(split)
    z, xbc, dt = row[..., :DI], row[..., DI:DI + D], row[..., DI + D:DI + D + H].contiguous()
    (x, B, C), _ = ssd.conv1d_fwd(xbc, par["w"], par["bias"], split=split)
    x4, B4, C4 = x.view(b, L, H, P), B.view(b, L, G, N), C.view(b, L, G, N)
    y, _ = ssd.chunk_scan_fwd(x4, dt, par["dt_bias"], par["A"], B4, C4, par["D"], 64)
    gn = ssd.group_norm_bwd(y.view(b, L, DI), par["nw"], None, dout, z, ngroups=G)
    gs = ssd.chunk_scan_bwd(x4, dt, par["dt_bias"], par["A"], B4, C4, par["D"], 64, gn["dx"].view(b, L, H, P))
    drow = t.zeros_like(row)
    dys = (gs["dx"].view(b, L, DI), gs["dB"].view(b, L, -1), gs["dC"].view(b, L, -1))
    gc = ssd.conv1d_bwd(xbc, par["w"], par["bias"], dys, dx=drow[..., DI:DI + D])
    drow[..., :DI] = gn["dz"]
    drow[..., DI + D:DI + D + H] = gs["ddt_raw"]
    return {"drow": drow, "dw": gc["dweight"], "dbias": gc["dbias"], "dnw": gn["dweight"], "dA": gs["dA"]}


def mamba2_backward_oracle(c, split, dims, dout):
    b, L, H, P, G, N, W = dims
    DI, D = split[0], sum(split)
    f = {k: f64(v) for k, v in c.items()}
    row = f["row"]
    z, xbc, dt = row[..., :DI], row[..., DI:DI + D], row[..., DI + D:DI + D + H]
    v, _ = O.conv1d(xbc, f["w"], f["bias"])
    x = v[..., :DI].reshape(b, L, H, P)
    B, C = v[..., DI:DI + split[1]].reshape(b, L, G, N), v[..., DI + split[1]:].reshape(b, L, G, N)
    y, _ = oracle.recurrent(x, dt, f["dt_bias"], f["A"], B, C, f["D"])
    gn = O.group_norm_bwd(y.reshape(b * L, DI), f["nw"], None, z.reshape(b * L, DI), dout.reshape(b * L, DI), G, 1e-5,
                          False, "before")
    gs = oracle.backward(x, dt, f["dt_bias"], f["A"], B, C, f["D"], None, gn["dx"].reshape(b, L, H, P))
    dys = np.concatenate([gs["dx"].reshape(b, L, DI), gs["dB"].reshape(b, L, -1), gs["dC"].reshape(b, L, -1)], -1)
    gc = O.conv1d_bwd(xbc, f["w"], f["bias"], None, dys)
    drow = np.zeros_like(row)
    drow[..., :DI], drow[..., DI:DI + D] = gn["dz"].reshape(b, L, DI), gc["dx"]
    drow[..., DI + D:DI + D + H] = gs["ddt_raw"]
    return {"drow": drow, "dw": gc["dweight"], "dbias": gc["dbias"], "dnw": gn["dweight"], "dA": gs["dA"]}


def test_mamba2_layer_backward():
    c, split, dims = mamba2(2)
    dout = draw(3, (dims[0], dims[1], split[0]), F)
    got = mamba2_backward(to_dev(c["row"]), {k: to_dev(v) for k, v in c.items()}, split, dims, to_dev(dout))
    ref = mamba2_backward_oracle(c, split, dims, f64(dout))
    for k in ref:
        assert metric(to_host64(got[k]), ref[k]) <= TOL_F32, k


def test_mamba2_layer_backward_bf16():
    """In bf16 every tensor between two calls is rounded: four roundings of half a step, 2^-9 rms each,
    reach the projection's gradient through sums of independent signs; the method's bf16 bound covers them."""
    c, split, dims = mamba2(4, io=I.BF16)
    dout = draw(5, (dims[0], dims[1], split[0]), I.BF16)
    got = mamba2_backward(to_dev(c["row"]), {k: to_dev(v) for k, v in c.items()}, split, dims, to_dev(dout))
    ref = mamba2_backward_oracle(c, split, dims, f64(dout))
    for k in ref:
        g = to_host64(got[k])
        assert np.linalg.norm(g - ref[k]) <= TOL_BF16 * np.linalg.norm(ref[k]), k


def selective(seed, b=2, L=50, D=72, N=16, W=4):
    rng = np.random.default_rng([seed, 9])
    return {"row": draw([seed, 0], (b, L, 2 * D), F), "w": draw([seed, 1], (D, W), F, 0.5),
            "bias": draw([seed, 2], (D,), F, 0.1), "dt_raw": draw([seed, 3], (b, L, D), F),
            "dt_bias": I.to_storage(np.log(np.expm1(rng.uniform(1e-3, 1e-1, D))), F),
            "A": I.to_storage(-np.arange(1, N + 1) * rng.uniform(0.8, 1.2, (D, N)), F),
            "B": draw([seed, 4], (b, L, 1, N), F), "C": draw([seed, 5], (b, L, 1, N), F), "D": draw([seed, 6], (D,), F)}


def test_selective_layer_prompt_then_tokens_of_a_padded_batch():
    t = torch()
    b, L, D, T = 2, 50, 72, 3
    c, pad = selective(7, b, L, D), [0, 13]
    d = {k: to_dev(v) for k, v in c.items()}
    pads = t.tensor(pad, dtype=t.int32, device="cuda")
    prompt = d["row"][:, :L - T].contiguous()
    xr, z = d["row"][..., :D], d["row"][..., D:]
    x, conv = ssd.conv1d_fwd(prompt[..., :D], d["w"], d["bias"], pad_left=pads)
    cut = lambda k, s: d[k][:, s].contiguous()
    p = slice(0, L - T)
    y, state = ssd.selective_scan_fwd(x, cut("dt_raw", p), d["dt_bias"], d["A"], cut("B", p), cut("C", p), d["D"],
                                      prompt[..., D:], pad_left=pads)
    outs = [y]
    for i in range(L - T, L):
        x = ssd.conv1d_update(conv, xr[:, i], d["w"], d["bias"])
        outs.append(ssd.selective_state_update(state, x, cut("dt_raw", i), d["dt_bias"], d["A"], cut("B", i),
                                               cut("C", i), d["D"], z[:, i])[:, None])
    f = {k: f64(v) for k, v in c.items()}
    v, _ = O.conv1d(f["row"][..., :D], f["w"], f["bias"], None, pad)
    ref, sref = O.selective_scan(v, f["dt_raw"], f["dt_bias"], f["A"], f["B"], f["C"], f["D"], f["row"][..., D:], None, pad)
    assert metric(to_host64(t.cat(outs, 1)), ref) <= TOL_F32
    assert metric(to_host64(state), sref) <= TOL_F32


def training_pass(d, dout, keep):
    """conv, scan and norm forward, then back; every output in `keep`."""
    D = d["w"].shape[0]
    xr, z = d["row"][..., :D], d["row"][..., D:]
    x, _ = ssd.conv1d_fwd(xr, d["w"], d["bias"])
    y, _ = ssd.selective_scan_fwd(x, d["dt_raw"], d["dt_bias"], d["A"], d["B"], d["C"], d["D"], z)
    gn = ssd.group_norm_bwd(y, None, None, dout, ngroups=3, center=True)
    gs = ssd.selective_scan_bwd(x, d["dt_raw"], d["dt_bias"], d["A"], d["B"], d["C"], d["D"], gn["dx"], z)
    gc = ssd.conv1d_bwd(xr, d["w"], d["bias"], gs["dx"])
    keep.update({"n." + k: v for k, v in gn.items() if v is not None})
    keep.update({"s." + k: v for k, v in gs.items() if v is not None})
    keep.update({"c." + k: v for k, v in gc.items() if v is not None})


def test_training_pass_in_graphs_that_share_the_pool():
    """Two captured passes over different inputs, replayed in turn, and an eager pass between them."""
    t = torch()
    sets = [{k: to_dev(v) for k, v in selective(30 + i).items()} for i in range(2)]
    douts = [to_dev(draw(40 + i, (2, 50, 72), F)) for i in range(2)]
    eager = [{}, {}]
    for d, g, e in zip(sets, douts, eager):
        training_pass(d, g, e)
    t.cuda.synchronize()
    want = [{k: v.clone() for k, v in e.items()} for e in eager]
    graphs, outs, pool = [], [{}, {}], t.cuda.graph_pool_handle()
    for d, g, o in zip(sets, douts, outs):
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, pool=pool):
            training_pass(d, g, o)
        graphs.append(graph)
    for _ in range(2):
        for graph, o, w in zip(graphs, outs, want):
            for v in o.values():
                v.zero_()
            graph.replay()
            t.cuda.synchronize()
            for k in w:
                assert t.equal(o[k], w[k]), k
        again = {}
        training_pass(sets[0], douts[0], again)
        assert all(t.equal(again[k], want[0][k]) for k in again)


def test_training_passes_on_two_streams_at_once():
    t = torch()
    sets = [{k: to_dev(v) for k, v in selective(50 + i, 2, 200, 264).items()} for i in range(2)]
    douts = [to_dev(draw(60 + i, (2, 200, 264), F)) for i in range(2)]
    want = [{}, {}]
    for d, g, w in zip(sets, douts, want):
        training_pass(d, g, w)
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(3):
        outs = [{}, {}]
        for d, g, o, s in zip(sets, douts, outs, streams):
            with t.cuda.stream(s):
                training_pass(d, g, o)
        t.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(t.equal(o[k], w[k]) for k in w)


def test_stream_argument_owns_what_the_call_allocates():
    """A call given a stream allocates its workspace for that stream: work of the current stream that
    follows at once does not get the same memory."""
    t = torch()
    d = {k: to_dev(v) for k, v in selective(70, 2, 400, 264).items()}
    dy = to_dev(draw(71, (2, 400, 264), F))
    call = lambda **kw: ssd.selective_scan_bwd(d["row"][..., :264].contiguous(), d["dt_raw"], d["dt_bias"], d["A"],
                                               d["B"], d["C"], d["D"], dy, **kw)
    want = call()
    s = t.cuda.Stream()
    t.cuda.synchronize()
    got = call(stream=s)
    junk = [t.full((1 << 20,), float("nan"), device="cuda") for _ in range(40)]
    raw = call(stream=s.cuda_stream)
    t.cuda.synchronize()
    del junk
    for k in want:
        if want[k] is not None:
            assert t.equal(got[k], want[k]) and t.equal(raw[k], want[k]), k


def test_a_given_stream_waits_for_inputs_made_just_before_and_keeps_them():
    """The inputs are written behind 20 ms of other work of the current stream and dropped after the call:
    the given stream reads what that work made, not what lay there before, and no later tensor of the
    current stream gets their memory while it reads."""
    t = torch()
    d = {k: to_dev(v) for k, v in selective(72, 2, 400, 264).items()}
    z = d["row"][..., 264:]
    par = [d["dt_bias"], d["A"], d["B"], d["C"], d["D"]]
    want = ssd.selective_scan_fwd(d["row"][..., :264].contiguous(), d["dt_raw"], *par, z)
    for s in (t.cuda.Stream(), t.cuda.Stream().cuda_stream):
        t.cuda.synchronize()
        t.cuda._sleep(40_000_000)
        x = d["row"][..., :264].contiguous()
        dt = d["dt_raw"] + 0.0
        got = ssd.selective_scan_fwd(x, dt, *par, z, stream=s)
        del x, dt
        junk = [t.full((2, 400, 264), float("nan"), device="cuda") for _ in range(8)]
        t.cuda.synchronize()
        del junk
        assert t.equal(got[0], want[0]) and t.equal(got[1], want[1])


def test_a_workspace_given_is_used_and_nothing_behind_it_is_written():
    t = torch()
    d = {k: to_dev(v) for k, v in selective(80).items()}
    x = d["row"][..., :72].contiguous()
    dy = to_dev(draw(81, (2, 50, 72), F))
    need = ssd.ssd_selective_scan_bwd_workspace_size(ssd.SelectiveDesc(2, 50, 72, 16, 1, 72, 0, 0, 0))
    big = t.full((need + 4096,), 77, dtype=t.uint8, device="cuda")
    a = ssd.selective_scan_bwd(x, d["dt_raw"], d["dt_bias"], d["A"], d["B"], d["C"], d["D"], dy)
    b = ssd.selective_scan_bwd(x, d["dt_raw"], d["dt_bias"], d["A"], d["B"], d["C"], d["D"], dy, workspace=big)
    t.cuda.synchronize()
    assert (big[need:] == 77).all() and (big[:need] != 77).any()
    assert all(t.equal(a[k], b[k]) for k in a if a[k] is not None)


def test_outputs_that_are_given_are_written_and_returned():
    t = torch()
    d = {k: to_dev(v) for k, v in selective(90).items()}
    x, z = d["row"][..., :72], d["row"][..., 72:]
    want, kept = ssd.conv1d_fwd(x, d["w"], d["bias"], split=(40, 32))
    ys = (t.empty(2, 50, 40, device="cuda"), t.empty(2, 50, 32, device="cuda"))
    final = t.empty_like(kept)
    got, f = ssd.conv1d_fwd(x, d["w"], d["bias"], split=(40, 32), y=ys, final_state=final)
    assert got[0] is ys[0] and got[1] is ys[1] and f is final
    assert t.equal(ys[0], want[0]) and t.equal(ys[1], want[1]) and t.equal(final, kept)
    assert ssd.conv1d_fwd(x, d["w"], d["bias"], want_final_state=False)[1] is None
    y1 = t.empty(2, 72, device="cuda")
    assert ssd.conv1d_update(kept.clone(), x[:, 0], d["w"], d["bias"], y=y1) is y1

    scan = (x.contiguous(), d["dt_raw"], d["dt_bias"], d["A"], d["B"], d["C"], d["D"], z)
    want, state = ssd.selective_scan_fwd(*scan)
    y, final = t.empty_like(want, dtype=t.bfloat16), t.empty_like(state)
    got, f = ssd.selective_scan_fwd(*scan, y=y, final_state=final)
    assert got is y and f is final and t.equal(y, want.bfloat16()) and t.equal(final, state)
    assert ssd.selective_scan_fwd(*scan, want_final_state=False)[1] is None
    y = t.empty(2, 50, 72, device="cuda")
    assert ssd.group_norm_fwd(want, None, None, z, ngroups=3, y=y) is y
    assert t.equal(y, ssd.group_norm_fwd(want, None, None, z, ngroups=3))


def test_calls_without_the_optional_gradients():
    """dinit, the norm's weight and bias, dt_bias and D left out give the others unchanged."""
    t = torch()
    d = {k: to_dev(v) for k, v in selective(91).items()}
    x, dy = d["row"][..., :72].contiguous(), to_dev(draw(92, (2, 50, 72), F))
    a = ssd.conv1d_bwd(x, d["w"], d["bias"], dy)
    b = ssd.conv1d_bwd(x, d["w"], d["bias"], dy, want_dinit=False)
    assert b["dinit_state"] is None and all(t.equal(a[k], b[k]) for k in ("dx", "dweight", "dbias"))
    zero = t.zeros(72, device="cuda")
    a = ssd.selective_scan_bwd(x, d["dt_raw"], zero, d["A"], d["B"], d["C"], zero, dy)
    b = ssd.selective_scan_bwd(x, d["dt_raw"], None, d["A"], d["B"], d["C"], None, dy, want_dinit=False)
    assert b["ddt_bias"] is None and b["dD"] is None and b["dinit_state"] is None
    assert all(t.equal(a[k], b[k]) for k in ("dx", "ddt_raw", "dA", "dB", "dC"))
    one = t.ones(72, device="cuda")
    a = ssd.group_norm_bwd(x, one, zero, dy, ngroups=3)
    b = ssd.group_norm_bwd(x, None, None, dy, ngroups=3)
    assert b["dweight"] is None and b["dbias"] is None and t.equal(a["dx"], b["dx"])


def test_the_last_tokens_of_long_rows_as_a_steps_inputs():
    """x and z of a token step cut out of a prompt's rows without a copy: 2^24 and more elements from one
    sequence to the next."""
    t = torch()
    b, L, D, N = 3, 2049, 72, 16
    c = selective(95, b, 1, D, N)
    d = {k: to_dev(v) for k, v in c.items()}
    rows = t.full((b, L, 8200), float("nan"), device="cuda")
    rows[:, -1, :2 * D] = d["row"][:, 0]
    x, z = rows[:, -1, :D], rows[:, -1, D:2 * D]
    assert x.stride(0) > 1 << 24
    kept, state = t.randn(b, 3, D, device="cuda"), t.randn(b, D, N, device="cuda")
    par = [d["dt_raw"][:, 0].contiguous(), d["dt_bias"], d["A"], d["B"][:, 0].contiguous(), d["C"][:, 0].contiguous(), d["D"]]
    outs = []
    for xs, zs in ((x, z), (x.contiguous(), z.contiguous())):
        k, h = kept.clone(), state.clone()
        v = ssd.conv1d_update(k, xs, d["w"], d["bias"])
        y = ssd.selective_state_update(h, v, *par, zs)
        outs.append((k, v, h, y, ssd.group_norm_fwd(y, None, None, zs, ngroups=3)))
        assert all(o.isfinite().all() for o in outs[-1])
    assert all(t.equal(a, b) for a, b in zip(*outs))


def test_a_convolution_and_a_norm_past_32_bits():
    """2^32 elements and more of x and y (bf16, 8.6 GB each): the last tokens as a call of their own gives them."""
    t = torch()
    b, L, D = 2, (1 << 18) + 37, 8200
    assert b * L * D > 1 << 32
    gen = t.Generator("cuda").manual_seed(3)
    x = t.empty(b, L, D, dtype=t.bfloat16, device="cuda").normal_(generator=gen)
    w, bias = t.randn(D, 4, device="cuda", generator=gen), t.randn(D, device="cuda", generator=gen)
    y, kept = ssd.conv1d_fwd(x, w, bias)
    tail = x[1:, -40:].contiguous()
    want, wkept = ssd.conv1d_fwd(tail, w, bias, x[1:, -43:-40].float().contiguous())
    assert t.equal(y[1:, -40:], want) and t.equal(kept[1:], wkept)
    g = ssd.conv1d_bwd(x, w, bias, y)["dx"]
    own = ssd.conv1d_bwd(tail, w, bias, want, x[1:, -43:-40].float().contiguous())["dx"]
    assert t.equal(g[1:, -40:], own)
    del g
    n = ssd.group_norm_fwd(x, bias, None, y, ngroups=5, y=t.empty_like(x))
    assert t.equal(n[1:, -40:], ssd.group_norm_fwd(tail, bias, None, want, ngroups=5))


def test_a_selective_scan_past_32_bits():
    """64 x 8192 tokens x 8192 channels, 256 states: 2^32 elements of x, dt and y, the same sequence in every
    place of the batch."""
    t = torch()
    b, L, D, N = 64, 8192, 8192, 256
    gen = t.Generator("cuda").manual_seed(4)
    one = lambda *s: t.empty(s, dtype=t.bfloat16, device="cuda").normal_(generator=gen)
    x, dt, B, C = one(1, L, D), one(1, L, D), one(1, L, 1, N), one(1, L, 1, N)
    A = -t.rand(D, N, device="cuda", generator=gen) - 0.1
    want, state = ssd.selective_scan_fwd(x, dt, None, A, B, C, None)
    y, final = ssd.selective_scan_fwd(*(v.expand(b, *v.shape[1:]).contiguous() for v in (x, dt)), None, A,
                                      *(v.expand(b, *v.shape[1:]).contiguous() for v in (B, C)), None)
    for i in (0, 31, 63):
        assert t.equal(y[i], want[0]) and t.equal(final[i], state[0])


def test_a_given_stream_inside_a_captured_fork():
    """A capture forked to the given stream: the wait becomes an edge of the graph, and replays repeat the result."""
    t = torch()
    d = {k: to_dev(v) for k, v in selective(96).items()}
    x, z = d["row"][..., :72], d["row"][..., 72:]
    want, kept = ssd.conv1d_fwd(x, d["w"], d["bias"])
    gated = ssd.group_norm_fwd(want, None, None, z, ngroups=3)
    side, graph = t.cuda.Stream(), t.cuda.CUDAGraph()
    t.cuda.synchronize()
    with t.cuda.graph(graph):
        main = t.cuda.current_stream()
        side.wait_stream(main)
        y, k = ssd.conv1d_fwd(x, d["w"], d["bias"], stream=side)
        n = ssd.group_norm_fwd(y, None, None, z, ngroups=3, stream=side)
        main.wait_stream(side)
    for _ in range(2):
        for v in (y, k, n):
            v.zero_()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(y, want) and t.equal(k, kept) and t.equal(n, gated)
