"""The layer operators around the scan, as they are measured: their cases, inputs,
plain forms and the calls of the framework that compute the same.

Three operators, each for prompts, for training and for single tokens:

conv   the short causal convolution over the tokens of every channel, with SiLU, whose
       outputs go to the scan as separate x, B and C
scan   the selective scan with a decay of its own per channel and state,
       h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,  y_t = (C_t . h_t + D x_t) silu(z_t)
norm   the group normalisation of the scan's output, channels last, with its SiLU gate

Where ``own`` is false ``run`` computes them with elementary torch operations in 32
bits; where it is true it makes the calls of ``mamba_ssd_scan_chunked_b200.ssd``.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"


def _t(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def _size(name):
    return 2 if name == BF16 else 4


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _conv(kind, b, L, channels, B, C, width, row, io, state, init, pad, silu, name=None):
    """row: elements of the row that the channels are a slice of (the projection's output)."""
    c = {"op": "conv", "kind": kind, "batch": b, "seqlen": L, "channels": channels, "B": B, "C": C, "width": width,
         "row": row, "io": io, "state": state, "init": init, "pad": pad, "silu": silu}
    return dict(c, name=name) if name else c


def _scan(kind, b, L, channels, N, G, io, state, init, pad, gate, row, name=None):
    """row: elements of the row that the gate z is a slice of."""
    c = {"op": "scan", "kind": kind, "batch": b, "seqlen": L, "channels": channels, "dstate": N, "groups": G, "io": io,
         "state": state, "init": init, "pad": pad, "gate": gate, "row": row}
    return dict(c, name=name) if name else c


def _norm(kind, rows, channels, G, x, io, center, gate, bias, row, name=None):
    """gate: "before" (the gated input is normalised), "after", "silu" (no z: SiLU of the result) or "none"."""
    c = {"op": "norm", "kind": kind, "rows": rows, "channels": channels, "groups": G, "x": x, "io": io,
         "center": center, "gate": gate, "bias": bias, "row": row}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the 1.3B-shaped layer (4 x 2048 tokens, 64 heads x 64, state 128, one group): x, B and C
        # cut out of the projection's rows of z, x, B, C and dt
        _conv("prompt", 4, 2048, 4352, 128, 128, 4, 8512, BF16, F32, False, False, True, "conv_prompt_layer"),
        # a left-padded batch of odd lengths that continues from kept states, in full precision
        _conv("prompt", 5, 1237, 1544, 0, 0, 3, 1544, F32, F32, True, True, True, "conv_prompt_padded"),
        # a step of 256 sequences, 128 heads x 64 and 8 groups of state 128
        _conv("token", 256, 1, 10240, 1024, 1024, 4, 18560, BF16, BF16, True, False, True, "conv_token"),
        # the training step of the 1.3B-shaped layer: the scan's three gradients back to the projection's rows
        _conv("train", 4, 2048, 4352, 128, 128, 4, 8512, BF16, F32, False, False, True, "conv_train"),
        # a selective layer of the same width, state 16, gated by its half of the projection's rows
        _scan("prompt", 4, 2048, 4096, 16, 1, BF16, F32, False, False, True, 8192, "scan_prompt_layer"),
        # one long prompt: few channels for the machine, many tokens
        _scan("prompt", 1, 16384, 2048, 16, 1, BF16, F32, False, False, True, 4096, "scan_prompt_long"),
        # a small left-padded batch of odd sizes in full precision, from kept states
        _scan("prompt", 3, 777, 520, 24, 1, F32, F32, True, True, False, 520, "scan_prompt_padded"),
        # a step of 256 sequences
        _scan("token", 256, 1, 8192, 16, 1, BF16, F32, True, False, True, 16384, "scan_token"),
        # a training step of the selective layer
        _scan("train", 2, 2048, 4096, 16, 1, BF16, F32, False, False, True, 8192, "scan_train"),
        # the 1.3B-shaped layer's output (in 32 bits, as the scan writes it), gated, one group
        _norm("prompt", 8192, 4096, 1, F32, BF16, False, "before", False, 8512, "norm_prompt_layer"),
        # a step of a few sequences, where only latency counts
        _norm("prompt", 8, 8192, 8, BF16, BF16, True, "after", True, 8192, "norm_token"),
        # the training step of the 1.3B-shaped layer, 8 groups
        _norm("train", 8192, 4096, 8, F32, BF16, False, "before", False, 8512, "norm_train_layer"),
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return min(hi // step, max(-(-lo // step), int(v / step))) * step


def draw(rng):
    op = rng.choice(("conv", "scan", "norm"))
    kind = rng.choice(("prompt", "train") if op == "norm" else ("prompt", "token", "train"))
    io = rng.choice((BF16, BF16, F32))
    flag = lambda: rng.random() < 0.5   # noqa: E731
    if op == "norm":
        size = rng.choice((_between(rng, 8, 8192, 8), 64, 512, 1024, 2048, 4096))
        groups = _between(rng, 1, max(1, 16384 // size))
        channels = size * groups
        rows = _between(rng, 1, max(1, min(16384, 8192 * 4096 // channels)))
        gate = rng.choice(("before", "before", "after", "silu", "none"))
        return _norm(kind, rows, channels, groups, rng.choice((F32, io)), io, flag(), gate, flag(),
                     channels + 8 * rng.randrange(0, 65))
    if op == "conv":
        channels = _between(rng, 64, 10240, 8)
        B = C = 8 * rng.randrange(1, channels // 24 + 1) if flag() else 0
        row = channels + 8 * rng.randrange(0, 513)
        width = rng.choice((2, 3, 4, 4))
        if kind == "token":
            return _conv(kind, _between(rng, 1, 512), 1, channels, B, C, width, row, io, rng.choice((F32, io)), True,
                         False, flag())
        tokens = min(16384, 8192 * 4352 // channels)
        b = _between(rng, 1, 8)
        return _conv(kind, b, _between(rng, 1, max(1, tokens // b)), channels, B, C, width, row, io, F32, flag(),
                     kind == "prompt" and flag(), flag())
    N = rng.choice((8, 16, 16, 24, 32, 64, 128))
    G = rng.choice((1, 1, 2, 4))
    channels = _between(rng, 64, 4096, 8 * G)
    gate = flag()
    row = channels + 8 * rng.randrange(0, 513)
    if kind == "token":
        b = _between(rng, 1, max(1, min(512, 256 * 8192 * 16 // (channels * N))))
        return _scan(kind, b, 1, channels, N, G, io, rng.choice((F32, io)), True, False, gate, row)
    most = (8192 if kind == "prompt" else 4096) * 4096 * 16 // (channels * N)
    b = _between(rng, 1, 8)
    return _scan(kind, b, _between(rng, 1, max(1, min(8192, most // b))), channels, N, G, io, F32, flag(),
                 kind == "prompt" and flag(), gate, row)


def work(case):
    """Each input read once, each output written once; flops with an exp as one."""
    e = _size(case["io"])
    if case["op"] == "norm":
        n, ex = case["rows"] * case["channels"], _size(case["x"])
        z = case["gate"] in ("before", "after")
        par = 4 * case["channels"] * (2 if case["bias"] else 1)
        if case["kind"] == "prompt":
            return {"bytes": n * (ex + e + (e if z else 0)) + par, "flops": n * (12 if z else 8)}
        return {"bytes": n * (ex + 2 * e + (2 * e if z else 0)) + 2 * par, "flops": n * (28 if z else 20)}
    b, L, D = case["batch"], case["seqlen"], case["channels"]
    tok, es = b * L, _size(case["state"])
    if case["op"] == "conv":
        W = case["width"]
        par, keep = 4 * D * (W + 1), b * (W - 1) * D * es
        if case["kind"] == "train":
            return {"bytes": tok * D * 3 * e + 2 * par + keep * ((2 if case["init"] else 0) + 1),
                    "flops": tok * D * (6 * W + 12)}
        return {"bytes": tok * D * 2 * e + par + keep * ((1 if case["init"] else 0) + 1), "flops": tok * D * (2 * W + 4)}
    N, G = case["dstate"], case["groups"]
    par, keep = 4 * D * (N + 2), b * D * N * es
    gate = 1 if case["gate"] else 0
    if case["kind"] == "train":
        return {"bytes": tok * (D * e * (5 + 2 * gate) + 4 * G * N * e) + 2 * par + keep * ((2 if case["init"] else 0) + 1),
                "flops": tok * D * (24 * N + 12)}
    return {"bytes": tok * (D * e * (3 + gate) + 2 * G * N * e) + par + keep * ((1 if case["init"] else 0) + 1),
            "flops": tok * D * (7 * N + 10)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(shape, dtype, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(_t(dtype))

    def uniform(shape, lo, hi):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    io = case["io"]
    s = {"case": case}
    if case["op"] == "norm":
        rows, D = case["rows"], case["channels"]
        s["x"] = normal((rows, D), case["x"], 2.0) + 0.5
        s["z"] = normal((rows, case["row"]), io)[:, case["row"] - D:] if case["gate"] in ("before", "after") else None
        s["weight"] = 1.0 + normal((D,), F32, 0.1)
        s["bias"] = normal((D,), F32, 0.1) if case["bias"] else None
        s["eps"] = 1e-5
        if case["kind"] == "train":
            s["dy"] = normal((rows, D), io)
        return s
    b, L, D = case["batch"], case["seqlen"], case["channels"]
    token = case["kind"] == "token"
    lead = (b,) if token else (b, L)
    if case["op"] == "conv":
        W, cut = case["width"], case["row"] - D
        s["x"] = normal(lead + (case["row"],), io)[..., cut:]
        s["weight"] = uniform((D, W), -W ** -0.5, W ** -0.5)
        s["bias"] = uniform((D,), -W ** -0.5, W ** -0.5)
        s["split"] = (D - case["B"] - case["C"], case["B"], case["C"]) if case["B"] else (D,)
        s["init"] = normal((b, W - 1, D), case["state"]) if case["init"] else None
        if case["kind"] == "train":
            s["dy"] = [normal(lead + (n,), io) for n in s["split"]]
            s["dfinal"] = normal((b, W - 1, D), case["state"])
    else:
        N, G = case["dstate"], case["groups"]
        s["x"] = normal(lead + (D,), io)
        s["dt_raw"] = normal(lead + (D,), io)
        s["dt_bias"] = torch.log(torch.expm1(uniform((D,), 1e-3, 1e-1)))
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * uniform((D, N), 0.8, 1.2)
        s["B"], s["C"] = normal(lead + (G, N), io), normal(lead + (G, N), io)
        s["D"] = normal((D,), F32)
        s["z"] = normal(lead + (case["row"],), io)[..., case["row"] - D:] if case["gate"] else None
        s["init"] = normal((b, D, N), case["state"], 0.1) if case["init"] else None
        if case["kind"] == "train":
            s["dy"] = normal(lead + (D,), io)
            s["dfinal"] = normal((b, D, N), case["state"], 0.1)
    if case["pad"]:
        pad = torch.randint(0, L + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        pad[0] = 0
        s["pad"] = pad
    else:
        s["pad"] = None
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own_run(s):
    from mamba_ssd_scan_chunked_b200 import ssd
    c = s["case"]
    if c["op"] == "norm":
        kw = dict(ngroups=c["groups"], eps=s["eps"], center=c["center"], gate_first=c["gate"] == "before",
                  activation="silu" if c["gate"] == "silu" else None)
        if c["kind"] == "prompt":
            return ssd.group_norm_fwd(s["x"], s["weight"], s["bias"], s["z"], y_dtype=_t(c["io"]), **kw)
        return ssd.group_norm_bwd(s["x"], s["weight"], s["bias"], s["dy"], s["z"], grad_dtype=_t(c["io"]), **kw)
    if c["op"] == "conv":
        kw = dict(activation="silu" if c["silu"] else None)
        if c["kind"] == "token":
            y = ssd.conv1d_update(s["init"], s["x"], s["weight"], s["bias"], split=s["split"], **kw)
            return {"y": y, "state": s["init"]}
        if c["kind"] == "prompt":
            y, final = ssd.conv1d_fwd(s["x"], s["weight"], s["bias"], s["init"], split=s["split"], pad_left=s["pad"],
                                      state_dtype=_t(c["state"]), **kw)
            return {"y": y, "state": final}
        return ssd.conv1d_bwd(s["x"], s["weight"], s["bias"], s["dy"], s["init"], s["dfinal"],
                              want_dinit=c["init"], **kw)
    if c["kind"] == "token":
        y = ssd.selective_state_update(s["init"], s["x"], s["dt_raw"], s["dt_bias"], s["A"], s["B"], s["C"], s["D"],
                                       s["z"])
        return {"y": y, "state": s["init"]}
    if c["kind"] == "prompt":
        y, final = ssd.selective_scan_fwd(s["x"], s["dt_raw"], s["dt_bias"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                          s["init"], pad_left=s["pad"], state_dtype=_t(c["state"]))
        return {"y": y, "state": final}
    return ssd.selective_scan_bwd(s["x"], s["dt_raw"], s["dt_bias"], s["A"], s["B"], s["C"], s["D"], s["dy"], s["z"],
                                  s["init"], s["dfinal"], want_dinit=c["init"])


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _silu(v):
    return v * _sigmoid(v)


def _dsilu(v):
    g = _sigmoid(v)
    return g * (1.0 + v * (1.0 - g))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _live(s, L):
    """[b, L] truth values: token t of sequence b exists (it is not padding)."""
    pad = s["pad"] if s["pad"] is not None else torch.zeros(s["x"].shape[0], dtype=torch.int32, device=s["x"].device)
    return torch.arange(L, device=pad.device)[None, :] >= pad[:, None], pad.long()


def _window(s, x):
    """The W inputs of every token, [W][b, L, D] oldest first, and the last W - 1 inputs of every
    sequence: the kept inputs, then the tokens from the padding on."""
    b, L, D = x.shape
    W = s["case"]["width"]
    live, pad = _live(s, L)
    keep = s["init"].float() if s["init"] is not None else torch.zeros(b, W - 1, D, device=x.device)
    both = torch.cat([keep, torch.where(live[..., None], x, torch.zeros_like(x))], 1)   # place i: token i - (W - 1)
    t = torch.arange(L, device=x.device)

    def at(tokens):   # [b, n] token indices; those before the padding's end count back into the kept inputs
        i = torch.where(tokens >= pad[:, None], tokens, (tokens - pad[:, None]).clamp(min=1 - W)) + W - 1
        return torch.gather(both, 1, i[..., None].expand(-1, -1, D))

    taps = [at((t - (W - 1 - k)).expand(b, L)) for k in range(W)]
    last = at(torch.arange(L - (W - 1), L, device=x.device).expand(b, W - 1))
    return taps, last, live


def _plain_conv(s):
    c = s["case"]
    W, y_dtype = c["width"], s["x"].dtype
    if c["kind"] == "token":
        both = torch.cat([s["init"].float(), s["x"].float()[:, None]], 1)
        v = (both * s["weight"].t()[None]).sum(1) + s["bias"]
        s["init"].copy_(both[:, 1:])
        y = (_silu(v) if c["silu"] else v).to(y_dtype)
        return {"y": [p.contiguous() for p in torch.split(y, s["split"], -1)], "state": s["init"]}
    taps, last, live = _window(s, s["x"].float())
    v = sum(taps[k] * s["weight"][:, k] for k in range(W)) + s["bias"]
    if c["kind"] == "prompt":
        y = torch.where(live[..., None], _silu(v) if c["silu"] else v, torch.zeros_like(v)).to(y_dtype)
        return {"y": [p.contiguous() for p in torch.split(y, s["split"], -1)], "state": last.to(_t(c["state"]))}
    dv = torch.cat(s["dy"], -1).float()
    if c["silu"]:
        dv = dv * _dsilu(v)
    L = dv.shape[1]
    dboth = torch.zeros(dv.shape[0], L + W - 1, dv.shape[2], device=dv.device)   # place i: token i - (W - 1)
    dboth[:, L:] = s["dfinal"].float()
    for k in range(W):
        dboth[:, k:k + L] += dv * s["weight"][:, k]
    return {"dx": dboth[:, W - 1:].to(y_dtype), "dweight": torch.stack([(dv * taps[k]).sum((0, 1)) for k in range(W)], 1),
            "dbias": dv.sum((0, 1)), "dinit_state": dboth[:, :W - 1].to(_t(c["state"])) if c["init"] else None}


def _carried(a, v):
    """h_t = a_t h_{t-1} + v_t along dim 1 from h_{-1} = 0, by doubling: after the step of length s each
    place holds its last 2 s terms, so there are log2(L) rounds over the data.  Overwrites both."""
    s, L = 1, v.shape[1]
    while s < L:
        v[:, s:] += a[:, s:] * v[:, :-s]
        a[:, s:] = a[:, s:] * a[:, :-s]
        s *= 2
    return v


def _scan_inputs(s, lead):
    """x, dt, A, B, C, D in 32 bits; channels as [groups][channels of the group], padding cleared."""
    c = s["case"]
    G, D = c["groups"], c["channels"]
    x, z = s["x"].float(), s["dt_raw"].float() + s["dt_bias"]
    dt, B, C = _softplus(z), s["B"].float()[..., None, :], s["C"].float()[..., None, :]
    if s["pad"] is not None:
        live = _live(s, lead[1])[0][..., None]
        x, dt = (torch.where(live, v, torch.zeros_like(v)) for v in (x, dt))
        B, C = (torch.where(live[..., None, None], v, torch.zeros_like(v)) for v in (B, C))
    shape = lead + (G, D // G)
    return x.view(shape), dt.view(shape), s["A"].view(G, D // G, -1), B, C, s["D"].view(G, D // G)


def _plain_scan(s):
    c = s["case"]
    token = c["kind"] == "token"
    b, L, D, N, G = c["batch"], c["seqlen"], c["channels"], c["dstate"], c["groups"]
    lead = (b,) if token else (b, L)
    io = s["x"].dtype
    x, dt, A, B, C, skip = _scan_inputs(s, lead)
    init = s["init"].float().view(b, G, D // G, N) if s["init"] is not None else torch.zeros(b, G, D // G, N, device=x.device)
    a = torch.exp(dt[..., None] * A)
    v = (dt * x)[..., None] * B
    if token:
        h = a * init + v
        y = ((h * C).sum(-1) + skip * x).view(b, D)
        if s["z"] is not None:
            y = y * _silu(s["z"].float())
        s["init"].copy_(h.view(b, D, N))
        return {"y": y.to(io), "state": s["init"]}
    v[:, 0] += a[:, 0] * init
    if c["kind"] == "prompt":
        h = _carried(a, v)
        y = ((h * C).sum(-1) + skip * x).view(b, L, D)
        if s["z"] is not None:
            y = y * _silu(s["z"].float())
        if s["pad"] is not None:
            y = torch.where(_live(s, L)[0][..., None], y, torch.zeros_like(y))
        return {"y": y.to(io), "state": h[:, -1].reshape(b, D, N).to(_t(c["state"]))}
    h = _carried(a.clone(), v)
    dy = s["dy"].float()
    g, dz = dy, None
    if s["z"] is not None:
        z = s["z"].float()
        g = dy * _silu(z)
        dz = (dy * ((h * C).sum(-1) + skip * x).view(b, L, D) * _dsilu(z)).to(io)
    g = g.view(b, L, G, D // G)
    # the adjoint of the state, carried from the last token back: w_t = C_t g_t + a_{t+1} w_{t+1}
    w = (g[..., None] * C).flip(1)
    w[:, 0] += s["dfinal"].float().view(b, G, D // G, N)
    w = _carried(torch.cat([torch.zeros_like(a[:, :1]), a[:, 1:].flip(1)], 1), w).flip(1)
    back = torch.cat([init[:, None], h[:, :-1]], 1) * a          # a_t h_{t-1}
    ddt = (w * (B * x[..., None] + A * back)).sum(-1)
    ddt = (ddt.view(b, L, D) * _sigmoid(s["dt_raw"].float() + s["dt_bias"]))
    return {"dx": (dt * (w * B).sum(-1) + skip * g).view(b, L, D).to(io), "ddt_raw": ddt.to(io), "dz": dz,
            "dB": (w * (dt * x)[..., None]).sum(-2).to(io), "dC": (h * g[..., None]).sum(-2).to(io),
            "dA": (w * back * dt[..., None]).sum((0, 1)).view(D, N), "ddt_bias": ddt.sum((0, 1)),
            "dD": (g * x).sum((0, 1)).view(D), "dinit_state": (a[:, 0] * w[:, 0]).view(b, D, N).to(_t(c["state"])) if c["init"] else None}


def _plain_norm(s):
    c = s["case"]
    rows, D, G = c["rows"], c["channels"], c["groups"]
    x = s["x"].float()
    z = s["z"].float() if s["z"] is not None else None
    u = (x * _silu(z) if c["gate"] == "before" else x).view(rows, G, D // G)
    if c["center"]:
        u = u - u.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((u * u).mean(-1, keepdim=True) + s["eps"])
    n = (u * r).view(rows, D)
    v = n * s["weight"] + (s["bias"] if s["bias"] is not None else 0.0)
    if c["kind"] == "prompt":
        y = v * _silu(z) if c["gate"] == "after" else _silu(v) if c["gate"] == "silu" else v
        return y.to(_t(c["io"]))
    io = _t(c["io"])
    dv, dz = s["dy"].float(), None
    if c["gate"] == "after":
        dz, dv = dv * v * _dsilu(z), dv * _silu(z)
    elif c["gate"] == "silu":
        dv = dv * _dsilu(v)
    dn = (dv * s["weight"]).view(rows, G, D // G)
    ng = n.view(rows, G, D // G)
    du = dn - ng * (dn * ng).mean(-1, keepdim=True)
    if c["center"]:
        du = du - dn.mean(-1, keepdim=True)
    du = (du * r).view(rows, D)
    if c["gate"] == "before":
        du, dz = du * _silu(z), du * x * _dsilu(z)
    return {"dx": du.to(io), "dz": dz.to(io) if dz is not None else None, "dweight": (dv * n).sum(0),
            "dbias": dv.sum(0) if s["bias"] is not None else None}


def run(state):
    if own:
        return _own_run(state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token
# ---------------------------------------------------------------------------
def _exact_conv(s):
    c = s["case"]
    W, split = c["width"], s["split"]
    token = c["kind"] == "token"
    x = s["x"].double()[:, None] if token else s["x"].double()
    b, L, D = x.shape
    w, bias = s["weight"].double(), s["bias"].double()
    kept = s["init"].double() if s["init"] is not None else x.new_zeros(b, W - 1, D)
    train = c["kind"] == "train"
    y, final = x.new_zeros(b, L, D), x.new_empty(b, W - 1, D)
    dx, dw, db, dinit = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias), torch.zeros_like(kept)
    for i in range(b):
        p = int(s["pad"][i]) if s["pad"] is not None else 0
        seq = torch.cat([kept[i], x[i, p:]], 0)
        n = L - p
        final[i] = seq[n:]
        if not n:
            continue
        win = seq.unfold(0, W, 1)                      # [n, D, W]
        v = torch.einsum("ndk,dk->nd", win, w) + bias
        sig = torch.sigmoid(v)
        y[i, p:] = v * sig if c["silu"] else v
        if train:
            d = torch.cat([q[i].double() for q in s["dy"]], -1)
            if c["silu"]:
                d = d * (sig + v * sig * (1 - sig))
            dw += torch.einsum("nd,ndk->dk", d, win)
            db += d.sum(0)
            dseq = torch.zeros_like(seq)
            dseq[n:] = s["dfinal"][i].double()
            for k in range(W):
                dseq[k:k + n] += d * w[:, k]
            dinit[i], dx[i] = dseq[:W - 1], dseq[W - 1:]
    if train:
        return {"dx": dx, "dweight": dw, "dbias": db, "dinit_state": dinit if c["init"] else None}
    y = y[:, 0] if token else y
    return {"y": list(torch.split(y, split, -1)), "state": final}


def _exact_scan(s):
    c = s["case"]
    token, train = c["kind"] == "token", c["kind"] == "train"
    G, D, N = c["groups"], c["channels"], c["dstate"]
    up = (lambda v: v.double()[:, None]) if token else (lambda v: v.double())
    x, zdt = up(s["x"]), up(s["dt_raw"]) + s["dt_bias"].double()
    b, L, _ = x.shape
    dt = torch.logaddexp(zdt, torch.zeros_like(zdt))
    B, C = up(s["B"]), up(s["C"])
    A, skip = s["A"].double(), s["D"].double()
    z = up(s["z"]) if s["z"] is not None else None
    gate = z * torch.sigmoid(z) if z is not None else torch.ones_like(x)
    pad = s["pad"] if s["pad"] is not None else torch.zeros(b, dtype=torch.int32, device=x.device)
    wide = lambda v: v.repeat_interleave(D // G, 1)   # noqa: E731  [b, G, N] -> [b, D, N]
    h = s["init"].double() if s["init"] is not None else x.new_zeros(b, D, N)
    raw, kept = torch.zeros_like(x), [h]
    for t in range(L):
        live = (pad <= t).double()[:, None]
        step = dt[:, t] * live
        h = torch.exp(step[..., None] * A) * h + (step * x[:, t])[..., None] * wide(B[:, t])
        raw[:, t] = ((h * wide(C[:, t])).sum(-1) + skip * x[:, t]) * live
        if train:
            kept.append(h)
    y = raw * gate
    if not train:
        return {"y": y[:, 0] if token else y, "state": h}
    dy = s["dy"].double()
    g = dy * gate
    dx, ddt, dB, dC = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C)
    dA, w = torch.zeros_like(A), s["dfinal"].double()
    for t in range(L - 1, -1, -1):
        Bt = wide(B[:, t])
        w = w + g[:, t, :, None] * wide(C[:, t])
        dC[:, t] = (kept[t + 1] * g[:, t, :, None]).view(b, G, D // G, N).sum(2)
        dB[:, t] = (w * (dt[:, t] * x[:, t])[..., None]).view(b, G, D // G, N).sum(2)
        wB = (w * Bt).sum(-1)
        dx[:, t] = dt[:, t] * wB + skip * g[:, t]
        a = torch.exp(dt[:, t, :, None] * A)
        wah = w * a * kept[t]
        ddt[:, t] = x[:, t] * wB + (wah * A).sum(-1)
        dA += (wah * dt[:, t, :, None]).sum(0)
        w = w * a
    ddt = ddt * torch.sigmoid(zdt)
    dz = None
    if z is not None:
        sig = torch.sigmoid(z)
        dz = dy * raw * (sig + z * sig * (1 - sig))
    return {"dx": dx, "ddt_raw": ddt, "dz": dz, "dB": dB, "dC": dC, "dA": dA, "ddt_bias": ddt.sum((0, 1)),
            "dD": (g * x).sum((0, 1)), "dinit_state": w if c["init"] else None}


def _exact_norm(s):
    """Gradients by automatic differentiation of the definition."""
    c = s["case"]
    rows, D, G = c["rows"], c["channels"], c["groups"]
    train = c["kind"] == "train"
    leaf = lambda v: None if v is None else v.double().detach().requires_grad_(train)   # noqa: E731
    x, z, w, bias = leaf(s["x"]), leaf(s["z"]), leaf(s["weight"]), leaf(s["bias"])
    u = (x * z * torch.sigmoid(z) if c["gate"] == "before" else x).view(rows, G, D // G)
    if c["center"]:
        u = u - u.mean(-1, keepdim=True)
    v = (u * (u.pow(2).mean(-1, keepdim=True) + s["eps"]).rsqrt()).view(rows, D) * w
    v = v + bias if bias is not None else v
    y = v * z * torch.sigmoid(z) if c["gate"] == "after" else v * torch.sigmoid(v) if c["gate"] == "silu" else v
    if not train:
        return y
    y.backward(s["dy"].double())
    return {"dx": x.grad, "dz": z.grad if z is not None else None, "dweight": w.grad,
            "dbias": bias.grad if bias is not None else None}


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)
