"""Refusals of the operators around the scan, checked without a GPU: every call
below returns before any CUDA call."""
import pytest
import torch

from mamba_ssd_scan_chunked_b200 import build as B
from mamba_ssd_scan_chunked_b200 import ssd

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
FAKE, STEP = 0x7f0000000000, 0x4000000


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def caller(fn, names, optional, tail):
    """A call with distinct aligned fake addresses for `names` (0 for the `optional` ones)."""
    base = {k: 0 if k in optional else FAKE + STEP * i for i, k in enumerate(names)}

    def call(desc, **kw):
        p = {**base, **tail, "stream": 0, **kw}
        return fn(desc, *(p[k] for k in (*names, *tail, "stream")))

    return call, base


def conv(**kw):
    d = dict(batch=2, seqlen=40, channels=64, width=4, x_stride=64, dx_stride=64, split1=0, split2=0,
             io_dtype=ssd.SSD_BF16, y_dtype=ssd.SSD_BF16, state_dtype=ssd.SSD_F32, activation=1)
    return ssd.Conv1dDesc(**{**d, **kw})


CONV_FWD = ("x", "weight", "bias", "init_state", "pad_left", "y0", "y1", "y2", "final_state")
CONV_UPD = ("state", "x", "weight", "bias", "y0", "y1", "y2")
CONV_BWD = ("x", "weight", "bias", "init_state", "dy0", "dy1", "dy2", "dfinal_state", "dx", "dweight", "dbias",
            "dinit_state")
BAD_CONV = [(dict(batch=-1), INVALID), (dict(channels=0), INVALID), (dict(io_dtype=3), INVALID),
            (dict(state_dtype=-1), INVALID), (dict(activation=2), INVALID), (dict(x_stride=56), INVALID),
            (dict(split1=64), INVALID), (dict(split2=8), INVALID), (dict(split1=-8), INVALID),
            (dict(split1=32, split2=32), INVALID), (dict(split1=1 << 62, split2=1 << 62), INVALID),
            (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(channels=60), UNSUPPORTED),
            (dict(split1=12), UNSUPPORTED), (dict(x_stride=68), UNSUPPORTED), (dict(batch=1 << 30), UNSUPPORTED),
            (dict(batch=1 << 24, seqlen=1 << 31), UNSUPPORTED), (dict(channels=1 << 21, x_stride=1 << 21), UNSUPPORTED)]


def test_conv1d_fwd_codes():
    call, p = caller(ssd.ssd_conv1d_fwd, CONV_FWD, ("bias", "init_state", "pad_left", "y1", "y2", "final_state"), {})
    for kw, code in BAD_CONV:
        assert call(conv(**kw)) == code, kw
    for k in ("x", "weight", "y0"):
        assert call(conv(), **{k: 0}) == INVALID, k
        assert call(conv(), **{k: p[k] + 8}) == ALIGN, k
    assert call(conv(), y1=FAKE + 0x80000000) == INVALID            # a second output without channels
    assert call(conv(split1=8)) == INVALID                          # channels without their output
    assert call(conv(split1=8, split2=8), y1=FAKE + 0x80000000) == INVALID
    assert call(conv(), y0=p["x"] + 16) == INVALID                  # y over x
    assert call(conv(), y0=p["weight"]) == INVALID
    assert call(conv(), init_state=FAKE + 0x80000000, final_state=FAKE + 0x80000000) == INVALID
    assert call(conv(), final_state=p["y0"]) == INVALID
    assert call(conv(), pad_left=FAKE + 0x90000002) == ALIGN
    assert call(conv(), pad_left=p["y0"] + 64) == INVALID           # the lengths inside an output
    assert call(conv(batch=0), x=0, y0=0) == OK                     # nothing to do, nothing launched
    assert call(conv(seqlen=0), x=0, y0=0) == OK


def test_conv1d_update_codes():
    call, p = caller(ssd.ssd_conv1d_update, CONV_UPD, ("bias", "y1", "y2"), {})
    for kw, code in BAD_CONV:
        assert call(conv(**{"seqlen": 1, **kw})) == code, kw
    assert call(conv()) == INVALID                                  # seqlen has to be 1
    for k in ("state", "x", "weight", "y0"):
        assert call(conv(seqlen=1), **{k: 0}) == INVALID, k
        assert call(conv(seqlen=1), **{k: p[k] + 4}) == ALIGN, k
    assert call(conv(seqlen=1), state=p["x"]) == INVALID
    assert call(conv(seqlen=1), y0=p["state"]) == INVALID
    assert call(conv(seqlen=1, batch=0), state=0, x=0, y0=0) == OK


def test_conv1d_bwd_codes():
    call, p = caller(ssd.ssd_conv1d_bwd, CONV_BWD, ("bias", "init_state", "dy1", "dy2", "dfinal_state", "dbias",
                                                    "dinit_state"), dict(workspace=FAKE + 0x100000000,
                                                                         workspace_bytes=1 << 30))
    for kw, code in BAD_CONV + [(dict(dx_stride=56), INVALID), (dict(dx_stride=68), UNSUPPORTED)]:
        assert call(conv(**kw)) == code, kw
    for k in ("x", "weight", "dy0", "dx", "dweight"):
        assert call(conv(), **{k: 0}) == INVALID, k
        assert call(conv(), **{k: p[k] + 8}) == ALIGN, k
    need = ssd.ssd_conv1d_bwd_workspace_size(conv())
    assert need >= 4 * 64 * 5
    assert call(conv(), workspace=0) == WORKSPACE
    assert call(conv(), workspace_bytes=need - 1) == WORKSPACE
    assert call(conv(), workspace=FAKE + 0x100000010) == ALIGN
    assert call(conv(), workspace=p["dx"]) == INVALID               # the workspace inside an argument
    assert call(conv(), dx=p["x"]) == INVALID
    assert call(conv(), dx=p["dy0"]) == INVALID
    assert call(conv(), dbias=p["dweight"]) == INVALID
    assert call(conv(), dy1=FAKE + 0x90000000) == INVALID


def sel(**kw):
    d = dict(batch=2, seqlen=40, channels=64, dstate=16, ngroups=2, z_stride=64, io_dtype=ssd.SSD_BF16,
             y_dtype=ssd.SSD_BF16, state_dtype=ssd.SSD_F32)
    return ssd.SelectiveDesc(**{**d, **kw})


SEL_IN = ("x", "dt_raw", "dt_bias", "A", "B", "C", "D", "z")
BAD_SEL = [(dict(batch=-1), INVALID), (dict(channels=0), INVALID), (dict(ngroups=3), INVALID), (dict(ngroups=0), INVALID),
           (dict(dstate=0), INVALID), (dict(y_dtype=2), INVALID), (dict(channels=72), UNSUPPORTED),
           (dict(dstate=12), UNSUPPORTED), (dict(dstate=264), UNSUPPORTED), (dict(batch=1 << 25), UNSUPPORTED),
           (dict(batch=1 << 24, seqlen=1 << 31), UNSUPPORTED), (dict(channels=1 << 21), UNSUPPORTED)]


def test_selective_scan_fwd_codes():
    call, p = caller(ssd.ssd_selective_scan_fwd, SEL_IN + ("init_state", "pad_left", "y", "final_state"),
                     ("dt_bias", "D", "z", "init_state", "pad_left", "final_state"),
                     dict(workspace=FAKE + 0x100000000, workspace_bytes=1 << 30))
    for kw, code in BAD_SEL:
        assert call(sel(**kw)) == code, kw
    z = FAKE + 0x90000000
    assert call(sel(z_stride=56), z=z) == INVALID
    assert call(sel(z_stride=68), z=z) == UNSUPPORTED
    for k in ("x", "dt_raw", "A", "B", "C", "y"):
        assert call(sel(), **{k: 0}) == INVALID, k
        assert call(sel(), **{k: p[k] + 8}) == ALIGN, k
    assert call(sel(), z=z + 8) == ALIGN
    for k in ("x", "dt_raw", "B", "C"):
        assert call(sel(), y=p[k]) == INVALID, k
    assert call(sel(), init_state=z, final_state=z) == INVALID
    assert call(sel(), final_state=p["y"]) == INVALID
    assert call(sel(), pad_left=z + 1) == ALIGN
    assert call(sel(), pad_left=p["y"]) == INVALID
    assert call(sel(), workspace=FAKE + 0x100000010) == ALIGN
    assert call(sel(batch=0), x=0, dt_raw=0, B=0, C=0, y=0) == OK
    assert call(sel(seqlen=0), x=0, dt_raw=0, B=0, C=0, y=0) == OK


def test_selective_state_update_codes():
    call, p = caller(ssd.ssd_selective_state_update, ("state",) + SEL_IN + ("y",), ("dt_bias", "D", "z"), {})
    for kw, code in BAD_SEL:
        assert call(sel(**{"seqlen": 1, **kw})) == code, kw
    assert call(sel()) == INVALID
    for k in ("state", "x", "dt_raw", "A", "B", "C", "y"):
        assert call(sel(seqlen=1), **{k: 0}) == INVALID, k
        assert call(sel(seqlen=1), **{k: p[k] + 8}) == ALIGN, k
    assert call(sel(seqlen=1), y=p["state"]) == INVALID
    assert call(sel(seqlen=1), state=p["B"]) == INVALID
    assert call(sel(seqlen=1, batch=0), state=0, x=0, dt_raw=0, B=0, C=0, y=0) == OK


def test_selective_scan_bwd_codes():
    names = SEL_IN + ("init_state", "dy", "dfinal_state", "dx", "ddt_raw", "ddt_bias", "dA", "dB", "dC", "dD", "dz",
                      "dinit_state")
    call, p = caller(ssd.ssd_selective_scan_bwd, names,
                     ("dt_bias", "D", "z", "init_state", "dfinal_state", "ddt_bias", "dD", "dz", "dinit_state"),
                     dict(workspace=FAKE + 0x200000000, workspace_bytes=1 << 32))
    for kw, code in BAD_SEL:
        assert call(sel(**kw)) == code, kw
    for k in ("x", "dt_raw", "A", "B", "C", "dy", "dx", "ddt_raw", "dA", "dB", "dC"):
        assert call(sel(), **{k: 0}) == INVALID, k
        assert call(sel(), **{k: p[k] + 8}) == ALIGN, k
    z, dz = FAKE + 0x180000000, FAKE + 0x190000000
    assert call(sel(), z=z) == INVALID                              # a gate without the place for its gradient
    assert call(sel(), dz=dz) == INVALID                            # and the other way round
    assert call(sel(), z=z, dz=z) == INVALID
    assert call(sel(), dx=p["dy"]) == INVALID
    assert call(sel(), dC=p["dB"]) == INVALID
    need = ssd.ssd_selective_scan_bwd_workspace_size(sel())
    assert need > 0
    assert call(sel(), workspace=0) == WORKSPACE
    assert call(sel(), workspace_bytes=need - 1) == WORKSPACE
    assert call(sel(), workspace=FAKE + 0x200000010) == ALIGN
    assert call(sel(), workspace=p["x"]) == INVALID


def norm(**kw):
    d = dict(rows=10, channels=64, ngroups=2, z_stride=64, eps=1e-5, x_dtype=ssd.SSD_F32, io_dtype=ssd.SSD_BF16,
             y_dtype=ssd.SSD_BF16, center=0, activation=ssd.SSD_NORM_GATE_BEFORE)
    return ssd.GroupNormDesc(**{**d, **kw})


BAD_NORM = [(dict(rows=-1), INVALID), (dict(ngroups=3), INVALID), (dict(x_dtype=2), INVALID), (dict(center=2), INVALID),
            (dict(activation=4), INVALID), (dict(activation=-1), INVALID), (dict(eps=0.0), INVALID),
            (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(z_stride=56), INVALID),
            (dict(z_stride=68), UNSUPPORTED), (dict(channels=72, z_stride=72), UNSUPPORTED),
            (dict(channels=16392, ngroups=1, z_stride=16392), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED)]


def test_group_norm_codes():
    fwd, p = caller(ssd.ssd_group_norm_fwd, ("x", "z", "weight", "bias", "y"), ("weight", "bias"), {})
    for kw, code in BAD_NORM:
        assert fwd(norm(**kw)) == code, kw
    for k in ("x", "z", "y"):
        assert fwd(norm(), **{k: 0}) == INVALID, k
        assert fwd(norm(), **{k: p[k] + 8}) == ALIGN, k
    for act in (ssd.SSD_NORM_NONE, ssd.SSD_NORM_SILU):
        assert fwd(norm(activation=act)) == INVALID                 # z without a gate
    assert fwd(norm(), y=p["x"]) == INVALID
    assert fwd(norm(), y=p["z"]) == INVALID
    assert fwd(norm(rows=0), x=0, z=0, y=0) == OK
    bwd, p = caller(ssd.ssd_group_norm_bwd, ("x", "z", "weight", "bias", "dy", "dx", "dz", "dweight", "dbias"),
                    ("weight", "bias", "dweight", "dbias"), dict(workspace=FAKE + 0x100000000, workspace_bytes=1 << 30))
    for kw, code in BAD_NORM:
        assert bwd(norm(**kw)) == code, kw
    for k in ("x", "z", "dy", "dx", "dz"):
        assert bwd(norm(), **{k: 0}) == INVALID, k
        assert bwd(norm(), **{k: p[k] + 8}) == ALIGN, k
    need = ssd.ssd_group_norm_bwd_workspace_size(norm())
    assert bwd(norm(), workspace=0) == WORKSPACE
    assert bwd(norm(), workspace_bytes=need - 1) == WORKSPACE
    assert bwd(norm(), workspace=FAKE + 0x100000080) == ALIGN
    assert bwd(norm(), dx=p["dy"]) == INVALID
    assert bwd(norm(), dz=p["dx"]) == INVALID
    assert bwd(norm(), dweight=FAKE + 0x90000000, dbias=FAKE + 0x90000000) == INVALID


def test_workspace_sizes_refuse_what_the_calls_refuse():
    for size, make, bad in ((ssd.ssd_conv1d_bwd_workspace_size, conv, BAD_CONV),
                            (ssd.ssd_selective_scan_workspace_size, sel, BAD_SEL),
                            (ssd.ssd_selective_scan_bwd_workspace_size, sel, BAD_SEL),
                            (ssd.ssd_group_norm_bwd_workspace_size, norm, BAD_NORM)):
        for kw, code in bad:
            with pytest.raises(ssd.SsdError) as e:
                size(make(**kw))
            assert e.value.status == code, kw


def test_binding_refuses_before_any_cuda_call():
    z = torch.zeros
    x, w = z(2, 5, 16), z(16, 4)
    bad = [
        (lambda: ssd.conv1d_fwd(x, w), "CUDA"),
        (lambda: ssd.conv1d_fwd(x, z(16, 4, dtype=torch.bfloat16)), "weight"),
        (lambda: ssd.conv1d_fwd(x, w, z(8)), "bias"),
        (lambda: ssd.conv1d_fwd(x, w, None, z(2, 4, 16)), "init_state"),
        (lambda: ssd.conv1d_fwd(x, w, split=(8, 4)), "split"),
        (lambda: ssd.conv1d_fwd(x, w, split=(4, 4, 4, 4)), "split"),
        (lambda: ssd.conv1d_fwd(x, w, split=(16, 0)), "split"),
        (lambda: ssd.conv1d_fwd(x, w, activation="relu"), "activation"),
        (lambda: ssd.conv1d_fwd(x, w, pad_left=z(2)), "pad_left"),
        (lambda: ssd.conv1d_fwd(x, w, pad_left=z(3, dtype=torch.int32)), "pad_left"),
        (lambda: ssd.conv1d_fwd(z(2, 16, 5).transpose(1, 2), w), "x"),
        (lambda: ssd.conv1d_fwd(z(5, 2, 16).transpose(0, 1), w), "x"),
        (lambda: ssd.conv1d_fwd(z(2, 1, 16).expand(2, 5, 16), w), "x"),
        (lambda: ssd.conv1d_fwd(x, w, y=z(2, 5, 8)), "y"),
        (lambda: ssd.conv1d_fwd(x, w, final_state=z(2, 3, 8)), "final_state"),
        (lambda: ssd.conv1d_update(z(2, 3, 8), z(2, 16), w), "state"),
        (lambda: ssd.conv1d_bwd(x, w, None, (z(2, 5, 8), z(2, 5, 4))), "split"),
        (lambda: ssd.conv1d_bwd(x, w, None, x.bfloat16()), "dy"),
        (lambda: ssd.conv1d_bwd(x, w, None, x, dx=z(2, 5, 8)), "dx"),
        (lambda: ssd.conv1d_bwd(x, w, None, x, dfinal_state=z(2, 3, 8)), "dfinal_state"),
    ]
    d, A, bc = z(2, 5, 16), z(16, 8), z(2, 5, 1, 8)
    bad += [
        (lambda: ssd.selective_scan_fwd(d, d, None, A, bc, bc, None), "CUDA"),
        (lambda: ssd.selective_scan_fwd(d, d[:, :4], None, A, bc, bc, None), "dt_raw"),
        (lambda: ssd.selective_scan_fwd(d, d, z(8), A, bc, bc, None), "dt_bias"),
        (lambda: ssd.selective_scan_fwd(d, d, None, z(16, 16), bc, bc, None), "A"),
        (lambda: ssd.selective_scan_fwd(d, d, None, A, bc, bc.bfloat16(), None), "C"),
        (lambda: ssd.selective_scan_fwd(d, d, None, A, bc, bc, z(16).double()), "D"),
        (lambda: ssd.selective_scan_fwd(d, d, None, A, bc, bc, None, d.bfloat16()), "z"),
        (lambda: ssd.selective_scan_fwd(d, d, None, A, bc, bc, None, None, z(2, 16, 4)), "init_state"),
        (lambda: ssd.selective_scan_fwd(d, d, None, A, bc, bc, None, y=z(2, 5, 8)), "y"),
        (lambda: ssd.selective_state_update(z(2, 16, 4), d[:, 0], d[:, 0], None, A, bc[:, 0], bc[:, 0], None), "state"),
        (lambda: ssd.selective_scan_bwd(d, d, None, A, bc, bc, None, d[:, :4]), "dy"),
        (lambda: ssd.selective_scan_bwd(d, d, None, A, bc, bc, None, d, None, None, z(2, 16, 4)), "dfinal_state"),
        (lambda: ssd.group_norm_fwd(d, z(8)), "weight"),
        (lambda: ssd.group_norm_fwd(d, None, z(8)), "bias"),
        (lambda: ssd.group_norm_fwd(d, None, None, d[:, :4]), "z"),
        (lambda: ssd.group_norm_fwd(d, None, None, d, activation="silu"), "activation"),
        (lambda: ssd.group_norm_fwd(d, None, y=d[:1]), "y"),
        (lambda: ssd.group_norm_fwd(d), "CUDA"),
        (lambda: ssd.group_norm_bwd(d, None, None, d[:, :4]), "dy"),
        (lambda: ssd.group_norm_bwd(d, None, None, d, d.bfloat16()), "z"),
    ]
    for call, what in bad:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(TypeError):
        ssd.group_norm_fwd(d.half())


def test_rows_of_wider_tensors():
    z = torch.zeros(3, 5, 24)
    assert ssd._row_stride(z[..., 8:], "x", (3, 5), 16, None) == 24
    assert ssd._row_stride(z[:, :1, 8:], "x", (3, 1), 16, None) == 120          # the only rows there are
    assert ssd._row_stride(z[:1, :, :16], "x", (1, 5), 16, None) == 24
    assert ssd._row_stride(z[:1, :1, :16], "x", (1, 1), 16, None) == 16
    assert ssd._row_stride(z[:0, :, :16], "x", (0, 5), 16, None) == 16
    assert ssd._row_stride(z[:, 2, :16], "x", (3,), 16, None) == 120
    with pytest.raises(ValueError, match="distance"):
        ssd._row_stride(z[:, :4, :16], "x", (3, 4), 16, None)                   # a gap after every fourth row


def test_tensors_on_several_devices_are_refused():
    class Fake:
        def __init__(self, i):
            self.i = i

        def get_device(self):
            return self.i

        def is_contiguous(self):
            return True

    assert ssd._one_device((Fake(1), None, Fake(1)), (None, Fake(1))) == 1
    for dense, rows in (((Fake(0), Fake(1)), ()), ((Fake(0),), (Fake(1),))):
        with pytest.raises(ValueError, match="one device"):
            ssd._one_device(dense, rows)
    for dense, rows in (((Fake(0), Fake(-1)), ()), ((Fake(0),), (Fake(-1),))):
        with pytest.raises(ValueError, match="CUDA"):
            ssd._one_device(dense, rows)


def test_the_stream_of_another_device_is_refused(monkeypatch):
    class Stream:
        cuda_stream, device = 0, torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream on device 1"):
        ssd._launch_on(0, Stream(), lambda handle: handle)


@pytest.mark.parametrize("captures", [(), ("main", "side"), ("side",), ("main",)])
def test_a_given_stream_waits_for_the_current_one_and_its_tensors_are_kept(monkeypatch, captures):
    """The inputs may be made on the current stream just before the call and dropped just after it: the
    given stream waits for the current one, and the allocator learns of the use.  A capture that one of the
    two alone takes part in cannot hold the wait."""
    events = []

    class Stream:
        device = torch.device("cuda", 0)

        def __init__(self, name, handle):
            self.name, self.cuda_stream = name, handle

        def wait_stream(self, other):
            events.append((self.name, "waits for", other.name))

    class Tensor:
        def record_stream(self, stream):
            events.append(("kept for", stream.name))

    class Inside:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            now.append(self.stream)

        def __exit__(self, *_):
            now.pop()

    main, side = Stream("main", 0), Stream("side", 64)
    now = [main]
    monkeypatch.setattr(torch.cuda, "device", lambda index: Inside(now[-1]))
    monkeypatch.setattr(torch.cuda, "stream", Inside)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: now[-1])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[-1].name in captures)
    call = lambda handle: events.append(("launched on", handle)) or now[-1].name

    assert ssd._launch_on(0, side, call, (Tensor(), None, Tensor())) == "side"
    kept = [("side", "waits for", "main"), ("kept for", "side"), ("kept for", "side")]
    assert events == (kept if len(captures) != 1 else []) + [("launched on", 64)]
    events.clear()
    assert ssd._launch_on(0, main, call, (Tensor(),)) == "main"       # the current stream itself
    assert events == [("launched on", 0)]


def test_calls_hand_over_every_tensor_they_use(monkeypatch):
    """What a call reads and writes among the caller's tensors is what a given stream has to keep."""
    seen = []
    monkeypatch.setattr(ssd, "_one_device", lambda dense, rows=(): 0)
    monkeypatch.setattr(ssd, "_launch_on", lambda index, stream, call, tensors=(): seen.append(tensors))
    z = lambda *shape: torch.zeros(shape)
    D, N = 16, 8
    io, tok, bc, tbc = (2, 5, D), (2, D), (2, 5, 1, N), (2, 1, N)
    i32 = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    par = [z(D), z(D, N)]                                             # dt_bias, A

    def same(call, *tensors, **named):
        call(*tensors, **named, stream=object())
        given = [t for t in (*tensors, *named.values()) for t in (t if isinstance(t, tuple) else (t,))]
        assert {id(t) for t in seen.pop() if t is not None} == {id(t) for t in given if torch.is_tensor(t)}, call

    same(ssd.conv1d_fwd, z(*io), z(D, 4), z(D), z(2, 3, D), split=(8, 8), pad_left=i32, y=(z(2, 5, 8), z(2, 5, 8)),
         final_state=z(2, 3, D))
    same(ssd.conv1d_update, z(2, 3, D), z(*tok), z(D, 4), z(D), y=z(*tok))
    same(ssd.conv1d_bwd, z(*io), z(D, 4), z(D), (z(2, 5, 8), z(2, 5, 8)), z(2, 3, D), z(2, 3, D), dx=z(*io), workspace=ws)
    same(ssd.selective_scan_fwd, z(*io), z(*io), *par, z(*bc), z(*bc), z(D), z(*io), z(2, D, N), y=z(*io),
         final_state=z(2, D, N), pad_left=i32, workspace=ws)
    same(ssd.selective_state_update, z(2, D, N), z(*tok), z(*tok), *par, z(*tbc), z(*tbc), z(D), z(*tok), y=z(*tok))
    same(ssd.selective_scan_bwd, z(*io), z(*io), *par, z(*bc), z(*bc), z(D), z(*io), z(*io), z(2, D, N), z(2, D, N),
         workspace=ws)
    same(ssd.group_norm_fwd, z(*io), z(D), z(D), z(*io), y=z(*io))
    same(ssd.group_norm_bwd, z(*io), z(D), z(D), z(*io), z(*io), workspace=ws)


@pytest.mark.parametrize("rows,gs,G", [(1, 8, 2047), (1, 8, 131071), (3, 16, 4099), (2, 8, 7), (5, 264, 601), (1, 1032, 1009)])
def test_the_norms_workspace_is_bounded_by_the_rows(rows, gs, G):
    """Two partial sums of 4 bytes for each element of x hold any order of summation; groups whose number
    shares no factor with the groups of a block do not ask for more."""
    need = ssd.ssd_group_norm_bwd_workspace_size(norm(rows=rows, channels=gs * G, ngroups=G, z_stride=gs * G))
    assert 0 < need <= 2 * 4 * rows * gs * G


ROW = 8192 * 8512          # from the last token of a prompt's rows to the next sequence's


def test_rows_far_apart_are_taken():
    """The last tokens of a prompt's rows, or one column block of very long ones, are strided rows like others."""
    upd, _ = caller(ssd.ssd_conv1d_update, CONV_UPD, ("bias", "y1", "y2"), {})
    assert upd(conv(batch=0, seqlen=1, x_stride=ROW), state=0, x=0, y0=0) == OK
    fwd, _ = caller(ssd.ssd_conv1d_fwd, CONV_FWD, ("bias", "init_state", "pad_left", "y1", "y2", "final_state"), {})
    assert fwd(conv(batch=0, x_stride=ROW), x=0, y0=0) == OK
    assert ssd.ssd_conv1d_bwd_workspace_size(conv(x_stride=ROW, dx_stride=1 << 40)) > 0
    step, _ = caller(ssd.ssd_selective_state_update, ("state",) + SEL_IN + ("y",), ("dt_bias", "D"), {})
    assert step(sel(seqlen=1, batch=0, z_stride=ROW), state=0, x=0, dt_raw=0, B=0, C=0, y=0) == OK
    gn, _ = caller(ssd.ssd_group_norm_fwd, ("x", "z", "weight", "bias", "y"), ("weight", "bias"), {})
    assert gn(norm(rows=0, z_stride=ROW), x=0, z=0, y=0) == OK


@pytest.mark.parametrize("far", [(1 << 40) + 8, 1 << 62])
def test_rows_beyond_any_memory_are_refused(far):
    upd, _ = caller(ssd.ssd_conv1d_update, CONV_UPD, ("bias", "y1", "y2"), {})
    assert upd(conv(seqlen=1, x_stride=far)) == UNSUPPORTED
    step, _ = caller(ssd.ssd_selective_state_update, ("state",) + SEL_IN + ("y",), ("dt_bias", "D"), {})
    assert step(sel(seqlen=1, z_stride=far)) == UNSUPPORTED
    for make in (lambda: ssd.ssd_conv1d_bwd_workspace_size(conv(dx_stride=far)),
                 lambda: ssd.ssd_conv1d_bwd_workspace_size(conv(batch=1 << 20, seqlen=2, x_stride=1 << 40)),
                 lambda: ssd.ssd_group_norm_bwd_workspace_size(norm(z_stride=far)),
                 lambda: ssd.ssd_group_norm_bwd_workspace_size(norm(rows=1 << 21, z_stride=1 << 40))):
        with pytest.raises(ssd.SsdError) as e:
            make()
        assert e.value.status == UNSUPPORTED


@pytest.mark.parametrize("batch,L,D,N", [(64, 8192, 8192, 256), (128, 8192, 8192, 128), (256, 1, 8192, 256),
                                         (1, 1 << 20, 8192, 256)])
def test_large_selective_scans_are_taken(batch, L, D, N):
    """x of 17 GB at most: the scan's tensors fit a GPU's memory, and its grids are far below 2^31 blocks."""
    ssd.ssd_selective_scan_workspace_size(sel(batch=batch, seqlen=L, channels=D, dstate=N, ngroups=1))
