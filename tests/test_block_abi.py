"""Refusals of the operators around the recurrence, on the CPU: the C ABI
returns the documented status before anything is launched, the binding raises
before any pointer crosses it.  Fake device addresses are never dereferenced."""

import ctypes

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

OK, NULL, SHAPE, DTYPE, CHUNK, ALIGN, WORKSPACE, VARIANT, HIP, VALUE, ALIAS = (
    0, -1, -2, -3, -4, -5, -6, -7, -8, -9, -10)
NONE = ctypes.c_size_t(-1).value
BASE, STRIDE = 1 << 40, 1 << 32


def fake(i, misalign=0):
    return ctypes.c_void_p(BASE + i * STRIDE + misalign)


@pytest.fixture(scope="module")
def lib():
    return fb.load_library()


def conv(**kw):
    return fb.FalconConvProblem(**{**dict(B=2, T=40, C=64, W=4, io_dtype=1, activation=1, x_row=64), **kw})


def norm(**kw):
    return fb.FalconNormProblem(**{**dict(B=2, T=40, G=4, d=64, io_dtype=1, activation=1, center=0, x_heads=0,
                                          y_heads=1, eps=1e-6, scale=1.0, x_row=256), **kw})


def scan(**kw):
    return fb.FalconScanProblem(**{**dict(B=2, T=40, D=64, N=16, G=2, io_dtype=1, softplus=1, x_row=64, dt_row=64,
                                          z_row=64, b_row=32, c_row=32), **kw})


class Call:
    """One entry point with valid arguments by name, any of which a test replaces."""

    def __init__(self, lib, name, problem, args):
        self.fn, self.problem, self.args = getattr(lib, name), problem, args

    def __call__(self, p="default", **over):
        a = {**self.args, **over}
        p = self.problem if p == "default" else p
        return self.fn(ctypes.byref(p) if p is not None else None, *a.values(), None)


def pointers(*names, absent=()):
    return {n: None if n in absent else fake(i) for i, n in enumerate(names)}


def calls(lib):
    need = {k: getattr(lib, f"falcon_{k}_workspace_bytes")(ctypes.byref(p))
            for k, p in (("conv_bwd", conv()), ("norm_bwd", norm()), ("scan_bwd", scan()), ("scan", scan()))}
    ws = fake(40)
    conv_in = ("x", "weight", "bias", "state", "lengths")
    scan_in = ("x", "dt", "A", "Bm", "Cm", "Dskip", "dt_bias", "z", "S0", "lengths")
    bwd = pointers(*conv_in, "dy", "dstate_out", "dx", "dweight", "dbias", "dstate")
    conv_bwd = {**{n: bwd[n] for n in (*conv_in, "dy")}, "dy_dtype": 0,
                **{n: bwd[n] for n in ("dstate_out", "dx", "dweight", "dbias", "dstate")}, "workspace": ws, "bytes": need["conv_bwd"]}
    nb = pointers("x", "weight", "bias", "dy", "dx", "dweight", "dbias")
    norm_bwd = {**{n: nb[n] for n in ("x", "weight", "bias", "dy")}, "dy_dtype": 0,
                **{n: nb[n] for n in ("dx", "dweight", "dbias")}, "workspace": ws, "bytes": need["norm_bwd"]}
    out = ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "ddt_bias", "dS0")
    sb = pointers(*scan_in, "dy", "dS_T", *out)
    scan_bwd = {**{n: sb[n] for n in (*scan_in, "dy")}, "dy_dtype": 0, **{n: sb[n] for n in ("dS_T", *out)}, "workspace": ws,
                "bytes": need["scan_bwd"]}
    scan_fwd = {**pointers(*scan_in, "y", "S_T"), "workspace": ws, "bytes": max(need["scan"], 16)}
    return {
        "scan_need": need["scan"],
        "conv_fwd": Call(lib, "falcon_conv_fwd", conv(), pointers(*conv_in, "y", "state_out")),
        "conv_step": Call(lib, "falcon_conv_step", conv(), pointers("x", "weight", "bias", "state", "is_first", "y")),
        "conv_bwd": Call(lib, "falcon_conv_bwd", conv(), conv_bwd),
        "norm_fwd": Call(lib, "falcon_norm_fwd", norm(), pointers("x", "weight", "bias", "y")),
        "norm_bwd": Call(lib, "falcon_norm_bwd", norm(), norm_bwd),
        "scan_fwd": Call(lib, "falcon_scan_fwd", scan(), scan_fwd),
        "scan_step": Call(lib, "falcon_scan_step", scan(), pointers("x", "dt", "A", "Bm", "Cm", "Dskip", "dt_bias", "z", "S",
                                                                    "is_first", "y")),
        "scan_bwd": Call(lib, "falcon_scan_bwd", scan(), scan_bwd),
    }


@pytest.fixture(scope="module")
def call(lib):
    return calls(lib)


REQUIRED = {
    "conv_fwd": ("x", "weight", "y"), "conv_step": ("x", "weight", "state", "y"), "conv_bwd": ("x", "weight", "dy", "dx", "dweight"),
    "norm_fwd": ("x", "y"), "norm_bwd": ("x", "dy", "dx"),
    "scan_fwd": ("x", "dt", "A", "Bm", "Cm", "y"), "scan_step": ("x", "dt", "A", "Bm", "Cm", "S", "y"),
    "scan_bwd": ("x", "dt", "A", "Bm", "Cm", "dy", "dx", "ddt", "dz", "dA", "dB", "dC"),
}
MAKE = {"conv": conv, "norm": norm, "scan": scan}


@pytest.mark.parametrize("name", REQUIRED)
def test_missing_and_misaligned_pointers(call, name):
    c = call[name]
    assert c(p=None) == NULL
    for arg in REQUIRED[name]:
        assert c(**{arg: None}) == NULL, arg
    for i, (arg, v) in enumerate(c.args.items()):
        if isinstance(v, ctypes.c_void_p) and arg not in ("is_first", "workspace"):
            assert c(**{arg: fake(50 + i, misalign=8)}) == ALIGN, arg


@pytest.mark.parametrize("name", REQUIRED)
def test_problems(call, name):
    c, make = call[name], MAKE[name.split("_")[0]]
    step = name.endswith("step")
    bad = [(dict(B=-1), SHAPE), (dict(io_dtype=2), DTYPE), (dict(io_dtype=-1), DTYPE)]
    if not step:
        bad += [(dict(T=-1), SHAPE), (dict(B=1 << 30, T=1 << 30), SHAPE), (dict(B=2, T=(1 << 29) + 1), SHAPE)]
    if make is not scan:
        bad += [(dict(activation=5), VALUE), (dict(activation=-1), VALUE)]
    if make is conv:
        bad += [(dict(W=1), SHAPE), (dict(W=5), SHAPE), (dict(C=-1), SHAPE), (dict(x_row=63), SHAPE), (dict(activation=2), VALUE)]
    if make is norm:
        bad += [(dict(d=0), SHAPE), (dict(d=4097), SHAPE), (dict(G=-1), SHAPE), (dict(x_row=255), SHAPE), (dict(eps=-1.0), VALUE),
                (dict(eps=float("nan")), VALUE), (dict(scale=float("inf")), VALUE)]
    if make is scan:
        bad += [(dict(x_row=(1 << 22) + 1), SHAPE)]
        bad += [(dict(N=12), SHAPE), (dict(N=128), SHAPE), (dict(G=0), SHAPE), (dict(G=3), SHAPE), (dict(D=-2), SHAPE)]
        bad += [({k: v}, SHAPE) for k, v in (("x_row", 63), ("dt_row", 8), ("z_row", 63), ("b_row", 31), ("c_row", 31))]
    for kw, want in bad:
        assert c(p=make(**kw)) == want, kw


def test_workspaces(call, lib):
    for name in ("conv_bwd", "norm_bwd", "scan_bwd"):
        c = call[name]
        need = c.args["bytes"]
        assert 0 < need < NONE
        assert c(workspace=None) == WORKSPACE
        assert c(bytes=need - 1) == WORKSPACE
        assert c(workspace=fake(40, misalign=4)) == ALIGN
        assert c(workspace=c.args["dx"]) == ALIAS and c(workspace=c.args["x"]) == ALIAS
    for fn, p in (("conv_bwd", conv(W=9)), ("norm_bwd", norm(d=0)), ("scan_bwd", scan(N=7)), ("scan", scan(N=7))):
        assert getattr(lib, f"falcon_{fn}_workspace_bytes")(ctypes.byref(p)) == NONE


def test_scans_of_long_prompts_need_a_workspace(call, lib):
    """Few channels and many tokens are cut into chunks, whose states it holds."""
    p = scan(B=1, T=5000)
    need = lib.falcon_scan_workspace_bytes(ctypes.byref(p))
    assert need > 0
    c = call["scan_fwd"]
    assert c(p=p, workspace=None, bytes=0) == WORKSPACE
    assert c(p=p, bytes=need - 1) == WORKSPACE
    assert c(p=p, bytes=need, workspace=fake(40, misalign=4)) == ALIGN
    for over in ("x", "S0", "y", "S_T", "lengths"):
        assert c(p=p, bytes=need, workspace=c.args[over]) == ALIAS, over


@pytest.mark.parametrize("name", REQUIRED)
def test_outputs_overlap_nothing(call, name):
    c = call[name]
    outs = {"conv_fwd": ("y", "state_out"), "conv_step": ("y", "state"), "conv_bwd": ("dx", "dweight", "dbias", "dstate"),
            "norm_fwd": ("y",), "norm_bwd": ("dx", "dweight", "dbias"), "scan_fwd": ("y", "S_T"), "scan_step": ("y", "S"),
            "scan_bwd": ("dx", "ddt", "dz", "dA", "dB", "dC", "dD", "ddt_bias", "dS0")}[name]
    for out in outs:
        for arg, v in c.args.items():
            if arg == out or not isinstance(v, ctypes.c_void_p):
                continue
            if {out, arg} == {"S_T", "S0"}:
                continue                   # may be the same
            if arg == "workspace" and name == "scan_fwd" and call["scan_need"] == 0:
                continue                   # not used
            assert c(**{out: v}) == ALIAS, (out, arg)
    if name == "scan_fwd":
        # S_T may be S0, but not a part of it
        assert c(S_T=ctypes.c_void_p(c.args["S0"].value + 16)) == ALIAS


def test_an_output_between_the_columns_of_an_input(call):
    p = conv(x_row=256)
    c = call["conv_fwd"]
    assert c(p=p, y=ctypes.c_void_p(c.args["x"].value + 128)) == ALIAS


def test_nothing_to_do(call):
    none = {a: None for a in ("x", "weight", "y")}
    assert call["conv_fwd"](p=conv(B=0), **none, state_out=None) == OK
    assert call["conv_fwd"](p=conv(T=0), **none, state_out=None) == OK
    assert call["conv_step"](p=conv(C=0, x_row=0), x=None, weight=None, state=None, y=None) == OK
    assert call["norm_fwd"](p=norm(T=0), x=None, y=None) == OK
    assert call["scan_fwd"](p=scan(B=0), x=None, A=None) == OK
    assert call["scan_fwd"](p=scan(T=0), x=None, S_T=None) == OK
    assert call["scan_step"](p=scan(B=0), S=None) == OK


def test_gate_rows_count_only_with_a_gate(call, lib):
    p = scan(z_row=0)
    assert call["scan_fwd"](p=p) == SHAPE
    assert call["scan_fwd"](p=p, z=None, y=call["scan_fwd"].args["x"]) == ALIAS   # past the problem's check


# ---- the binding ---------------------------------------------------------------

bf = torch.bfloat16


def test_binding_refuses_convolutions():
    x, w, b, s = torch.zeros(2, 9, 16, dtype=bf), torch.zeros(16, 4), torch.zeros(16), torch.zeros(2, 3, 16, dtype=bf)
    cases = [
        (lambda: fb.falcon_conv_fwd(x[0], w), "x: expected"),
        (lambda: fb.falcon_conv_fwd(x.half(), w), "io dtype"),
        (lambda: fb.falcon_conv_fwd(x, w[:8]), "weight"),
        (lambda: fb.falcon_conv_fwd(x, w.to(bf)), "weight"),
        (lambda: fb.falcon_conv_fwd(x, w[:, 0]), "weight"),
        (lambda: fb.falcon_conv_fwd(x, w, b[:3]), "bias"),
        (lambda: fb.falcon_conv_fwd(x, w, activation="relu"), "activation"),
        (lambda: fb.falcon_conv_fwd(x, w, activation="elu1"), "activation"),
        (lambda: fb.falcon_conv_fwd(x, w, state=s.float()), "state"),
        (lambda: fb.falcon_conv_fwd(x, w, state=s[:, :2]), "state"),
        (lambda: fb.falcon_conv_fwd(x, w, lengths=torch.zeros(2, dtype=torch.int64)), "lengths"),
        (lambda: fb.falcon_conv_fwd(x, w, y=x.float()), "^y:"),
        (lambda: fb.falcon_conv_fwd(x.transpose(0, 1), w), "evenly spaced"),
        (lambda: fb.falcon_conv_fwd(x[:, ::2, :].expand(2, 5, 16)[:, :, ::2], torch.zeros(8, 4)), "dense"),
        (lambda: fb.falcon_conv_fwd(x[:, :4], w), "evenly spaced"),
        (lambda: fb.falcon_conv_fwd(x[:1, :1].expand(2, 9, 16), w), "rows"),
        (lambda: fb.falcon_conv_step(x, w, s), "x: expected"),
        (lambda: fb.falcon_conv_step(x[:, 0].contiguous(), w, s, is_first=torch.zeros(2)), "is_first"),
        (lambda: fb.falcon_conv_bwd(x, w, torch.zeros(2, 9, 8)), "dy"),
        (lambda: fb.falcon_conv_bwd(x, w, x.half()), "dy"),
        (lambda: fb.falcon_conv_bwd(x, w, x, dstate_out=s), "dstate_out"),
        (lambda: fb.falcon_conv_bwd(x, w, x, grads={"dy": x}), "unknown"),
        (lambda: fb.falcon_conv_bwd(x, w, x, grads={"dx": x}), "grads"),
        (lambda: fb.falcon_conv_bwd(x, w, x, workspace=torch.zeros(4, dtype=torch.uint8)), "workspace"),
        (lambda: fb.falcon_conv_fwd(x, w), "device"),
    ]
    for i, (f, what) in enumerate(cases):
        with pytest.raises(ValueError, match=what):
            f()
            pytest.fail(f"case {i} was accepted")


def test_binding_refuses_norms():
    x, w = torch.zeros(2, 9, 16, dtype=bf), torch.ones(16)
    cases = [
        (lambda: fb.falcon_norm_fwd(x, 3), "groups"),
        (lambda: fb.falcon_norm_fwd(x, 0), "groups"),
        (lambda: fb.falcon_norm_fwd(x, 2, x_layout="heads"), "x: expected"),
        (lambda: fb.falcon_norm_fwd(torch.zeros(2, 3, 9, 8), 2, x_layout="heads"), "groups"),
        (lambda: fb.falcon_norm_fwd(torch.zeros(2, 9, 2, 8).transpose(1, 2), 2, x_layout="heads"), "contiguous"),
        (lambda: fb.falcon_norm_fwd(x, 2, y_layout="columns"), "y_layout"),
        (lambda: fb.falcon_norm_fwd(x, 2, w[:8]), "weight"),
        (lambda: fb.falcon_norm_fwd(x, 2, w, w.double()), "bias"),
        (lambda: fb.falcon_norm_fwd(x, 2, activation="relu"), "activation"),
        (lambda: fb.falcon_norm_fwd(x, 2, y_layout="heads", y=torch.zeros(2, 9, 16, dtype=bf)), "^y:"),
        (lambda: fb.falcon_norm_bwd(x, 2, torch.zeros(2, 9, 16), y_layout="heads"), "dy"),
        (lambda: fb.falcon_norm_bwd(x, 2, x, grads={"dw": w}), "unknown"),
        (lambda: fb.falcon_norm_fwd(x, 2), "device"),
    ]
    for i, (f, what) in enumerate(cases):
        with pytest.raises(ValueError, match=what):
            f()
            pytest.fail(f"case {i} was accepted")


def test_binding_refuses_scans():
    x, A, bc, v = torch.zeros(2, 9, 8), -torch.ones(8, 16), torch.zeros(2, 9, 2, 16), torch.zeros(8)
    S = torch.zeros(2, 8, 16)
    cases = [
        (lambda: fb.falcon_scan_fwd(x[0], x, A, bc, bc), "x: expected"),
        (lambda: fb.falcon_scan_fwd(x, x[:, :4], A, bc, bc), "dt"),
        (lambda: fb.falcon_scan_fwd(x, x.to(bf), A, bc, bc), "dt"),
        (lambda: fb.falcon_scan_fwd(x, x, A[:4], bc, bc), "A"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc[..., 0], bc), "B: expected"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc, bc[..., :8]), "C"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc.transpose(2, 3).contiguous().transpose(2, 3), bc), "dense"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc, bc, D=v[:4]), "^D:"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc, bc, dt_bias=v.to(bf)), "dt_bias"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc, bc, z=x[:, :3]), "z"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc, bc, S0=S.to(bf)), "S0"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc, bc, lengths=torch.zeros(3, dtype=torch.int32)), "lengths"),
        (lambda: fb.falcon_scan_step(x[:, 0].contiguous(), x[:, 0].contiguous(), A, bc[:, 0].contiguous(), bc[:, 0].contiguous(), S[:1]),
         "^S:"),
        (lambda: fb.falcon_scan_bwd(x, x, A, bc, bc, x[:, :2]), "dy"),
        (lambda: fb.falcon_scan_bwd(x, x, A, bc, bc, x, grads={"dz": x}), "dz"),
        (lambda: fb.falcon_scan_bwd(x, x, A, bc, bc, x, grads={"dA": v}), "dA"),
        (lambda: fb.falcon_scan_fwd(x, x, A, bc, bc), "device"),
    ]
    for i, (f, what) in enumerate(cases):
        with pytest.raises(ValueError, match=what):
            f()
            pytest.fail(f"case {i} was accepted")
    with pytest.raises(TypeError, match="dy"):
        fb.falcon_scan_bwd(x, x, A, bc, bc, None)
    # sizes the kernels do not have reach the C ABI's status
    A12, bc12 = -torch.ones(8, 12), torch.zeros(2, 9, 2, 12)
    assert fb.falcon_scan_workspace_bytes(fb.FalconScanProblem(2, 9, 8, 12, 2, 0, 1, 8, 8, 8, 24, 24)) == NONE
    with pytest.raises((ValueError, fb.FalconError)):
        fb.falcon_scan_fwd(x, x, A12, bc12, bc12)


def test_columns_of_one_projection_are_rows():
    wide = torch.zeros(2, 9, 48, dtype=bf)
    step = lambda t, tail=1: fb._row_step(t, "t", t.shape, bf, t.device, tail)  # noqa: E731
    assert step(wide) == 48 and step(wide[..., 16:32]) == 48 and step(wide[:, 3, :16]) == 9 * 48
    assert step(wide[..., 16:32].unflatten(-1, (2, 8)), 2) == 48
    assert step(wide[:1, :1, 8:16]) == 8          # one row: no step to take
    assert step(wide[:, :1, :16]) == 9 * 48 and step(wide[:1, :, :16]) == 48
