"""Refusals of linear attention and of the residual update, on the CPU: the C ABI returns
the documented status before anything is launched, the binding raises before any
pointer crosses it.  Fake device addresses are never dereferenced."""

import ctypes

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from test_block_abi import ALIAS, ALIGN, DTYPE, NONE, NULL, OK, SHAPE, VALUE, WORKSPACE, Call, fake, pointers


@pytest.fixture(scope="module")
def lib():
    return fb.load_library()


def linear(**kw):
    return fb.FalconLinearProblem(**{**dict(B=2, H=3, T=300, dk=64, dv=32, io_dtype=1, qk_heads=0, v_heads=0, o_heads=0, scale=0.5,
                                            q_row=192, k_row=192, v_row=96), **kw})


def residual(**kw):
    return fb.FalconResidualProblem(**{**dict(B=2, T=40, G=4, d=16, io_dtype=1, stream_dtype=0, activation=1, post_norm=1, pre_norm=1,
                                              eps=1e-6, y_row=64, gate_row=64), **kw})


def kept(first=30, **over):
    names = ("y_codes", "y_steps", "gate_codes", "gate_steps")
    return fb.FalconSavedPointers(**{n: over.get(n, fake(first + i)) for i, n in enumerate(names)})


def calls(lib):
    ws = fake(40)
    need = lib.falcon_linear_workspace_bytes(ctypes.byref(linear()))
    back = lib.falcon_linear_bwd_workspace_bytes(ctypes.byref(linear()))
    rneed = lib.falcon_residual_bwd_workspace_bytes(ctypes.byref(residual()))
    lin = ("q", "k", "v", "log_decay", "S0", "lengths")
    lb = pointers(*lin, "dO", "dS_T", "dq", "dk", "dv", "dlog_decay", "dS0")
    res = pointers("y", "gate", "h", "post_weight", "alpha", "pre_weight", "lengths", "h_out", "n")
    rb = pointers("y", "gate", "h_out", "post_weight", "alpha", "pre_weight", "lengths", "dh_out", "dn", "dy", "dgate", "dh", "dalpha",
                  "dpost_weight", "dpre_weight")
    first = {n: rb[n] for n in ("y", "gate")}
    rest = {n: rb[n] for n in ("h_out", "post_weight", "alpha", "pre_weight", "lengths")}
    grads = {n: rb[n] for n in ("dy", "dgate", "dh", "dalpha", "dpost_weight", "dpre_weight")}
    return {
        "linear_fwd": Call(lib, "falcon_linear_fwd", linear(), {**pointers(*lin, "o", "S_T"), "workspace": ws, "bytes": need}),
        "linear_step": Call(lib, "falcon_linear_step", linear(), pointers("q", "k", "v", "log_decay", "S", "is_first", "o")),
        "linear_bwd": Call(lib, "falcon_linear_bwd", linear(), {**lb, "workspace": ws, "bytes": back}),
        "residual_fwd": Call(lib, "falcon_residual_fwd", residual(), {**res, "saved": None}),
        "residual_bwd": Call(lib, "falcon_residual_bwd", residual(),
                             {**first, "saved": None, **rest, "dh_out": rb["dh_out"], "dh_out_dtype": 0, "dn": rb["dn"], "dn_dtype": 1,
                              **grads, "workspace": ws, "bytes": rneed}),
    }


@pytest.fixture(scope="module")
def call(lib):
    return calls(lib)


REQUIRED = {
    "linear_fwd": ("q", "k", "v", "log_decay", "o"), "linear_step": ("q", "k", "v", "log_decay", "S", "o"),
    "linear_bwd": ("q", "k", "v", "log_decay", "dO", "dq", "dk", "dv"), "residual_fwd": ("y", "h_out", "n"),
    "residual_bwd": ("y", "h_out", "dn", "dy", "dgate"),
}
OUTPUTS = {
    "linear_fwd": ("o", "S_T", "workspace"), "linear_step": ("o", "S"), "linear_bwd": ("dq", "dk", "dv", "dlog_decay", "dS0", "workspace"),
    "residual_fwd": ("h_out", "n"), "residual_bwd": ("dy", "dgate", "dh", "dalpha", "dpost_weight", "dpre_weight", "workspace"),
}
MAKE = {"linear": linear, "residual": residual}


@pytest.mark.parametrize("name", REQUIRED)
def test_missing_and_misaligned_pointers(call, name):
    c = call[name]
    assert c(p=None) == NULL
    for arg in REQUIRED[name]:
        assert c(**{arg: None}) == NULL, arg
    for i, (arg, v) in enumerate(c.args.items()):
        if isinstance(v, ctypes.c_void_p) and arg != "is_first":
            assert c(**{arg: fake(50 + i, misalign=8)}) == ALIGN, arg


@pytest.mark.parametrize("name", REQUIRED)
def test_problems(call, name):
    c, make = call[name], MAKE[name.split("_")[0]]
    bad = [(dict(B=-1), SHAPE), (dict(io_dtype=2), DTYPE), (dict(io_dtype=-1), DTYPE)]
    if not name.endswith("step"):
        bad += [(dict(T=-1), SHAPE), (dict(B=1 << 30, T=1 << 30), SHAPE), (dict(B=2, T=(1 << 29) + 1), SHAPE)]
    if make is linear:
        bad += [({k: v}, SHAPE) for k in ("dk", "dv") for v in (0, 8, 48, 256)]
        bad += [(dict(H=-1), SHAPE), (dict(B=1 << 12, H=1 << 10), SHAPE), (dict(scale=float("nan")), VALUE)]
        bad += [(dict(q_row=191), SHAPE), (dict(k_row=100), SHAPE), (dict(v_row=95), SHAPE), (dict(q_row=196), ALIGN), (dict(v_row=100), ALIGN)]
        bad += [({k: (1 << 22) + 8}, SHAPE) for k in ("q_row", "k_row", "v_row")]
    else:
        bad += [(dict(G=0), SHAPE), (dict(d=0), SHAPE), (dict(G=129, d=64), SHAPE), (dict(y_row=63), SHAPE), (dict(gate_row=8), SHAPE)]
        bad += [(dict(stream_dtype=2), DTYPE), (dict(activation=2), VALUE), (dict(activation=4), VALUE), (dict(eps=-1.0), VALUE),
                (dict(eps=float("inf")), VALUE)]
    for kw, want in bad:
        assert c(p=make(**kw)) == want, kw


@pytest.mark.parametrize("name", REQUIRED)
def test_outputs_overlap_nothing(call, name):
    c = call[name]
    for out in OUTPUTS[name]:
        for arg, v in c.args.items():
            same = {out, arg}
            if arg == out or not isinstance(v, ctypes.c_void_p) or same in ({"S_T", "S0"}, {"h_out", "h"}, {"dh", "dh_out"}):
                continue
            if arg == "workspace" and c.args["bytes"] == 0:
                continue
            assert c(**{out: v}) == ALIAS, (out, arg)
    inside = lambda arg: ctypes.c_void_p(c.args[arg].value + 16)  # noqa: E731
    if name == "linear_fwd":
        assert c(S_T=inside("S0")) == ALIAS
    if name == "residual_fwd":
        assert c(h_out=inside("h")) == ALIAS and c(h=c.args["h_out"], n=c.args["h_out"]) == ALIAS
    if name == "residual_bwd":
        assert c(dh=inside("dh_out")) == ALIAS
        assert c(dh=c.args["dh_out"], dh_out_dtype=1) == ALIAS     # of another type: not in place


def test_workspaces(call, lib):
    for name in ("linear_fwd", "linear_bwd", "residual_bwd"):
        c = call[name]
        need = c.args["bytes"]
        assert 0 < need < NONE
        assert c(workspace=None) == WORKSPACE and c(bytes=need - 1) == WORKSPACE
        assert c(workspace=fake(40, misalign=4)) == ALIGN
    for fn, p in (("linear", linear(dk=12)), ("linear_bwd", linear(dv=7)), ("residual_bwd", residual(G=0))):
        assert getattr(lib, f"falcon_{fn}_workspace_bytes")(ctypes.byref(p)) == NONE
    # a prompt of one tile a head takes none
    assert lib.falcon_linear_workspace_bytes(ctypes.byref(linear(B=400, H=2, q_row=128, k_row=128, v_row=64))) == 0


def test_eight_bits(call):
    f, b = call["residual_fwd"], call["residual_bwd"]
    saved = lambda **over: ctypes.byref(kept(**over))  # noqa: E731
    for n in ("y_codes", "y_steps", "gate_codes", "gate_steps"):
        assert f(saved=saved(**{n: None})) == NULL, n
        assert f(saved=saved(**{n: fake(60, misalign=4)})) == ALIGN, n
        for arg in ("y", "gate", "h", "h_out", "n", "alpha", "lengths"):
            assert f(saved=saved(**{n: f.args[arg]})) == ALIAS, (n, arg)
    assert f(saved=saved(y_codes=fake(33))) == ALIAS                       # one array twice
    assert f(gate=None, p=residual(gate_row=0), saved=saved(gate_codes=None, gate_steps=None), n=f.args["y"]) == ALIAS   # past the arrays
    none = dict(y=None, gate=None)
    assert b(saved=saved()) == VALUE and b(y=None, saved=saved()) == VALUE and b(gate=None, saved=saved()) == VALUE
    for n in ("y_codes", "y_steps", "gate_steps"):
        assert b(**none, saved=saved(**{n: None})) == NULL, n
    for n in ("y_codes", "y_steps", "gate_codes", "gate_steps"):
        assert b(**none, saved=saved(**{n: fake(60, misalign=8)})) == ALIGN, n
        assert b(**none, saved=saved(**{n: b.args["dy"]})) == ALIAS, n
    assert b(**none, saved=saved(), dgate=None) == NULL
    # rows of y and of a gate do not count where there are none
    assert b(**none, p=residual(y_row=0, gate_row=0), saved=saved(), dy=b.args["dn"]) == ALIAS
    assert b(gate=None, p=residual(gate_row=0), dy=b.args["dn"]) == ALIAS


def test_parts_that_are_left_out(call):
    f, b = call["residual_fwd"], call["residual_bwd"]
    p = residual(pre_norm=0)
    assert f(p=p, n=None, h_out=f.args["y"]) == ALIAS                      # past the check of n
    assert b(p=p, h_out=None, dn=None, dpre_weight=None, dy=b.args["y"]) == ALIAS
    assert b(dh_out_dtype=3) == DTYPE and b(dn_dtype=-1) == DTYPE


def test_nothing_to_do(call):
    lin = {a: None for a in ("q", "k", "v", "log_decay", "o")}
    assert call["linear_fwd"](p=linear(B=0), **lin, S_T=None) == OK
    assert call["linear_fwd"](p=linear(T=0), **lin, S_T=None) == OK
    assert call["linear_step"](p=linear(B=0), S=None) == OK
    assert call["residual_fwd"](p=residual(T=0), y=None, h_out=None, n=None) == OK
    assert call["residual_bwd"](p=residual(B=0), y=None, dy=None, dn=None, dalpha=None, dpost_weight=None, dpre_weight=None) == OK


# ---- the binding ---------------------------------------------------------------

bf = torch.bfloat16


def refused(cases, error=ValueError):
    for i, (f, what) in enumerate(cases):
        with pytest.raises(error, match=what):
            f()
            pytest.fail(f"case {i} was accepted")


def test_binding_refuses_linear_attention():
    q, v, g = torch.zeros(2, 3, 9, 16, dtype=bf), torch.zeros(2, 3, 9, 32, dtype=bf), torch.zeros(3)
    S, rows = torch.zeros(2, 3, 16, 32), torch.zeros(2, 9, 48, dtype=bf)
    f, b, s = fb.falcon_linear_fwd, fb.falcon_linear_bwd, fb.falcon_linear_step
    one = lambda t: t[:, :, 0].contiguous()  # noqa: E731
    refused([
        (lambda: f(q[0], q, v, g), "q"), (lambda: f(q, q.float(), v, g), "k"), (lambda: f(q, q[:, :2], v, g), "k"),
        (lambda: f(q, q, v[:1], g), "v"), (lambda: f(q, q, v, g[:2]), "heads"), (lambda: f(q, q, v, g.to(bf)), "log_decay"),
        (lambda: f(q.half(), q.half(), v.half(), g), "io dtype"), (lambda: f(q, q, v, g, S0=S.to(bf)), "S0"),
        (lambda: f(q, q, v, g, S0=S[:, :, :8]), "S0"), (lambda: f(q, q, v, g, lengths=torch.zeros(2)), "lengths"),
        (lambda: f(q.transpose(1, 2), q, v, g), ""), (lambda: f(q, q, v, g, qk_layout="columns"), "qk_layout"),
        (lambda: f(rows, rows, v, g, qk_layout="rows", v_layout="columns"), "v_layout"),
        (lambda: f(q, q, v, g, o=v.float()), "^o:"), (lambda: f(q, q, v, g, S_T=S[:1]), "S_T"),
        (lambda: f(q, q, v, g), "device"), (lambda: b(q, q, v, g, v[:, :2]), "dO"), (lambda: b(q, q, v, g, v, dS_T=S[:1]), "dS_T"),
        (lambda: b(q, q, v, g, v, grads={"dS1": S}), "unknown"), (lambda: b(q, q, v, g, v, grads={"dq": q}), "dq"),
        (lambda: s(q, q, v, g, S), "q"), (lambda: s(one(q), one(q), one(v), g, S[:1]), "^S:"),
        (lambda: s(one(q), one(q), one(v), g, S, is_first=torch.zeros(2)), "is_first"),
    ])


def test_binding_refuses_residual_updates():
    y, h, w = torch.zeros(2, 9, 48, dtype=bf), torch.zeros(2, 9, 48), torch.ones(48)
    f, b = fb.falcon_residual_fwd, fb.falcon_residual_bwd
    codes, steps = torch.zeros(2, 9, 48, dtype=torch.int8), torch.zeros(2, 9, 2, dtype=torch.uint8)
    saved = fb.FalconSaved(codes, steps, codes, steps)
    refused([
        (lambda: f(y[0]), "y: expected"), (lambda: f(y.half()), "io dtype"), (lambda: f(y, h[:1]), "^h:"),
        (lambda: f(y, gate=y.float()), "gate"), (lambda: f(y, gate=y[..., :16]), "gate"), (lambda: f(y, groups=5), "groups"),
        (lambda: f(y, groups=0), "groups"), (lambda: f(y, activation="elu1"), "activation"), (lambda: f(y, post_weight=w[:5]), "post_weight"),
        (lambda: f(y, alpha=w.to(bf)), "alpha"), (lambda: f(y, pre_weight=w.double()), "pre_weight"),
        (lambda: f(y, lengths=torch.zeros(2, dtype=torch.int64)), "lengths"), (lambda: f(y, h, h_out=y), "h_out"),
        (lambda: f(y, n=h), "^n:"), (lambda: f(y, n=y, pre_norm=False), "pre_norm"), (lambda: f(y.transpose(0, 1)), "evenly spaced"),
        (lambda: f(y), "device"), (lambda: b(y, h, h), "dn"), (lambda: b(y, None, h, y), "h_out"),
        (lambda: b(y, h, h, y, pre_norm=False), "pre_norm"), (lambda: b(y, h, h.half(), y), "dh_out"),
        (lambda: b(y, h, h, y, saved=saved), "saved"), (lambda: b(None, h, h, y, gate=y, saved=saved), "saved"),
        (lambda: b(None, h, h, y, saved=saved._replace(y_steps=steps[..., :1])), "y_steps"),
        (lambda: b(None, h, h, y, saved=saved._replace(gate_codes=codes.float())), "gate_codes"),
        (lambda: b(y, h, h, y, grads={"dgate": h}), "gate"), (lambda: b(y, None, h, pre_norm=False, grads={"dpre_weight": w}), "pre_norm"),
        (lambda: b(y, h, h, y, post_norm=False, grads={"dpost_weight": w}), "post_norm"), (lambda: b(y, h, h, y, grads={"dx": h}), "unknown"),
        (lambda: b(y, h, h, y, grads={"dalpha": w[:3]}), "dalpha"),
        (lambda: b(y, h, h, y, workspace=torch.zeros(4, dtype=torch.uint8)), "workspace"), (lambda: b(y, h, h, y), "device"),
    ])
    refused([(lambda: b(None, h, h, y, saved=[codes, steps]), "saved"), (lambda: b("y", h, h, y), "y")], (TypeError, ValueError))
    # wider rows than the kernels have reach the C ABI's status
    assert fb.falcon_residual_bwd_workspace_bytes(fb.FalconResidualProblem(1, 1, 1, 8193, 0, 0, 0, 1, 1, 1e-6, 8193, 8193)) == NONE
