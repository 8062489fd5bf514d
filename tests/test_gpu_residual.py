"""The residual update between two blocks, its gradients and its 8 bits against their
oracle, on the GPU."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from oracle import residual_oracle as ro

from block_utils import IO, UNIT, close, columns, cuda, draws, f64

pytestmark = pytest.mark.gpu

# (B, T, G, d, y's type, the stream's type, gate, post norm, pre norm, weights, h, lengths, columns of a wider y and gate)
CASES = [
    (1, 1, 1, 1, "f32", "f32", "silu", True, True, True, True, None, False),
    (1, 1, 1, 33, "bf16", "f32", "none", True, True, True, True, None, False),
    (2, 37, 12, 64, "bf16", "f32", "silu", True, True, True, True, None, False),
    (2, 19, 3, 128, "f32", "bf16", "sigmoid", True, True, True, True, None, True),
    (3, 7, 5, 16, "bf16", "bf16", "identity", True, False, False, False, None, False),
    (1, 65, 7, 9, "f32", "f32", "silu", True, True, True, True, None, False),
    (2, 11, 2, 80, "bf16", "f32", "silu", False, True, True, True, None, True),
    (2, 5, 3, 33, "bf16", "bf16", "silu", True, True, False, True, None, True),
    (1, 9, 40, 32, "bf16", "f32", "sigmoid", True, True, True, True, None, False),
    (1, 6, 2, 600, "f32", "f32", "silu", True, True, True, False, None, False),
    (1, 5, 1, 1001, "bf16", "f32", "none", True, False, True, True, None, True),
    (1, 3, 3, 512, "f32", "f32", "silu", True, True, True, True, None, False),
    (1, 3, 2, 1024, "bf16", "bf16", "silu", True, True, True, True, None, False),
    (1, 3, 1, 8192, "bf16", "f32", "silu", True, True, True, True, None, False),
    (1, 3, 1, 8191, "f32", "f32", "silu", True, True, True, True, None, False),
    (1, 2, 4096, 2, "f32", "f32", "silu", True, True, True, True, None, False),
    (1, 1300, 6, 64, "f32", "f32", "silu", True, True, True, True, None, True),
    (300, 3, 1, 8, "f32", "f32", "silu", True, True, True, True, None, False),
    (2, 2049, 2, 8, "bf16", "bf16", "none", False, True, True, True, None, False),
    (4, 50, 3, 24, "bf16", "f32", "silu", True, True, True, True, [0, 1, 50, 33], False),
    (3, 21, 1, 77, "f32", "bf16", "sigmoid", True, True, True, True, [21, 0, 20], True),
]


def inputs(case, seed=3):
    B, T, G, d, io, stream, gate, post, pre, weights, has_h, lengths, wide = case
    n, C = draws(seed), G * d
    w = lambda on: n(C, scale=0.3, mean=1.0) if on and weights else None  # noqa: E731
    t = dict(y=n(B, T, C, dtype=IO[io], mean=0.3), h=n(B, T, C, dtype=IO[stream]) if has_h else None,
             gate=n(B, T, C, dtype=IO[io]) if gate != "none" else None)
    p = dict(post_weight=w(post), alpha=w(True), pre_weight=w(pre))
    a = dict(groups=G, post_norm=post, pre_norm=pre, eps=1e-5)
    back = dict(h_out=n(B, T, C, dtype=IO[stream]) if pre else None, dh_out=n(B, T, C), dn=n(B, T, C, dtype=IO[io]) if pre else None)
    return t, p, a, back, "none" if gate in ("none", "identity") else gate


def ends_of(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32)


def wide_or_not(t, wide):
    return None if t is None else columns(t) if wide else t.cuda()


def oracle_forward(t, p, a, act, lengths):
    return ro.residual_forward(f64(t["y"]), f64(t["h"]), gate=f64(t["gate"]), act=act, lengths=lengths,
                               **{k: f64(v) for k, v in p.items()}, **a)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    lengths, wide = case[-2:]
    t, p, a, _, act = inputs(case)
    want, n_want = oracle_forward(t, p, a, act, lengths)
    h_out, n, kept = fb.falcon_residual_fwd(wide_or_not(t["y"], wide), cuda(t["h"]), gate=wide_or_not(t["gate"], wide), activation=act,
                                            lengths=cuda(ends_of(lengths)), **{k: cuda(v) for k, v in p.items()}, **a)
    C = case[2] * case[3]
    assert kept is None and h_out.dtype == (t["h"] if t["h"] is not None else t["y"]).dtype
    close(h_out, want, case[3], "h_out")
    if a["pre_norm"]:
        close(n, n_want, C + case[3], "n")
    else:
        assert n is None


def gradients_close(g, want, t, p, a, back, case):
    B, T, G, d = case[:4]
    C = G * d
    close(g["dh"], want["dh"], 2 * C, "dh") if case[10] else None
    if t["gate"] is not None:
        close(g["dgate"], want["dgate"], 2 * C + d, "dgate")
    if a["post_norm"] and d <= 2:
        # One or two channels a group: dy is what cancels.  s - yhat mean(s yhat) of terms up to
        # 2 |s| (|yhat| <= sqrt(d)), over the root of the group: off by the terms' errors.
        # sized by the errors of s, of 4 (16 + 2 C) units, and a few more of the difference.
        root = np.sqrt((f64(t["y"]).reshape(B, T, G, d) ** 2).mean(-1, keepdims=True) + a["eps"])
        size = (np.abs(want["dh"]) * 4).reshape(B, T, G, d) / root
        for q in (p["alpha"], p["post_weight"]):
            if q is not None:
                size = size * np.abs(f64(q)).reshape(G, d).max()
        if t["gate"] is not None:
            size = size * (1 + np.abs(f64(t["gate"])).reshape(B, T, G, d).max())
        assert np.abs(f64(g["dy"]) - want["dy"]).max() <= 4 * (20 + 2 * C) * UNIT * size.max()
    else:
        close(g["dy"], want["dy"], 2 * C + 2 * d, "dy")
    for name, on in (("dalpha", p["alpha"] is not None), ("dpost_weight", p["post_weight"] is not None),
                     ("dpre_weight", p["pre_weight"] is not None)):
        if on:
            close(g[name], want[name], B * T + 2 * C, name)
        else:
            assert g[name] is None


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradients(case):
    lengths, wide = case[-2:]
    t, p, a, back, act = inputs(case)
    want = ro.residual_backward(f64(t["y"]), f64(back["h_out"]), f64(back["dh_out"]), f64(back["dn"]), gate=f64(t["gate"]), act=act,
                                lengths=lengths, **{k: f64(v) for k, v in p.items()}, **a)
    g = fb.falcon_residual_bwd(wide_or_not(t["y"], wide), *(cuda(back[k]) for k in ("h_out", "dh_out", "dn")),
                               gate=wide_or_not(t["gate"], wide), activation=act, lengths=cuda(ends_of(lengths)), added=case[10],
                               **{k: cuda(v) for k, v in p.items()}, **a)
    gradients_close(g, want, t, p, a, back, case)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_eight_bits(case):
    """What the forward keeps is what 8 bits of y and gate are, to the bit, and the backward
    pass from it is that of those values."""
    lengths, wide = case[-2:]
    t, p, a, back, act = inputs(case)
    args = dict(activation=act, lengths=cuda(ends_of(lengths)), **{k: cuda(v) for k, v in p.items()}, **a)
    h_out, n, kept = fb.falcon_residual_fwd(wide_or_not(t["y"], wide), cuda(t["h"]), gate=wide_or_not(t["gate"], wide), save=True, **args)
    plain = fb.falcon_residual_fwd(wide_or_not(t["y"], wide), cuda(t["h"]), gate=wide_or_not(t["gate"], wide), **args)
    assert torch.equal(h_out, plain[0]) and (n is None or torch.equal(n, plain[1]))
    C = case[2] * case[3]
    values = {}
    for name, codes, steps in (("y", kept.y_codes, kept.y_steps), ("gate", kept.gate_codes, kept.gate_steps)):
        if t[name] is None:
            assert codes is None and steps is None
            values[name] = None
            continue
        want = ro.eight_bits(f64(t[name]))
        for b, end in enumerate(lengths or ()):
            want[b, end:] = 0
        step = np.exp2(steps.cpu().numpy().astype(np.float64) - 127).repeat(32, -1)[..., :C]
        values[name] = codes.cpu().numpy().astype(np.float64) * step
        assert np.array_equal(values[name], want), name
    want = ro.residual_backward(values["y"], f64(back["h_out"]), f64(back["dh_out"]), f64(back["dn"]), gate=values["gate"], act=act,
                                lengths=lengths, **{k: f64(v) for k, v in p.items()}, **a)
    g = fb.falcon_residual_bwd(None, *(cuda(back[k]) for k in ("h_out", "dh_out", "dn")), saved=kept, added=case[10], **args)
    t = dict(t, y=torch.from_numpy(values["y"]))
    gradients_close(g, want, t, p, a, back, case)


@pytest.mark.parametrize("dh_type,dn_type", [("bf16", "f32"), ("f32", "bf16"), (None, "bf16")])
def test_types_of_incoming_gradients(dh_type, dn_type):
    case = CASES[2]
    t, p, a, back, act = inputs(case)
    dh = None if dh_type is None else back["dh_out"].to(IO[dh_type])
    dn = back["dn"].to(IO[dn_type])
    want = ro.residual_backward(f64(t["y"]), f64(back["h_out"]), f64(dh), f64(dn), gate=f64(t["gate"]), act=act,
                                **{k: f64(v) for k, v in p.items()}, **a)
    g = fb.falcon_residual_bwd(t["y"].cuda(), back["h_out"].cuda(), cuda(dh), dn.cuda(), gate=t["gate"].cuda(), activation=act,
                               **{k: cuda(v) for k, v in p.items()}, **a)
    gradients_close(g, want, t, p, a, back, case)


def test_gradients_of_absent_parameters_may_be_asked_for():
    case = CASES[7]
    t, p, a, back, act = inputs(case)
    C = case[2] * case[3]
    asked = {k: torch.empty(C, device="cuda") for k in ("dalpha", "dpost_weight", "dpre_weight")}
    want = ro.residual_backward(f64(t["y"]), f64(back["h_out"]), f64(back["dh_out"]), f64(back["dn"]), gate=f64(t["gate"]), act=act, **a)
    g = fb.falcon_residual_bwd(t["y"].cuda(), *(cuda(back[k]) for k in ("h_out", "dh_out", "dn")), gate=t["gate"].cuda(),
                               activation=act, added=False, grads=asked, **a)
    assert g["dh"] is None
    for k in asked:
        assert g[k] is asked[k]
        close(g[k], want[k], case[0] * case[1] + 2 * C, k)


@pytest.mark.parametrize("G,d", [(12, 64), (3, 24), (1, 77)])
def test_padded_batches(G, d):
    """Rows behind the ends are not read; outputs there stay, gradients are zero."""
    lengths, B, T, C = [0, 1, 30, 19], 4, 30, G * d
    n = draws(41)
    t = {k: n(B, T, C) for k in ("y", "h", "gate", "h_out", "dh_out", "dn")}
    w = n(C, scale=0.3, mean=1.0)
    clean = {k: v.clone() for k, v in t.items()}
    for b, end in enumerate(lengths):
        for k in t:
            t[k][b, end:] = float("nan")
    D = {k: v.cuda() for k, v in t.items()}
    seven = lambda *s, dtype=torch.float32: torch.full(s, 7, dtype=dtype, device="cuda")  # noqa: E731
    kept = fb.FalconSaved(seven(B, T, C, dtype=torch.int8), seven(B, T, (C + 31) // 32, dtype=torch.uint8),
                          seven(B, T, C, dtype=torch.int8), seven(B, T, (C + 31) // 32, dtype=torch.uint8))
    a = dict(groups=G, post_weight=w.cuda(), pre_weight=w.cuda(), alpha=w.cuda(), lengths=ends_of(lengths).cuda())
    h_out, normed = seven(B, T, C), seven(B, T, C)
    fb.falcon_residual_fwd(D["y"], D["h"], gate=D["gate"], h_out=h_out, n=normed, saved=kept, **a)
    want, n_want = ro.residual_forward(f64(clean["y"]), f64(clean["h"]), gate=f64(clean["gate"]), groups=G, post_weight=f64(w),
                                       pre_weight=f64(w), alpha=f64(w), lengths=lengths)
    for b, end in enumerate(lengths):
        for x in (h_out, normed, *kept):
            assert torch.all(x[b, end:] == 7)
        h_out[b, end:] = 0
        normed[b, end:] = 0
    close(h_out, want, d, "h_out")
    close(normed, n_want, C + d, "n")
    for from_8 in (False, True):
        src = dict(saved=kept) if from_8 else dict(gate=D["gate"])
        g = fb.falcon_residual_bwd(None if from_8 else D["y"], D["h_out"], D["dh_out"], D["dn"], **src, **a)
        value = ro.eight_bits if from_8 else (lambda x: x)
        ref = ro.residual_backward(value(f64(clean["y"])), f64(clean["h_out"]), f64(clean["dh_out"]), f64(clean["dn"]),
                                   gate=value(f64(clean["gate"])), groups=G, post_weight=f64(w), pre_weight=f64(w), alpha=f64(w), lengths=lengths)
        for k in ("dy", "dgate", "dh"):
            close(g[k], ref[k], 2 * C + 2 * d, k)
            for b, end in enumerate(lengths):
                assert torch.all(g[k][b, end:] == 0)
        for k in ("dalpha", "dpost_weight", "dpre_weight"):
            close(g[k], ref[k], B * T + 2 * C, k)


def test_in_place():
    """h_out over h and dh over dh_out."""
    n = draws(43)
    y, h, gate, dn, dh = (n(3, 40, 192).cuda() for _ in range(5))
    want, n1, _ = fb.falcon_residual_fwd(y, h, gate=gate, groups=3)
    stream = h.clone()
    got, n2, _ = fb.falcon_residual_fwd(y, stream, gate=gate, groups=3, h_out=stream)
    assert got is stream and torch.equal(got, want) and torch.equal(n1, n2)
    ref = fb.falcon_residual_bwd(y, want, dh, dn, gate=gate, groups=3)
    into = dh.clone()
    g = fb.falcon_residual_bwd(y, want, into, dn, gate=gate, groups=3, grads={"dh": into})
    assert g["dh"] is into
    for k in ("dy", "dgate", "dh"):
        assert torch.equal(g[k], ref[k])


def test_values_that_are_not_finite_stay_in_their_row():
    n = draws(45)
    y, h, gate, dn, dh = (n(2, 20, 96).cuda() for _ in range(5))
    a = dict(groups=3)
    clean = fb.falcon_residual_fwd(y, h, gate=gate, save=True, **a)
    bad = [t.clone() for t in (y, h, gate)]
    bad[0][0, 3, 5], bad[1][0, 4, 6], bad[2][1, 5, 70] = float("inf"), float("nan"), -float("inf")
    h_out, normed, kept = fb.falcon_residual_fwd(bad[0], bad[1], gate=bad[2], save=True, **a)
    rows = torch.ones(2, 20, dtype=torch.bool, device="cuda")
    rows[0, 3] = rows[0, 4] = rows[1, 5] = False
    for got, want in zip((h_out, normed, *kept), (*clean[:2], *clean[2])):
        assert torch.equal(got[rows], want[rows])
    assert h_out[0, 4, 6].isnan() and normed[0, 4].isnan().all()
    # the block of 32 channels that holds it is NaN in 8 bits, the others stand
    assert kept.y_steps[0, 3].tolist()[0] == 255 and torch.all(kept.y_codes[0, 3, :32] == 0)
    assert torch.equal(kept.y_codes[0, 3, 32:], clean[2].y_codes[0, 3, 32:])
    g0 = fb.falcon_residual_bwd(None, clean[0], dh, dn, saved=clean[2], **a)
    g = fb.falcon_residual_bwd(None, clean[0], dh, dn, saved=kept, **a)
    for k in ("dy", "dgate", "dh"):
        assert torch.equal(g[k][rows], g0[k][rows])
    assert g["dy"][0, 3, :32].isnan().all()
    assert torch.isfinite(g["dy"][0, 3, 32:]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("G,d", [(3, 64), (2, 5), (1, 1000)])
@pytest.mark.parametrize("exponent,eps", [(66, 1e-6), (100, 1e-6), (113, 1e-6), (-64, 0.0), (-90, 0.0)])
def test_squares_out_of_range(io, G, d, exponent, eps):
    """Rows whose squares leave float32's normal numbers, above and below."""
    n, T, C = draws(71), 6, G * d
    y, h = n(1, T, C, mean=0.5), n(1, T, C)
    y[:, ::2] *= 2.0 ** exponent
    h[:, ::3] *= 2.0 ** exponent
    y, h = y.to(IO[io]), h.to(IO[io])
    dh, dn = n(1, T, C), n(1, T, C)
    a = dict(groups=G, eps=eps)
    h_out, normed, _ = fb.falcon_residual_fwd(y.cuda(), h.cuda(), **a)
    want, n_want = ro.residual_forward(f64(y), f64(h), **a)
    for row in range(T):
        close(h_out[:, row], want[:, row], d, f"h_out of row {row}")
        close(normed[:, row], n_want[:, row], C + d, f"n of row {row}")
    _, alone, _ = fb.falcon_residual_fwd(h.cuda(), post_norm=False, **a)
    close(alone, ro.residual_forward(f64(h), post_norm=False, **a)[1], C, "n alone")
    g = fb.falcon_residual_bwd(y.cuda(), h.cuda(), dh.cuda(), dn.cuda(), **a)
    ref = ro.residual_backward(f64(y), f64(h), f64(dh), f64(dn), **a)
    for row in range(T):
        # compared at a size of about one: dy is of the size of dh over y, dh of dn over h
        small_h = 2.0 ** min(exponent, 0) if row % 3 == 0 else 1.0
        size = (2.0 ** exponent if row % 2 == 0 else 1.0) * small_h
        close((g["dh"][0, row].double() * small_h).float(), ref["dh"][0, row] * small_h, 2 * C, f"dh of row {row}")
        if np.abs(ref["dy"][0, row]).max() < 2.0 ** 127:
            close((g["dy"][0, row].double() * size).float(), ref["dy"][0, row] * size, 2 * C + 2 * d, f"dy of row {row}")


def test_zero_rows():
    """A row of zeros norms to zero (eps keeps it finite); its gradients are finite."""
    z = torch.zeros(1, 3, 64, device="cuda")
    h_out, n, kept = fb.falcon_residual_fwd(z, z, gate=z, groups=2, save=True)
    assert torch.all(h_out == 0) and torch.all(n == 0) and torch.all(kept.y_codes == 0)
    g = fb.falcon_residual_bwd(z, h_out, z + 1, z + 1, gate=z, groups=2)
    assert all(torch.isfinite(g[k]).all() for k in ("dy", "dgate", "dh"))


def test_empty_calls():
    z = torch.zeros(2, 0, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    h_out, n, kept = fb.falcon_residual_fwd(z, z, gate=z, pre_weight=w, save=True)
    assert h_out.shape == n.shape == kept.y_codes.shape == (2, 0, 32)
    g = fb.falcon_residual_bwd(z, h_out, z, z, gate=z, alpha=w, post_weight=w, pre_weight=w)
    assert all(torch.all(g[k] == 0) for k in ("dalpha", "dpost_weight", "dpre_weight"))


def test_results_are_the_same_every_time():
    n = draws(21)
    y, gate, h, dh, dn = (n(3, 900, 768).cuda() for _ in range(5))
    w = n(768).cuda()
    a = dict(gate=gate, groups=12, post_weight=w, alpha=w, pre_weight=w)
    first = fb.falcon_residual_bwd(y, h, dh, dn, **a)
    for _ in range(3):
        again = fb.falcon_residual_bwd(y, h, dh, dn, **a)
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("C", [8, 2048])
def test_sums_of_one_sign_over_many_tokens(C):
    """Parameter gradients that all have one sign and size, whose rounding errors do not
    cancel: y, h_out and the gradients are one everywhere, so dalpha is the tokens over
    sqrt(1 + eps).  A thread adds at most 64 rows in float32, each off by 2^-24 of a partial
    sum; what joins the threads is in double, its parts are rounded once; at most 8
    operations make a term."""
    tokens = 1 << 18
    one = torch.ones(1, tokens, C, dtype=torch.bfloat16, device="cuda")
    dn, w = one.float(), torch.ones(C, device="cuda")
    g = fb.falcon_residual_bwd(one, one, None, dn, post_weight=w, alpha=w, pre_weight=w)
    want = tokens / (1 + 1e-6) ** 0.5
    err = float((g["dpre_weight"].double() / want - 1).abs().max())
    assert err <= (64 + 2 + 8) * UNIT
    g = fb.falcon_residual_bwd(one, None, dn, pre_norm=False, post_weight=w, alpha=w)
    for k in ("dalpha", "dpost_weight"):
        assert float((g[k].double() / want - 1).abs().max()) <= (64 + 2 + 8) * UNIT, k


@pytest.mark.parametrize("d", [64, 33])
def test_zeros_behind_the_ends_whatever_the_weights(d):
    n, C = draws(47), 2 * d
    y, h, dh, dn, gate = (n(2, 9, C).cuda() for _ in range(5))
    w = torch.full((C,), float("inf"), device="cuda")
    ends = torch.tensor([4, 0], dtype=torch.int32, device="cuda")
    g = fb.falcon_residual_bwd(y, h, dh, dn, gate=gate, groups=2, post_weight=w, alpha=w, pre_weight=w, lengths=ends)
    for k in ("dy", "dgate", "dh"):
        assert torch.all(g[k][0, 4:] == 0) and torch.all(g[k][1] == 0)


@pytest.mark.parametrize("C", [2, 7, 8, 9, 15, 17, 31, 65, 505, 511, 513, 519, 521, 1025, 2049, 4095, 4099])
@pytest.mark.parametrize("post,io", [(True, "bf16"), (False, "f32")])
def test_widths_around_a_piece(C, post, io):
    """Rows whose last piece of 8 channels is short, alone in a wave among them, in place."""
    n, T = draws(80 + C), 5
    y, gate = n(2, T, C, dtype=IO[io]), n(2, T, C, dtype=IO[io])
    h, dh, dn = n(2, T, C), n(2, T, C), n(2, T, C)
    w = n(C, scale=0.3, mean=1.0)
    a = dict(post_norm=post, eps=1e-5)
    p = dict(post_weight=w if post else None, alpha=w, pre_weight=w)
    stream = h.cuda()
    h_out, normed, kept = fb.falcon_residual_fwd(y.cuda(), stream, gate=gate.cuda(), h_out=stream, save=True,
                                                 **{k: cuda(v) for k, v in p.items()}, **a)
    want, n_want = ro.residual_forward(f64(y), f64(h), gate=f64(gate), **{k: f64(v) for k, v in p.items()}, **a)
    close(h_out, want, C, "h_out")
    close(normed, n_want, 2 * C, "n")
    into = dh.cuda()
    g = fb.falcon_residual_bwd(None, h_out, into, dn.cuda(), saved=kept, grads={"dh": into}, **{k: cuda(v) for k, v in p.items()}, **a)
    ref = ro.residual_backward(ro.eight_bits(f64(y)), f64(h_out), f64(dh), f64(dn), gate=ro.eight_bits(f64(gate)),
                               **{k: f64(v) for k, v in p.items()}, **a)
    for k in ("dh", "dgate", *(() if post and C == 2 else ("dy",))):
        close(g[k], ref[k], 4 * C, k)
    for k in ("dalpha", "dpre_weight", *(("dpost_weight",) if post else ())):
        close(g[k], ref[k], 2 * T + 2 * C, k)


@pytest.mark.parametrize("C", [96, 77, 5])
def test_outputs_given_and_allocated_on_padded_batches(C):
    """Those given stay behind the ends, those allocated are zero there."""
    n = draws(51)
    y, h = n(3, 20, C).cuda(), n(3, 20, C).cuda()
    ends = torch.tensor([20, 7, 0], dtype=torch.int32, device="cuda")
    behind = torch.arange(20, device="cuda")[None] >= ends[:, None]
    want = fb.falcon_residual_fwd(y, h, gate=y, lengths=ends, save=True)
    assert all(torch.all(t[behind] == 0) for t in (*want[:2], *want[2]))
    for given in ("h_out", "n", "saved"):
        seven = lambda t: torch.full_like(t, 7)  # noqa: E731
        into = {"h_out": seven(h), "n": seven(y), "saved": fb.FalconSaved(*(seven(t) for t in want[2]))}[given]
        h_out, normed, kept = fb.falcon_residual_fwd(y, h, gate=y, lengths=ends, save=True, **{given: into})
        for name, got, ref in (("h_out", h_out, want[0]), ("n", normed, want[1]), *(("saved", a, b) for a, b in zip(kept, want[2]))):
            assert torch.equal(got[~behind], ref[~behind])
            assert torch.all(got[behind] == (7 if name == given else 0)), (given, name)
