"""The operators around the recurrence run together, as a fast-weight block and
a state space block use them: prompts, their gradients, token by token, under
HIP graphs and on several streams."""

import numpy as np
import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb
from delta_rule_recurrence_amd import inputs as I
from oracle import block_oracle as ob
from oracle import falcon_backward as obb
from oracle import falcon_oracle as fo

from block_utils import close, draws, f64

pytestmark = pytest.mark.gpu

B, T, H, d = 2, 96, 3, 64
C = H * d


def fast_weight_parts(io, seed=31):
    n = draws(seed)
    # q, k and v side by side in one projection
    p = dict(qkv=n(B, T, 3 * C, dtype=io), conv_w=n(3 * C, 4, scale=0.5), conv_b=n(3 * C, scale=0.1),
             qk_w=1 + 0.1 * n(2 * C), qk_b=n(2 * C, scale=0.1), out_w=1 + 0.1 * n(C), out_b=n(C, scale=0.1))
    g = I.make_inputs(B, H, T, d, d, seed=seed)
    return p, g["beta"], g["lam"]


NORM = dict(activation="elu1", eps=1e-5, scale=d ** -0.5)
OUT = dict(center=True, activation="silu", eps=1e-5)


def heads(t):
    return t.reshape(B, -1, H, d).transpose(1, 2).contiguous()


def fast_weight_block(p, beta, lam):
    """conv + SiLU over q, k, v; norm + feature map of q and k into heads; the
    chunked recurrence; norm + SiLU of its heads into rows."""
    x, _ = fb.falcon_conv_fwd(p["qkv"], p["conv_w"], p["conv_b"])
    q, k, v = x.split(C, -1)
    phi_q = fb.falcon_norm_fwd(q, H, p["qk_w"][:C], p["qk_b"][:C], y_layout="heads", **NORM)
    phi_k = fb.falcon_norm_fwd(k, H, p["qk_w"][C:], p["qk_b"][C:], y_layout="heads", **NORM)
    v = heads(v)
    o, S = fb.falcon_fwd_chunked(phi_k, phi_q, v, beta, lam)
    return x, phi_q, phi_k, v, o, S, fb.falcon_norm_fwd(o, H, p["out_w"], p["out_b"], x_layout="heads", **OUT)


def test_fast_weight_block_with_gradients():
    """Forward and every gradient, stage by stage from the loss to the
    projection, against the oracles composed the same way.  float32 throughout;
    the recurrence's own bound is 1e-4 forward and 1e-5 backward, its errors
    pass through maps of slope of order one."""
    p, beta, lam = fast_weight_parts(torch.float32)
    n = draws(32)
    dy = n(B, T, C)
    D = {k: v.cuda() for k, v in p.items()}
    x, phi_q, phi_k, v, o, S, y = fast_weight_block(D, beta.cuda(), lam.cuda())

    onorm = dict(act="elu1", eps=1e-5, scale=d ** -0.5)
    oout = dict(center=True, act="silu", eps=1e-5)
    f = f64
    rx, _ = ob.conv_forward(f(p["qkv"]), f(p["conv_w"]), f(p["conv_b"]))
    rq, rk, rv = np.split(rx, 3, -1)
    wq, wk, bq, bk = f(p["qk_w"][:C]), f(p["qk_w"][C:]), f(p["qk_b"][:C]), f(p["qk_b"][C:])
    rphi_q = ob.norm_forward(rq, H, wq, bq, y_layout="heads", **onorm)
    rphi_k = ob.norm_forward(rk, H, wk, bk, y_layout="heads", **onorm)
    rvh = rv.reshape(B, T, H, d).transpose(0, 2, 1, 3)
    ro, rS = fo.falcon_forward("falcon1", rphi_k, rphi_q, rvh, f(beta), f(lam), eps=1e-6)
    ry = ob.norm_forward(ro, H, f(p["out_w"]), f(p["out_b"]), x_layout="heads", **oout)
    close(y, ry, T + d, "block output")

    # backwards
    go = fb.falcon_norm_bwd(o, H, dy.cuda(), D["out_w"], D["out_b"], x_layout="heads", **OUT)
    gr = fb.falcon_bwd_chunked(phi_k, phi_q, v, beta.cuda(), lam.cuda(), go["dx"])
    split = lambda t: t.split(C, -1)  # noqa: E731
    q, k, _ = split(x)
    gq = fb.falcon_norm_bwd(q, H, gr["dphi_q"], D["qk_w"][:C], D["qk_b"][:C], y_layout="heads", **NORM)
    gk = fb.falcon_norm_bwd(k, H, gr["dphi_k"], D["qk_w"][C:], D["qk_b"][C:], y_layout="heads", **NORM)
    dqkv = torch.cat((gq["dx"], gk["dx"], gr["dv"].transpose(1, 2).reshape(B, T, C)), -1)
    gc = fb.falcon_conv_bwd(D["qkv"], D["conv_w"], dqkv, D["conv_b"])

    ro_ = ob.norm_backward(ro, H, f(dy), f(p["out_w"]), f(p["out_b"]), x_layout="heads", **oout)
    rr = obb.falcon1_backward(rphi_k, rphi_q, rvh, f(beta), f(lam), ro_["dx"], eps=1e-6)
    rgq = ob.norm_backward(rq, H, rr["dphi_q"], wq, bq, y_layout="heads", **onorm)
    rgk = ob.norm_backward(rk, H, rr["dphi_k"], wk, bk, y_layout="heads", **onorm)
    rdv = rr["dv"].transpose(0, 2, 1, 3).reshape(B, T, C)
    rc = ob.conv_backward(f(p["qkv"]), f(p["conv_w"]), np.concatenate((rgq["dx"], rgk["dx"], rdv), -1), f(p["conv_b"]))
    for got, want, name in ((go["dweight"], ro_["dweight"], "output weights"), (gq["dweight"], rgq["dweight"], "query weights"),
                            (gk["dbias"], rgk["dbias"], "key biases"), (gr["dbeta"], rr["dbeta"], "beta"),
                            (gc["dx"], rc["dx"], "projection"), (gc["dweight"], rc["dweight"], "taps"), (gc["dbias"], rc["dbias"], "bias")):
        close(got, want, 4 * B * T, name)


def test_fast_weight_block_token_by_token():
    """A prompt by the prompt calls, then tokens by the single-token calls: the
    outputs of the whole sequence's prompt calls."""
    p, beta, lam = fast_weight_parts(torch.float32, seed=35)
    D = {k: v.cuda() for k, v in p.items()}
    beta, lam = beta.cuda(), lam.cuda()
    *_, y = fast_weight_block(D, beta, lam)
    first = T - 9
    # the prompt's part, and what goes on from it
    rows, state = fb.falcon_conv_fwd(D["qkv"][:, :first].contiguous(), D["conv_w"], D["conv_b"], return_state=True)
    q, k, v = rows.split(C, -1)
    phi_k = fb.falcon_norm_fwd(k, H, D["qk_w"][C:], D["qk_b"][C:], y_layout="heads", **NORM)
    phi_q = fb.falcon_norm_fwd(q, H, D["qk_w"][:C], D["qk_b"][:C], y_layout="heads", **NORM)
    _, S = fb.falcon_fwd_chunked(phi_k, phi_q, heads(v), beta[:, :, :first].contiguous(), lam[:, :, :first].contiguous())
    prev = phi_k[:, :, -1].contiguous()
    for t in range(first, T):
        row = fb.falcon_conv_step(D["qkv"][:, t], D["conv_w"], state, D["conv_b"])   # a column of [B, T, 3 C]
        q, k, v = row[:, None].split(C, -1)
        fq = fb.falcon_norm_fwd(q, H, D["qk_w"][:C], D["qk_b"][:C], y_layout="heads", **NORM)
        fk = fb.falcon_norm_fwd(k, H, D["qk_w"][C:], D["qk_b"][C:], y_layout="heads", **NORM)
        o = fb.falcon_decode_step(prev, fq[:, :, 0].contiguous(), v.reshape(B, H, d).contiguous(), beta[:, :, t].contiguous(),
                                  lam[:, :, t].contiguous(), S)
        out = fb.falcon_norm_fwd(o[:, :, None], H, D["out_w"], D["out_b"], x_layout="heads", **OUT)
        # two float32 ways to the same numbers
        close(out[:, 0], f64(y[:, t]), 2 * (T + d), f"token {t}")
        prev = fk[:, :, 0].contiguous()


def state_space_parts(io, D=192, N=16, seed=33):
    n = draws(seed)
    return dict(xz=n(B, T, 2 * D, dtype=io), conv_w=n(D, 4, scale=0.5), conv_b=n(D, scale=0.1), dt=n(B, T, D, dtype=io),
                bc=n(B, T, 2, 1, N, dtype=io), A=-torch.arange(1.0, N + 1).repeat(D, 1), skip=n(D), dt_bias=n(D, mean=-3.0, scale=0.3),
                norm_w=1 + 0.1 * n(D))


def state_space_block(p, D=192):
    x, z = p["xz"].split(D, -1)
    b, c = p["bc"].unbind(2)
    x, rows = fb.falcon_conv_fwd(x, p["conv_w"], p["conv_b"], return_state=True)
    y, S = fb.falcon_scan_fwd(x, p["dt"], p["A"], b, c, D=p["skip"], dt_bias=p["dt_bias"], z=z)
    return x, y, rows, S, fb.falcon_norm_fwd(y, 3, p["norm_w"])


def state_space_gradients(p, dy, x, y, D=192):
    z = p["xz"].split(D, -1)[1]
    b, c = p["bc"].unbind(2)
    gn = fb.falcon_norm_bwd(y, 3, dy, p["norm_w"])
    gs = fb.falcon_scan_bwd(x, p["dt"], p["A"], b, c, gn["dx"], D=p["skip"], dt_bias=p["dt_bias"], z=z)
    gc = fb.falcon_conv_bwd(p["xz"].split(D, -1)[0], p["conv_w"], gs["dx"], p["conv_b"])
    return gn, gs, gc


def test_state_space_block_with_gradients():
    p = state_space_parts(torch.float32)
    dy = draws(34)(B, T, 192)
    P = {k: v.cuda() for k, v in p.items()}
    x, y, rows, S, out = state_space_block(P)
    gn, gs, gc = state_space_gradients(P, dy.cuda(), x, y)
    f = {k: f64(v) for k, v in p.items()}
    fx, fz = np.split(f["xz"], 2, -1)
    a = dict(D=f["skip"], dt_bias=f["dt_bias"], z=fz)
    rx, _ = ob.conv_forward(fx, f["conv_w"], f["conv_b"])
    ry, rS = ob.scan_forward(rx, f["dt"], f["A"], f["bc"][:, :, 0], f["bc"][:, :, 1], **a)
    close(out, ob.norm_forward(ry, 3, f["norm_w"]), 2 * T, "block output")
    close(S, rS, T, "state")
    rn = ob.norm_backward(ry, 3, f64(dy), f["norm_w"])
    rs = ob.scan_backward(rx, f["dt"], f["A"], f["bc"][:, :, 0], f["bc"][:, :, 1], rn["dx"], **a)
    rc = ob.conv_backward(fx, f["conv_w"], rs["dx"], f["conv_b"])
    for got, want, name in ((gn["dweight"], rn["dweight"], "norm weights"), (gs["dA"], rs["dA"], "A"), (gs["dB"], rs["dB"], "B"),
                            (gs["dC"], rs["dC"], "C"), (gs["ddt"], rs["ddt"], "dt"), (gs["dz"], rs["dz"], "z"),
                            (gc["dx"], rc["dx"], "x"), (gc["dweight"], rc["dweight"], "taps")):
        close(got, want, 4 * B * T, name)


def test_state_space_block_token_by_token():
    p = state_space_parts(torch.bfloat16, seed=36)
    P = {k: v.cuda() for k, v in p.items()}
    whole = state_space_block(P)[-1]
    D, first = 192, T - 7
    cut = {k: (v[:, :first].contiguous() if v.dim() > 2 else v) for k, v in P.items()}
    _, _, rows, S, _ = state_space_block(cut)
    for t in range(first, T):
        x, z = P["xz"][:, t].split(D, -1)
        b, c = P["bc"][:, t].unbind(1)
        x = fb.falcon_conv_step(x, P["conv_w"], rows, P["conv_b"])
        y = fb.falcon_scan_step(x, P["dt"][:, t], P["A"], b, c, S, D=P["skip"], dt_bias=P["dt_bias"], z=z)
        out = fb.falcon_norm_fwd(y[:, None], 3, P["norm_w"])
        # bfloat16 three times on the way (x, y, the output), and once more where
        # the two float32 sums round to different neighbours
        err = (out[:, 0].float() - whole[:, t].float()).norm() / whole[:, t].float().norm()
        assert err <= 4 * 2.0 ** -8, f"token {t}: {err:.2e}"


def everything(P, W, dy):
    """Every entry point once, on the given buffers."""
    x, y, rows, S, out = state_space_block(P)
    gn, gs, gc = state_space_gradients(P, dy, x, y)
    row = fb.falcon_conv_step(P["xz"].split(192, -1)[0][:, 3], P["conv_w"], W["rows"].copy_(rows), P["conv_b"])
    b, c = P["bc"][:, 3].unbind(1)
    step = fb.falcon_scan_step(row, P["dt"][:, 3], P["A"], b, c, W["S"].copy_(S), D=P["skip"], dt_bias=P["dt_bias"])
    named = {"out": out, "rows": rows, "S": S, "row": row, "step": step, "rows after": W["rows"].clone(), "S after": W["S"].clone()}
    for g in (gn, gs, gc):
        named.update({f"{len(named)} {k}": v for k, v in g.items() if v is not None})
    return named


def test_graph_replay():
    """All of it captured into one HIP graph; replays on other contents, with
    eager calls of the same kind between them, give the eager results."""
    P = {k: v.cuda() for k, v in state_space_parts(torch.bfloat16).items()}
    Q = {k: v.cuda() for k, v in state_space_parts(torch.bfloat16, seed=77).items()}
    dy = draws(40)(B, T, 192).cuda()
    W = dict(rows=torch.empty(B, 3, 192, dtype=torch.bfloat16, device="cuda"), S=torch.empty(B, 192, 16, device="cuda"))
    want = {name: {k: v.clone() for k, v in everything(p, W, dy).items()} for name, p in (("P", P), ("Q", Q))}
    held = {k: v.clone() for k, v in P.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(held, W, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(held, W, dy)
    for turn, name in enumerate(("P", "Q", "Q", "P")):
        for k, v in held.items():
            v.copy_((P if name == "P" else Q)[k])
        graph.replay()
        torch.cuda.synchronize()
        for k, v in got.items():
            assert torch.equal(v, want[name][k]), f"replay {turn}: {k}"
        everything(Q if name == "P" else P, W, dy)
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls on two streams, interleaved, keep apart what each allocates."""
    P = {k: v.cuda() for k, v in state_space_parts(torch.bfloat16).items()}
    Q = {k: v.cuda() for k, v in state_space_parts(torch.bfloat16, seed=78).items()}
    dy = draws(41)(B, T, 192).cuda()
    W = [dict(rows=torch.empty(B, 3, 192, dtype=torch.bfloat16, device="cuda"), S=torch.empty(B, 192, 16, device="cuda")) for _ in "12"]
    want = [{k: v.clone() for k, v in everything(p, w, dy).items()} for p, w in zip((P, Q), W)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, p, w in zip(streams, (P, Q), W):
            with torch.cuda.stream(s):
                got.append(everything(p, w, dy))
        torch.cuda.synchronize()
        for g, r in zip(got, want):
            for k, v in g.items():
                assert torch.equal(v, r[k]), k


def test_stream_argument():
    """`stream=` launches there and takes what it allocates from there."""
    n = draws(42)
    x, w, dy = n(4, 200, 72).cuda(), n(72, 4).cuda(), n(4, 200, 72).cuda()
    want, grads = fb.falcon_conv_fwd(x, w)[0], fb.falcon_conv_bwd(x, w, dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y, _ = fb.falcon_conv_fwd(x, w, stream=s)
        g = fb.falcon_conv_bwd(x, w, dy, stream=s)
        s.synchronize()
        assert torch.equal(y, want) and torch.equal(g["dweight"], grads["dweight"]) and torch.equal(g["dx"], grads["dx"])


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one device")
def test_other_device():
    n = draws(43)
    x, w = n(2, 50, 24), n(24, 4)
    want, _ = fb.falcon_conv_fwd(x.cuda(0), w.cuda(0))
    with torch.cuda.device(0):
        got, _ = fb.falcon_conv_fwd(x.cuda(1), w.cuda(1))
    assert got.device.index == 1 and torch.equal(got.cpu(), want.cpu())
