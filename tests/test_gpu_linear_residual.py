"""Linear attention and the residual update as they are used: a block's training step
against automatic differentiation in 64 bits, a prompt and the tokens behind it, HIP
graphs, streams, and tensors whose offsets pass 32 bits."""

import pytest
import torch

from delta_rule_recurrence_amd import falcon as fb

from block_utils import IO, UNIT, close, draws, f64
from test_gpu_block_graph import replayed

pytestmark = pytest.mark.gpu


# ---- a block: projections, linear attention, heads normed and gated, projection, residual --------

B, T, H, D = 2, 150, 3, 32
C = H * D
NORM = dict(groups=H, pre_norm=False, activation="silu")


def block_inputs(seed):
    n = draws(seed)
    p = dict(w_in=n(C, 4 * C, scale=C ** -0.5), w_out=n(C, C, scale=C ** -0.5), log_decay=-torch.rand(H) - 0.01,
             head_weight=n(C, scale=0.2, mean=1.0), alpha=n(C, scale=0.2, mean=0.5), post_weight=n(C, scale=0.2, mean=1.0),
             pre_weight=n(C, scale=0.2, mean=1.0))
    return p, n(B, T, C), n(B, T, C), n(B, T, C)


def block_forward(p, x, save=False):
    """The stream x, normed for the block by the residual update of the block before it."""
    _, n0, _ = fb.falcon_residual_fwd(x, post_norm=False, pre_weight=p["pre_weight"], eps=1e-5)
    wide = n0 @ p["w_in"]
    q, k, v, gate = (wide[..., i * C:(i + 1) * C] for i in range(4))       # columns of one projection
    o, _ = fb.falcon_linear_fwd(q, k, v, p["log_decay"], scale=D ** -0.5, qk_layout="rows", v_layout="rows", o_layout="rows")
    z, _, _ = fb.falcon_residual_fwd(o, gate=gate, post_weight=p["head_weight"], eps=1e-5, **NORM)
    y = z @ p["w_out"]
    h_out, n1, kept = fb.falcon_residual_fwd(y, x, post_weight=p["post_weight"], alpha=p["alpha"], pre_weight=p["pre_weight"], eps=1e-5,
                                             save=save)
    return dict(n0=n0, q=q, k=k, v=v, gate=gate, o=o, z=z, y=y, h_out=h_out, n1=n1, kept=kept)


def block_backward(p, x, s, dh_out, dn1):
    kept = s["kept"]
    g = fb.falcon_residual_bwd(None if kept else s["y"], s["h_out"], dh_out, dn1, saved=kept, post_weight=p["post_weight"], alpha=p["alpha"],
                               pre_weight=p["pre_weight"], eps=1e-5)
    grads = {k: g["d" + k] for k in ("post_weight", "alpha", "pre_weight")}
    rows = lambda t: t.flatten(0, 1)  # noqa: E731
    grads["w_out"] = rows(s["z"]).T @ rows(g["dy"])
    gz = fb.falcon_residual_bwd(s["o"], None, g["dy"] @ p["w_out"].T, gate=s["gate"], post_weight=p["head_weight"], eps=1e-5, added=False,
                                **NORM)
    grads["head_weight"] = gz["dpost_weight"]
    gl = fb.falcon_linear_bwd(s["q"], s["k"], s["v"], p["log_decay"], gz["dy"], scale=D ** -0.5, learned_decay=True, qk_layout="rows",
                              v_layout="rows", o_layout="rows")
    grads["log_decay"] = gl["dlog_decay"]
    dwide = torch.cat((gl["dq"], gl["dk"], gl["dv"], gz["dgate"]), -1)
    grads["w_in"] = rows(s["n0"]).T @ rows(dwide)
    g0 = fb.falcon_residual_bwd(x, x, g["dh"], dwide @ p["w_in"].T, post_norm=False, pre_weight=p["pre_weight"], eps=1e-5, added=False)
    grads["pre_weight"] = grads["pre_weight"] + g0["dpre_weight"]
    return grads, g0["dy"]


def block_exact(p, x, dh_out, dn1):
    """The same in 64 bits by torch's own differentiation, on the CPU."""
    p = {k: v.double().requires_grad_() for k, v in p.items()}
    x = x.double().requires_grad_()
    norm = lambda t: t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt()  # noqa: E731
    q, k, v, gate = ((norm(x) * p["pre_weight"]) @ p["w_in"]).split(C, -1)
    head = lambda t: t.reshape(B, T, H, D).transpose(1, 2)  # noqa: E731
    gap = torch.arange(T)[:, None] - torch.arange(T)[None]
    w = torch.where(gap >= 0, (p["log_decay"][:, None, None] * gap.clamp(min=0)).exp(), 0.0)
    o = (head(q) @ head(k).transpose(2, 3) * w) @ head(v) * D ** -0.5
    z = norm(o).transpose(1, 2).reshape(B, T, C) * p["head_weight"] * torch.nn.functional.silu(gate)
    y = z @ p["w_out"]
    h_out = x + p["alpha"] * norm(y) * p["post_weight"]
    n1 = norm(h_out) * p["pre_weight"]
    ((h_out * dh_out.double()).sum() + (n1 * dn1.double()).sum()).backward()
    return h_out.detach(), n1.detach(), {k: v.grad for k, v in p.items()}, x.grad


@pytest.mark.parametrize("save", [False, True])
def test_a_blocks_training_step(save):
    p, x, dh_out, dn1 = block_inputs(7)
    P = {k: v.cuda() for k, v in p.items()}
    s = block_forward(P, x.cuda(), save)
    grads, dx = block_backward(P, x.cuda(), s, dh_out.cuda(), dn1.cuda())
    h_want, n_want, want, dx_want = block_exact(p, x, dh_out, dn1)
    # five results follow one another, of products over C and 4 C channels, T tokens and D features
    depth = 2 * (5 * C + T + D)
    close(s["h_out"], f64(h_want), depth, "h_out")
    close(s["n1"], f64(n_want), depth, "n1")
    if not save:
        close(dx, f64(dx_want), 2 * depth, "dx")
        for k in p:
            if k != "log_decay":
                close(grads[k], f64(want[k]), 2 * depth + B * T, k)
            else:   # a sum of terms of both signs, whose size is that of its parts by token
                assert torch.allclose(grads[k].cpu().double(), want[k], rtol=1e-3, atol=1e-3 * float(want[k].abs().max()))
        return
    # y comes back from 8 bits: off by at most half a step, 2^-7 of the largest of 32 channels,
    # which enters the gradients of the block's output once and is at most 4 of their size
    for got, w in ((dx, dx_want), *((grads[k], want[k]) for k in p)):
        assert float((got.cpu().double() - w).norm()) <= 4 * 2.0 ** -7 * float(w.norm())


def test_a_prompt_and_tokens_behind_it():
    """The block's forward over whole sequences, and over a prompt and then single tokens."""
    p, x, _, _ = block_inputs(9)
    P, x = {k: v.cuda() for k, v in p.items()}, x.cuda()
    whole = block_forward(P, x)
    cut = 140
    s = block_forward(P, x[:, :cut].contiguous())
    _, S = fb.falcon_linear_fwd(s["q"], s["k"], s["v"], P["log_decay"], qk_layout="rows", v_layout="rows", o_layout="rows")
    for t in range(cut, T):
        xt = x[:, t:t + 1].contiguous()
        _, n0, _ = fb.falcon_residual_fwd(xt, post_norm=False, pre_weight=P["pre_weight"], eps=1e-5)
        wide = n0[:, 0] @ P["w_in"]
        q, k, v = (wide[:, i * C:(i + 1) * C].unflatten(1, (H, D)) for i in range(3))
        o = fb.falcon_linear_step(q, k, v, P["log_decay"], S, scale=D ** -0.5).flatten(1)[:, None]
        z, _, _ = fb.falcon_residual_fwd(o, gate=wide[:, None, 3 * C:], post_weight=P["head_weight"], eps=1e-5, **NORM)
        h_out, n1, _ = fb.falcon_residual_fwd(z @ P["w_out"], xt, post_weight=P["post_weight"], alpha=P["alpha"], pre_weight=P["pre_weight"],
                                              eps=1e-5)
        close(h_out[:, 0], f64(whole["h_out"][:, t]), 2 * (5 * C + T + D), f"h_out of token {t}")
        close(n1[:, 0], f64(whole["n1"][:, t]), 2 * (5 * C + T + D), f"n1 of token {t}")


# ---- graphs and streams ------------------------------------------------------------------------

def linear_set(seed, io, dk=64, dv=128, T=333):
    n = draws(seed)
    main = [n(2, 3, T, d, dtype=io).cuda() for d in (dk, dk, dv, dv)]
    return main, -torch.rand(3).cuda() - 0.01, n(2, 3, dk, dv).cuda(), torch.tensor([T, T - 70], dtype=torch.int32, device="cuda")


def filler(sets, into):
    def fill(k):
        for t, v in zip(into, sets[k]):
            t.copy_(v)
    return fill


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_linear_attention_in_a_graph(io):
    flat = lambda s: [*s[0], *s[1:]]  # noqa: E731
    sets = [flat(linear_set(s, IO[io])) for s in (1, 2)]
    q, k, v, dO, g, S, ends = into = [t.clone() for t in sets[0]]
    replayed(lambda: fb.falcon_linear_fwd(q, k, v, g, S0=S, lengths=ends), filler(sets, into))

    def backward():
        out = fb.falcon_linear_bwd(q, k, v, g, dO, S0=S, dS_T=S, lengths=ends, learned_decay=True)
        return [out[n] for n in ("dq", "dk", "dv", "dS0", "dlog_decay")]

    replayed(backward, filler(sets, into))


def test_single_tokens_in_a_graph():
    """The state moves on with every replay."""
    n = draws(3)
    q, k, v, S = n(4, 3, 64).cuda(), n(4, 3, 64).cuda(), n(4, 3, 32).cuda(), n(4, 3, 64, 32).cuda()
    g = -torch.rand(3).cuda()
    want_S, outs = S.clone(), []
    for _ in range(4):
        outs.append(fb.falcon_linear_step(q, k, v, g, want_S))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fb.falcon_linear_step(q, k, v, g, S.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = fb.falcon_linear_step(q, k, v, g, S)
    for want in outs:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        fb.falcon_linear_step(q, k, v, g, S.clone())
    assert torch.equal(S, want_S)


@pytest.mark.parametrize("width,groups", [(96, 3), (77, 1), (2304, 1)])
def test_a_saved_update_in_a_graph(width, groups):
    n = draws(4)
    sets = [[n(3, 50, width).cuda() for _ in range(5)] for _ in range(2)]
    y, h, gate, dh, dn = into = [t.clone() for t in sets[0]]
    w = n(width).cuda()
    a = dict(groups=groups, post_weight=w, alpha=w, pre_weight=w)

    def run():
        h_out, normed, kept = fb.falcon_residual_fwd(y, h, gate=gate, save=True, **a)
        g = fb.falcon_residual_bwd(None, h_out, dh, dn, saved=kept, **a)
        return [h_out, normed, *kept, *g.values()]

    replayed(run, filler(sets, into))


def test_two_graphs_share_a_workspace():
    """One after the other; each leaves nothing in it that the other needs."""
    sets = [linear_set(s, torch.bfloat16) for s in (5, 6)]
    p = fb.FalconLinearProblem(2, 3, 333, 64, 128, 1, 1, 1, 1, 1.0, 192, 192, 384)
    ws = torch.empty(fb.falcon_linear_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    call = lambda s: fb.falcon_linear_bwd(*s[0][:3], s[1], s[0][3], S0=s[2], lengths=s[3], learned_decay=True, workspace=ws)  # noqa: E731
    want = [call(s) for s in sets]
    want = [{k: v.clone() for k, v in g.items()} for g in want]
    graphs, got = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(call(s))
    for _ in range(3):
        for i in (0, 1):
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(got[i][k], want[i][k]) for k in want[i])


def test_other_streams_and_two_calls_at_once():
    (q, k, v, dO), g, S, ends = linear_set(8, torch.bfloat16)
    y, h = draws(9)(4, 200, 768).cuda(), draws(10)(4, 200, 768).cuda()
    want = fb.falcon_linear_bwd(q, k, v, g, dO, S0=S)
    want_r = fb.falcon_residual_bwd(y, h, h, y, groups=12)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = fb.falcon_linear_bwd(q, k, v, g, dO, S0=S, stream=a)
        with torch.cuda.stream(b):
            got2 = fb.falcon_linear_bwd(q, k, v, g, dO, S0=S)
            got_r = fb.falcon_residual_bwd(y, h, h, y, groups=12)
        torch.cuda.synchronize()
        for x, w in ((got, want), (got2, want), (got_r, want_r)):
            assert all(torch.equal(x[n], w[n]) for n in w if w[n] is not None)


# ---- offsets past 32 bits -------------------------------------------------------------------------

def test_rows_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    width = 8192
    tokens = (1 << 19) + 77                      # past 2^32 elements
    y = torch.empty(1, tokens, width, dtype=torch.bfloat16, device="cuda").normal_()
    h = torch.empty(1, tokens, width, dtype=torch.bfloat16, device="cuda").normal_()
    h_out, n, kept = fb.falcon_residual_fwd(y, h, gate=y, save=True, h_out=h)
    cut = (0, (1 << 18) + 1, tokens - 3)
    parts = [slice(at, at + 3) for at in cut]
    x = [y[:, s].contiguous() for s in parts]
    del h
    g = fb.falcon_residual_bwd(None, h_out, None, y, saved=kept, grads={"dgate": torch.empty(y.shape, device="cuda")}, added=False)
    for s, part in zip(parts, x):
        aligned = [t[:, s].contiguous() for t in (h_out, *kept)]
        want = fb.falcon_residual_bwd(None, aligned[0], None, part, saved=fb.FalconSaved(*aligned[1:]), added=False)
        assert torch.equal(g["dy"][:, s], want["dy"]) and torch.equal(g["dgate"][:, s], want["dgate"])
        close(n[:, s], f64(aligned[0].float() / (aligned[0].float().square().mean(-1, keepdim=True) + 1e-6).sqrt()), 1 << 16, "n")
    del y, h_out, n, kept, g
    torch.cuda.empty_cache()


@pytest.mark.parametrize("layout", ["heads", "rows"])
def test_prompts_past_32_bits(layout):
    """A state forgets within 64 tokens what lies 128 back (to 2^-92 of it): the last tokens
    by themselves, from some way before."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    T, H, d = (1 << 25) + 70, 2, 64              # past 2^32 elements of a tensor
    shape = (1, H, T, d) if layout == "heads" else (1, T, H * d)
    q, k, v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(3))
    g = torch.full((H,), -0.5, device="cuda")
    a = dict(scale=0.1, qk_layout=layout, v_layout=layout, o_layout=layout)
    o, S_T = fb.falcon_linear_fwd(q, k, v, g, **a)
    last = (lambda t, n: t[:, :, -n:]) if layout == "heads" else (lambda t, n: t[:, -n:])
    short = [last(t, 400).contiguous() for t in (q, k, v)]
    o2, S2 = fb.falcon_linear_fwd(*short, g, **a)
    close(last(o, 200), f64(last(o2, 200).float()), 1 << 16, "o")
    close(S_T, f64(S2), 400, "S_T")
    del q, k, v, o
    torch.cuda.empty_cache()
