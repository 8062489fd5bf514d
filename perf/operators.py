"""What the block around a fast-weight recurrence runs, measured: the short
causal convolution of the projections, the group norm with an activation that
makes features per head (and norms the heads' outputs), and the selective
state space scan, each for whole prompts, for training and (convolution and
scan) for single tokens.

``run`` is one pass, in its plain form of elementary torch operations in 32
bits, or, where ``own`` is set, by the calls of ``delta_rule_recurrence_amd``.
"""

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------

def conv(form, B, T, C, W, dtype, act="silu", carry=False, ragged=False):
    return {"op": "conv", "form": form, "B": B, "T": T, "C": C, "W": W, "dtype": dtype, "act": act,
            "carry": carry, "ragged": ragged}


def norm(form, B, T, G, d, dtype, center=False, act="none", affine=True, x="rows", y="rows"):
    return {"op": "norm", "form": form, "B": B, "T": T, "G": G, "d": d, "dtype": dtype, "center": center,
            "act": act, "affine": affine, "x_layout": x, "y_layout": y}


def scan(form, B, T, D, N, G, dtype, gate=True, carry=False, ragged=False):
    return {"op": "scan", "form": form, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype, "gate": gate,
            "carry": carry, "ragged": ragged}


def listed():
    cases = {
        # the q, k and v projections of 12 heads of 64, side by side, at the training shape 8 x 2048
        "conv_prompt": conv("prompt", 8, 2048, 3 * 12 * 64, 4, "bf16"),
        # prompts of unequal lengths that go on from carried rows; odd sizes, float32
        "conv_ragged": conv("prompt", 5, 777, 1001, 3, "f32", carry=True, ragged=True),
        # its gradients at the training shape
        "conv_train": conv("train", 8, 2048, 3 * 12 * 64, 4, "bf16"),
        # one token of 512 sequences, 12 heads of 128: q, k and v
        "conv_step": conv("step", 512, 1, 3 * 12 * 128, 4, "bf16"),
        # phi(k) of 12 heads of 64: rows in, heads out, at the training shape
        "norm_features": norm("prompt", 8, 2048, 12, 64, "bf16", act="elu1", y="heads"),
        # the heads' outputs of one token of four sequences: the smallest call
        "norm_token": norm("prompt", 4, 1, 12, 128, "bf16", center=True, act="silu", x="heads"),
        # the gradients of the features at the training shape
        "norm_train": norm("train", 8, 2048, 12, 64, "bf16", act="elu1", y="heads"),
        # a batch of prompts
        "scan_prompt": scan("prompt", 8, 2048, 1536, 16, 1, "bf16"),
        # one long prompt
        "scan_long": scan("prompt", 1, 16384, 768, 16, 1, "bf16"),
        # prompts of unequal lengths from carried states; two groups, wide states, odd sizes, float32
        "scan_ragged": scan("prompt", 3, 601, 250, 64, 2, "f32", gate=False, carry=True, ragged=True),
        # the gradients at the training shape
        "scan_train": scan("train", 8, 2048, 768, 16, 1, "bf16"),
        # one token of 512 sequences
        "scan_step": scan("step", 512, 1, 1536, 16, 1, "bf16"),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("conv", "norm", "scan"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    carry, ragged = rng.random() < 0.4, rng.random() < 0.4
    if op == "norm":
        form = rng.choice(("prompt", "train"))
        G, d = spread(rng, 1, 32), rng.choice((16, 32, 64, 80, 128, spread(rng, 3, 1024)))
        rows = spread(rng, 1, 8 * 2048 * 768 // (G * d))
        B = min(rows, spread(rng, 1, 32))
        return norm(form, B, rows // B, G, d, dtype, rng.random() < 0.5, rng.choice(("none", "silu", "elu1")),
                    rng.random() < 0.8, rng.choice(("rows", "heads")), rng.choice(("rows", "heads")))
    form = rng.choice(("prompt", "train", "step"))
    if op == "conv":
        C, W = rng.choice((spread(rng, 16, 4608), 64 * spread(rng, 1, 72))), rng.choice((2, 3, 4))
        act = rng.choice(("silu", "silu", "none"))
        if form == "step":
            return conv(form, spread(rng, 1, 1024), 1, C, W, dtype, act)
        T = spread(rng, 1, 16384)
        B = spread(rng, 1, min(64, max(1, 8 * 2048 * 1536 // (T * C))))
        return conv(form, B, min(T, max(1, 8 * 2048 * 1536 // (B * C))), C, W, dtype, act, carry, ragged)
    N, G = rng.choice((8, 16, 16, 32, 64)), rng.choice((1, 1, 2, 4))
    D = G * rng.choice((spread(rng, 4, 512), 64 * spread(rng, 1, 8)))
    gate = rng.random() < 0.7
    if form == "step":
        return scan(form, spread(rng, 1, min(1024, max(1, 512 * 1536 * 16 // (D * N)))), 1, D, N, G, dtype, gate)
    most = (8 * 2048 * 768 * 16 if form == "train" else 8 * 2048 * 1536 * 16) // (D * N)
    T = spread(rng, 1, min(16384, most))
    return scan(form, spread(rng, 1, min(64, max(1, most // T))), T, D, N, G, dtype, gate, carry, ragged)


# ---- inputs -------------------------------------------------------------------

def heads_or_rows(case, which):
    B, T, G, d = case["B"], case["T"], case["G"], case["d"]
    return (B, T, G * d) if case[which] == "rows" else (B, G, T, d)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    io = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=io):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    f32 = torch.float32
    s = dict(case)
    B, T = case["B"], case["T"]
    if case.get("ragged"):
        # prompts of one token up to the whole row
        s["lengths"] = torch.randint(1, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        s["x"] = normal(B, C) if case["form"] == "step" else normal(B, T, C)
        s["weight"], s["bias"] = normal(C, W, scale=W ** -0.5, dtype=f32), normal(C, scale=0.1, dtype=f32)
        if case["carry"] or case["form"] == "step":
            s["state"] = normal(B, W - 1, C)
        if case["form"] == "train":
            # as the backward of what reads the features gives it: 32 bits
            s["dy"] = normal(B, T, C, dtype=f32)
            if case["carry"]:
                s["dstate_out"] = normal(B, W - 1, C, dtype=f32)
    elif case["op"] == "norm":
        G, d = case["G"], case["d"]
        s["x"] = normal(*heads_or_rows(case, "x_layout"))
        if case["affine"]:
            s["weight"], s["bias"] = 1 + normal(G * d, scale=0.1, dtype=f32), normal(G * d, scale=0.1, dtype=f32)
        s["scale"] = d ** -0.5
        if case["form"] == "train":
            s["dy"] = normal(*heads_or_rows(case, "y_layout"), dtype=f32)
    else:
        D, N, G = case["D"], case["N"], case["G"]
        t = () if case["form"] == "step" else (T,)
        s["x"], s["dt"] = normal(B, *t, D), normal(B, *t, D)
        # B and C are columns of one projection
        s["bc"] = normal(B, *t, 2, G, N)
        # decays of 1 to N a unit of time, steps of about 0.01 to 0.1
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=f32).repeat(D, 1) * (1 + normal(D, 1, scale=0.1, dtype=f32)).abs()
        s["D_skip"], s["dt_bias"] = 1 + normal(D, scale=0.1, dtype=f32), -3.5 + normal(D, scale=0.5, dtype=f32)
        if case["gate"]:
            s["z"] = normal(B, *t, D)
        if case["carry"] or case["form"] == "step":
            s["S0"] = normal(B, D, N, dtype=f32)
        if case["form"] == "train":
            s["dy"] = normal(B, T, D)
            if case["carry"]:
                s["dS_T"] = normal(B, D, N, dtype=f32)
    return s


# ---- one pass -------------------------------------------------------------------

def run(s):
    if own:
        return given(ours(s))
    return given({"conv": plain_conv, "norm": plain_norm, "scan": plain_scan}[s["op"]](s))


def given(out):
    """The outputs that the call has: by name and without those it does not have."""
    if torch.is_tensor(out):
        return out
    if isinstance(out, dict):
        return {k: out[k] for k in sorted(out) if out[k] is not None}
    return [t for t in out if t is not None]


def ours(s):
    from delta_rule_recurrence_amd import falcon as fb

    if s["op"] == "conv":
        a = dict(bias=s["bias"], activation=s["act"])
        if s["form"] == "step":
            return fb.falcon_conv_step(s["x"], s["weight"], s["state"], **a), s["state"]
        a.update(state=s.get("state"), lengths=s.get("lengths"))
        if s["form"] == "prompt":
            return fb.falcon_conv_fwd(s["x"], s["weight"], return_state=s["carry"], **a)
        return fb.falcon_conv_bwd(s["x"], s["weight"], s["dy"], dstate_out=s.get("dstate_out"), **a)
    if s["op"] == "norm":
        a = dict(weight=s.get("weight"), bias=s.get("bias"), center=s["center"], activation=s["act"],
                 eps=EPS, scale=s["scale"], x_layout=s["x_layout"], y_layout=s["y_layout"])
        if s["form"] == "prompt":
            return fb.falcon_norm_fwd(s["x"], s["G"], **a)
        return fb.falcon_norm_bwd(s["x"], s["G"], s["dy"], **a)
    b, c = s["bc"].unbind(-3)
    a = dict(D=s["D_skip"], dt_bias=s["dt_bias"], softplus=True, z=s.get("z"))
    if s["form"] == "step":
        return fb.falcon_scan_step(s["x"], s["dt"], s["A"], b, c, s["S0"], **a), s["S0"]
    a.update(S0=s.get("S0"), lengths=s.get("lengths"))
    if s["form"] == "prompt":
        return fb.falcon_scan_fwd(s["x"], s["dt"], s["A"], b, c, **a)
    return fb.falcon_scan_bwd(s["x"], s["dt"], s["A"], b, c, s["dy"], dS_T=s.get("dS_T"), **a)


EPS = 1e-6


def sigmoid(p):
    return 1 / (1 + torch.exp(-p))


def activated(p, act):
    if act == "silu":
        return p * sigmoid(p)
    if act == "elu1":
        return torch.where(p > 0, p + 1, torch.exp(p.clamp(max=0)))
    return p


def slope(p, act):
    """The activation's derivative."""
    if act == "silu":
        q = sigmoid(p)
        return q * (1 + p * (1 - q))
    if act == "elu1":
        return torch.where(p > 0, torch.ones_like(p), torch.exp(p.clamp(max=0)))
    return torch.ones_like(p)


def live(s):
    """[B, T]: the tokens before each sequence's end, or None where all are."""
    if "lengths" not in s:
        return None
    return torch.arange(s["T"], device="cuda")[None] < s["lengths"][:, None]


# y_t = act(bias + sum_j weight_j x_(t - (W - 1) + j)), a channel at a time; the
# rows before the first token are the carried state's, or zero.

def plain_conv(s):
    io, W = s["x"].dtype, s["W"]
    x = s["x"].float()
    if s["form"] == "step":
        rows = torch.cat((s["state"].float(), x[:, None]), 1)
        y = activated((rows * s["weight"].t()).sum(1) + s["bias"], s["act"]).to(io)
        s["state"].copy_(rows[:, 1:])
        return y, s["state"]
    B, T, C = x.shape
    first = s["state"].float() if "state" in s else x.new_zeros(B, W - 1, C)
    rows = torch.cat((first, x), 1)
    seen = rows.unfold(1, W, 1)                       # [B, T, C, W]
    p = (seen * s["weight"]).sum(-1) + s["bias"]
    m = live(s)
    # the last W - 1 rows before each sequence's end
    ends = s["lengths"].long() if "lengths" in s else torch.full((B,), T, device="cuda")
    last = (ends[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(B, W - 1, C)
    if s["form"] == "prompt":
        y = activated(p, s["act"])
        y = y if m is None else y * m[..., None]
        return y.to(io), rows.gather(1, last).to(io) if s["carry"] else None
    dp = s["dy"] * slope(p, s["act"])
    dp = dp if m is None else dp * m[..., None]
    pad = dp.new_zeros(B, W - 1, C)
    drows = (torch.cat((pad, dp, pad), 1).unfold(1, W, 1) * s["weight"].flip(1)).sum(-1)
    if "dstate_out" in s:
        drows.scatter_add_(1, last, s["dstate_out"])
    return {"dx": drows[:, W - 1:].contiguous(), "dstate": drows[:, :W - 1].contiguous() if "state" in s else None,
            "dweight": (dp[..., None] * seen).sum((0, 1), dtype=torch.float64).float(),
            "dbias": dp.sum((0, 1), dtype=torch.float64).float()}


# y = scale act(weight xhat + bias) over each token's group of d channels, with
# xhat = (x - mean) / sqrt(mean((x - mean)^2) + eps), the mean only if centred.

def tokens_first(t, s, which):
    """[B, T, G, d] of either layout, in 32 bits."""
    if s[which] == "heads":
        return t.float().transpose(1, 2)
    return t.float().unflatten(-1, (s["G"], s["d"]))


def in_layout(t, s, which):
    return (t.transpose(1, 2) if s[which] == "heads" else t.flatten(2)).contiguous()


def plain_norm(s):
    G, d = s["G"], s["d"]
    x = tokens_first(s["x"], s, "x_layout")
    if s["center"]:
        x = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat = x * r
    w = s["weight"].view(G, d) if s["affine"] else x.new_ones(G, d)
    p = xhat * w + (s["bias"].view(G, d) if s["affine"] else 0)
    if s["form"] == "prompt":
        return in_layout((activated(p, s["act"]) * s["scale"]).to(s["x"].dtype), s, "y_layout")
    dp = tokens_first(s["dy"], s, "y_layout") * slope(p, s["act"]) * s["scale"]
    dh = dp * w
    dx = dh - xhat * (dh * xhat).mean(-1, keepdim=True)
    if s["center"]:
        dx = dx - dh.mean(-1, keepdim=True)
    out = {"dx": in_layout(dx * r, s, "x_layout"), "dweight": None, "dbias": None}
    if s["affine"]:
        out["dweight"] = (dp * xhat).sum((0, 1), dtype=torch.float64).float().flatten()
        out["dbias"] = dp.sum((0, 1), dtype=torch.float64).float().flatten()
    return out


# S_t = exp(delta_t A) S_(t-1) + delta_t x_t B_t, y_t = (<C_t, S_t> + D x_t) silu(z_t),
# with delta_t = softplus(dt_t + dt_bias), a state of N a channel.

def softplus(p):
    return p.clamp(min=0) + torch.log1p(torch.exp(-p.abs()))


def scanned(a, b):
    """S_t = a_t S_(t-1) + b_t over axis 1 from S = 0, by doubling spans."""
    a, b, span = a.clone(), b.clone(), 1
    while span < a.shape[1]:
        b[:, span:] += a[:, span:] * b[:, :-span].clone()
        a[:, span:] *= a[:, :-span].clone()
        span *= 2
    return b


def plain_scan(s):
    io, G = s["x"].dtype, s["G"]
    each = s["D"] // G
    x, dt, bc = s["x"].float(), s["dt"].float(), s["bc"].float()
    z = s["z"].float() if s["gate"] else None
    step = s["form"] == "step"
    if step:
        x, dt, bc, z = x[:, None], dt[:, None], bc[:, None], z[:, None] if s["gate"] else None
    b, c = (t.repeat_interleave(each, 2) for t in bc.unbind(2))  # [B, T, D, N]
    delta = softplus(dt + s["dt_bias"])
    m = live(s)
    # behind its end a sequence keeps its state
    held = delta if m is None else delta * m[..., None]
    a = torch.exp(held[..., None] * s["A"])
    u = (held * x)[..., None] * b
    S0 = s["S0"] if "S0" in s else torch.zeros_like(u[:, 0])
    u[:, 0] += a[:, 0] * S0
    S = scanned(a, u)
    read = (c * S).sum(-1) + s["D_skip"] * x
    if s["form"] != "train":
        y = read * activated(z, "silu") if s["gate"] else read
        y = (y if m is None else y * m[..., None]).to(io)
        if step:
            s["S0"].copy_(S[:, -1])
            return y[:, 0], s["S0"]
        return y, S[:, -1].contiguous()
    dy = s["dy"].float()
    dy = dy if m is None else dy * m[..., None]
    dread = dy * activated(z, "silu") if s["gate"] else dy
    q = dread[..., None] * c
    if "dS_T" in s:
        q[:, -1] += s["dS_T"]
    after = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    dS = scanned(after.flip(1), q.flip(1)).flip(1)
    del after, q
    decayed = dS * a * torch.cat((S0[:, None], S[:, :-1]), 1)
    if m is not None:
        decayed = decayed * m[..., None, None]
    du = (dS * b).sum(-1)
    du = du if m is None else du * m[..., None]
    ddelta = (decayed * s["A"]).sum(-1) + du * x
    ddt = ddelta * sigmoid(dt + s["dt_bias"])
    group = lambda t: t.unflatten(2, (G, each)).sum(3)  # noqa: E731  over the channels of a group
    return {"dx": du * delta + s["D_skip"] * dread, "ddt": ddt, "dA": (decayed * delta[..., None]).sum((0, 1), dtype=torch.float64).float(),
            "dB": group(dS * (held * x)[..., None]), "dC": group(dread[..., None] * S),
            "dD": (dread * x).sum((0, 1), dtype=torch.float64).float(),
            "ddt_bias": ddt.sum((0, 1), dtype=torch.float64).float(),
            "dz": dy * read * slope(z, "silu") if s["gate"] else None,
            "dS0": a[:, 0] * dS[:, 0] if "S0" in s else None}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    B, T, es = case["B"], case["T"], 4 if case["dtype"] == "f32" else 2
    train = case["form"] == "train"
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        n, rows = B * T * C, B * (W - 1) * C * es * (2 if case["form"] == "step" else 2 * case["carry"])
        if train:
            return {"bytes": n * (es + 8) + rows * 3 + C * (W + 1) * 8, "flops": n * (6 * W + 10)}
        return {"bytes": 2 * n * es + rows + C * (W + 1) * 4, "flops": n * (2 * W + 5)}
    if case["op"] == "norm":
        C = case["G"] * case["d"]
        n = B * T * C
        par = C * 8 if case["affine"] else 0
        return {"bytes": n * (es + 8) + 2 * par, "flops": 20 * n} if train else {"bytes": 2 * n * es + par, "flops": 8 * n}
    D, N, G = case["D"], case["N"], case["G"]
    n, shared, states = B * T * D, B * T * 2 * G * N, B * D * N * 4
    par, gate = D * (N + 2) * 4, int(case["gate"])
    if train:
        return {"bytes": n * (es * (3 + gate) + 4 * (2 + gate)) + shared * (es + 4) + states * 3 * case["carry"] + 2 * par,
                "flops": n * N * 20}
    return {"bytes": n * es * (3 + gate) + shared * es + states * (2 if "step" == case["form"] or case["carry"] else 1) + par,
            "flops": n * N * 6}


# ---- the definitions in 64 bits, a token and a tap at a time --------------------------

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    out = {"conv": exact_conv, "norm": exact_norm, "scan": exact_scan}[case["op"]](s)
    return given(out)


def exact_act(p, act):
    """The activation and its derivative."""
    if act == "silu":
        q = torch.sigmoid(p)
        return p * q, q + p * q * (1 - q)
    if act == "elu1":
        return torch.where(p > 0, p + 1, p.exp()), torch.where(p > 0, 1.0, p.exp())
    return p, torch.ones_like(p)


def exact_ends(s):
    return s["lengths"].tolist() if "lengths" in s else [s["T"]] * s["B"]


def exact_conv(s):
    B, T, C, W = s["B"], s["T"], s["C"], s["W"]
    x = s["x"].reshape(B, T, C)
    before = s["state"] if "state" in s else x.new_zeros(B, W - 1, C)
    w, parts = s["weight"], []
    for i, n in enumerate(exact_ends(s)):
        r = torch.cat((before[i], x[i, :n]))
        p = s["bias"] + sum(r[j:j + n] * w[:, j] for j in range(W))
        f, df = exact_act(p, s["act"])
        behind = x.new_zeros(T - n, C)
        if s["form"] != "train":
            parts.append((torch.cat((f, behind)), r[n:]))
            continue
        dp, dr = s["dy"][i, :n] * df, torch.zeros_like(r)
        for j in range(W):
            dr[j:j + n] += dp * w[:, j]
        if "dstate_out" in s:
            dr[n:] += s["dstate_out"][i]
        dw = torch.stack([(dp * r[j:j + n]).sum(0) for j in range(W)], 1)
        parts.append((torch.cat((dr[W - 1:], behind)), dr[:W - 1], dw, dp.sum(0)))
    a = [torch.stack(v) for v in zip(*parts)]
    if s["form"] == "train":
        return {"dx": a[0], "dstate": a[1] if "state" in s else None, "dweight": a[2].sum(0), "dbias": a[3].sum(0)}
    if s["form"] == "step":
        return a[0][:, 0], a[1]
    return a if s["carry"] else a[:1]


def exact_norm(s):
    B, T, G, d = s["B"], s["T"], s["G"], s["d"]
    rows = lambda t, which: t.reshape(B, T, G, d) if s[which] == "rows" else t.permute(0, 2, 1, 3)  # noqa: E731
    laid = lambda t, which: t.reshape(B, T, G * d) if s[which] == "rows" else t.permute(0, 2, 1, 3).contiguous()  # noqa: E731
    x = rows(s["x"], "x_layout")
    mean = x.mean(-1, keepdim=True) if s["center"] else 0.0
    dev = ((x - mean).square().mean(-1, keepdim=True) + EPS).sqrt()
    h = (x - mean) / dev
    w, b = (s["weight"].reshape(G, d), s["bias"].reshape(G, d)) if s["affine"] else (1.0, 0.0)
    f, df = exact_act(h * w + b, s["act"])
    if s["form"] == "prompt":
        return laid(f * s["scale"], "y_layout")
    dp = rows(s["dy"], "y_layout") * df * s["scale"]
    dh = dp * w
    # (I - P) / dev, with P the projection on h and, if centred, on the constant
    dx = (dh - h * (dh * h).sum(-1, keepdim=True) / d - (dh.mean(-1, keepdim=True) if s["center"] else 0.0)) / dev
    affine = {"dweight": (dp * h).sum((0, 1)).reshape(-1), "dbias": dp.sum((0, 1)).reshape(-1)} if s["affine"] else {}
    return {"dx": laid(dx, "x_layout"), **affine}


def exact_scan(s):
    B, T, D, N, G = (s[k] for k in ("B", "T", "D", "N", "G"))
    per = D // G
    x, dt, bc = s["x"].reshape(B, T, D), s["dt"].reshape(B, T, D), s["bc"].reshape(B, T, 2, G, N)
    z = s["z"].reshape(B, T, D) if s["gate"] else None
    wide = lambda t: t[:, :, None].expand(B, G, per, N).reshape(B, D, N)  # noqa: E731
    ends = torch.tensor(exact_ends(s), device="cuda")
    raw = dt + s["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    S = s["S0"].clone() if "S0" in s else x.new_zeros(B, D, N)
    kept, reads = [], []
    for t in range(T):
        on = (t < ends)[:, None, None]
        if s["form"] == "train":
            kept.append(S)
        new = (delta[:, t, :, None] * s["A"]).exp() * S + (delta[:, t] * x[:, t])[..., None] * wide(bc[:, t, 0])
        S = torch.where(on, new, S)
        reads.append((wide(bc[:, t, 1]) * S).sum(-1) + s["D_skip"] * x[:, t])
    read = torch.stack(reads, 1)
    on = (torch.arange(T, device="cuda")[None] < ends[:, None])[..., None]
    f, df = exact_act(z, "silu") if s["gate"] else (torch.ones_like(read), None)
    if s["form"] != "train":
        y = torch.where(on, read * f, 0.0)
        return (y[:, 0] if s["form"] == "step" else y), S
    dy = torch.where(on, s["dy"], 0.0)
    dread = dy * f
    dS = s["dS_T"].clone() if "dS_T" in s else torch.zeros_like(S)
    dA, last = torch.zeros_like(s["A"]), S
    ddelta, dx, dB, dC = torch.zeros_like(x), torch.zeros_like(x), [], []
    over = lambda t: t.reshape(B, G, per, N).sum(2)  # noqa: E731
    for t in range(T - 1, -1, -1):
        live_t, prev = (t < ends)[:, None, None], kept.pop()
        dS = dS + dread[:, t, :, None] * wide(bc[:, t, 1])
        dC.append(over(dread[:, t, :, None] * last))
        db = torch.where(live_t, dS * (delta[:, t] * x[:, t])[..., None], 0.0)
        dB.append(over(db))
        du = torch.where(live_t, dS * wide(bc[:, t, 0]), 0.0).sum(-1)
        decay = torch.where(live_t, (delta[:, t, :, None] * s["A"]).exp(), 1.0)
        turn = torch.where(live_t, dS * decay * prev, 0.0)
        ddelta[:, t] = (turn * s["A"]).sum(-1) + du * x[:, t]
        dA += (turn * delta[:, t, :, None]).sum(0)
        dx[:, t] = du * delta[:, t] + s["D_skip"] * dread[:, t]
        dS, last = dS * decay, prev
    ddt = ddelta * torch.sigmoid(raw)
    return {"dx": dx, "ddt": ddt, "dA": dA, "dB": torch.stack(dB[::-1], 1), "dC": torch.stack(dC[::-1], 1),
            "dD": (dread * x).sum((0, 1)), "ddt_bias": ddt.sum((0, 1)),
            "dz": dy * read * df if s["gate"] else None, "dS0": dS if "S0" in s else None}
