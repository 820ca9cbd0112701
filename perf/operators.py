"""The state-space block's operators, as they are measured: the short causal convolution, the
selective scan and the norms around a block, in their plain form (elementary torch operations in
32 bits) and, where `own` is true, through this package's entry points.

Notation: B sequences, T tokens, D channels (or H heads of d channels), N states per channel, G
groups of channels that share B and C, K taps.  `lens` are the tokens of each sequence of a padded
batch; outputs behind them are zero.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # One token for each of 64 sequences: the convolution of the queries of 16 heads of 128,
        # the state moved on in place (the smallest call: latency).
        dict(name="conv_step", op="conv", B=64, H=16, T=1, d=128, K=4, dtype="bf16", fresh=False,
             ragged=False),
        # A prompt batch of the mid-size prefill, head layout [B][H][T][d].
        dict(name="conv_mid_prefill", op="conv", B=2, H=4, T=4096, d=128, K=4, dtype="bf16",
             fresh=True, ragged=False),
        # Training on the headline prefill's shape: heads of 64.
        dict(name="conv_headline_backward", op="conv_bwd", B=8, H=16, T=8192, d=64, K=4,
             dtype="bf16", ragged=False),
        # Decode of 64 sequences at the mid workload's layer width: state read and written.
        dict(name="scan_step", op="scan", B=64, T=1, D=4096, N=16, G=1, dtype="bf16", fresh=False,
             ragged=False),
        # A padded batch of unequal prompts that go on from a state, odd widths.
        dict(name="scan_ragged_prompts", op="scan", B=4, T=777, D=1000, N=16, G=2, dtype="bf16",
             fresh=False, ragged=True),
        # Prefill at the mid workload's batch, length and layer width (the largest case).
        dict(name="scan_mid_prefill", op="scan", B=2, T=4096, D=4096, N=16, G=1, dtype="bf16",
             fresh=True, ragged=False),
        # One long sequence of few channels in fp32: the work has to be split over time.
        dict(name="scan_long_f32", op="scan", B=1, T=16384, D=512, N=16, G=1, dtype="f32",
             fresh=True, ragged=False),
        # A training step's backward pass.
        dict(name="scan_backward", op="scan_bwd", B=2, T=2048, D=2048, N=16, G=1, dtype="bf16",
             ragged=False),
        # A small fp32 training step, odd sizes, few states, padded.
        dict(name="scan_backward_odd_f32", op="scan_bwd", B=3, T=301, D=200, N=8, G=1, dtype="f32",
             ragged=True),
        # The norms of one decode step of 64 sequences.
        dict(name="norm_step", op="norm", rows=64, D=4096, rdt="bf16", fdt="f32", xdt="bf16"),
        # The norms of the mid prefill (8192 rows); the block's output comes in fp32.
        dict(name="norm_mid_prefill", op="norm", rows=8192, D=4096, rdt="f32", fdt="f32",
             xdt="bf16"),
        # Their backward pass, an odd number of rows.
        dict(name="norm_backward", op="norm_bwd", rows=4099, D=4096, rdt="bf16", fdt="bf16",
             xdt="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "scan", "scan", "scan_bwd", "scan_bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "conv_bwd"):
        d = rng.choice([16, 30, 64, 72, 100, 128, 192, 256])
        H = rng.choice([1, 2, 3, 4, 8, 16])
        B = rng.choice([1, 2, 3, 8, 64])
        T = min(_log_int(rng, 1, 16384), max(1, (1 << 25) // (B * H * d)))
        c = dict(op=op, B=B, H=H, T=T, d=d, K=rng.choice([2, 3, 4, 4, 5, 7]), dtype=dtype,
                 ragged=rng.random() < 0.4)
        if op == "conv":
            c["fresh"] = rng.random() < 0.5
        return c
    if op in ("scan", "scan_bwd"):
        G = rng.choice([1, 1, 2, 4])
        D = G * _log_int(rng, 40, 4096 // G)
        N = rng.choice([4, 8, 11, 16, 16, 16, 32, 64])
        B = rng.choice([1, 2, 3, 4, 16])
        cap = (1 << 28) if op == "scan" else (1 << 26)
        T = min(_log_int(rng, 1, 16384), max(1, cap // (B * D * N)))
        c = dict(op=op, B=B, T=T, D=D, N=N, G=G, dtype=dtype, ragged=rng.random() < 0.4)
        if op == "scan":
            c["fresh"] = rng.random() < 0.5
        return c
    D = _log_int(rng, 64, 8192)
    rows = min(_log_int(rng, 1, 16384), max(1, (1 << 24) // D))
    return dict(op=op, rows=rows, D=D, rdt=rng.choice(["bf16", "f32"]),
                fdt=rng.choice(["bf16", "f32"]), xdt=rng.choice(["bf16", "f32"]))


# ---- inputs --------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return lo + (hi - lo) * torch.rand(shape, device="cuda", generator=g)

    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        rdt, fdt, xdt = (_DT[case[k]] for k in ("rdt", "fdt", "xdt"))
        s.update(r=normal(R, D, dtype=rdt, std=2.0), f=normal(R, D, dtype=fdt),
                 gate=normal(R, D, dtype=xdt), w_post=uniform(D, lo=0.5, hi=1.5),
                 scale=uniform(D, lo=0.05, hi=0.3), w_pre=uniform(D, lo=0.5, hi=1.5))
        if op == "norm_bwd":
            s.update(dr_out=normal(R, D, dtype=rdt), dn=normal(R, D, dtype=xdt))
        return s
    B, T, dt = case["B"], case["T"], _DT[case["dtype"]]
    s["lens"] = None
    if case["ragged"]:
        lens = torch.randint(0, T + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        lens[0] = T
        s["lens"] = lens
    if op in ("conv", "conv_bwd"):
        H, d, K = case["H"], case["d"], case["K"]
        s.update(x=normal(B, H, T, d, dtype=dt), w=normal(H, d, K, std=1.0 / math.sqrt(K)),
                 bias=normal(H, d, std=0.1), state=normal(B, H, K - 1, d, dtype=dt))
        if op == "conv_bwd":
            s["dy"] = normal(B, H, T, d, dtype=dt)
        return s
    D, N, G = case["D"], case["N"], case["G"]
    # steps between 1/1000 and 1/10 through the softplus, decays 1..N: the usual start of training
    dt0 = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s.update(u=normal(B, T, D, dtype=dt), delta=normal(B, T, D, dtype=dt, std=0.7),
             A=-(torch.arange(1, N + 1, device="cuda", dtype=torch.float32) *
                 uniform(D, 1, lo=0.8, hi=1.2)).contiguous(),
             Bm=normal(B, T, G, N, dtype=dt), Cm=normal(B, T, G, N, dtype=dt),
             Dskip=uniform(D, lo=0.5, hi=1.5), z=normal(B, T, D, dtype=dt),
             dt_bias=torch.log(torch.expm1(dt0)), state=normal(B, D, N, std=0.3))
    if op == "scan_bwd":
        s["dy"] = normal(B, T, D, dtype=dt)
    return s


# ---- the framework's calls -----------------------------------------------------------------

def _run_own(s):
    import sparse_state_linear_score_b200 as sdm
    c = s["case"]
    op = c["op"]
    if op == "conv":
        y = sdm.short_conv(s["x"], s["w"], s["bias"], state=s["state"], lens=s["lens"],
                           fresh=c["fresh"])
        return {"y": y, "state": s["state"]}
    if op == "conv_bwd":
        return sdm.short_conv_backward(s["x"], s["w"], s["dy"], s["bias"], state=s["state"],
                                       lens=s["lens"])
    if op == "scan":
        y = sdm.selective_scan(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], D=s["Dskip"], z=s["z"],
                               dt_bias=s["dt_bias"], state=s["state"], lens=s["lens"],
                               fresh=c["fresh"])
        return {"y": y, "state": s["state"]}
    if op == "scan_bwd":
        return sdm.selective_scan_backward(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["dy"],
                                           D=s["Dskip"], z=s["z"], dt_bias=s["dt_bias"],
                                           state=s["state"], lens=s["lens"])
    if op == "norm":
        r_out, n = sdm.block_norm(s["r"], s["f"], w_post=s["w_post"], gate=s["gate"],
                                  scale=s["scale"], w_pre=s["w_pre"])
        return {"r_out": r_out, "n": n}
    return sdm.block_norm_backward(s["r"], s["f"], s["dr_out"], s["dn"], w_post=s["w_post"],
                                   gate=s["gate"], scale=s["scale"], w_pre=s["w_pre"])


# ---- the plain form ------------------------------------------------------------------------

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _dsilu(x):
    sg = _sigmoid(x)
    return sg * (1.0 + x * (1.0 - sg))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def _valid(lens, T, like):
    """1 where token t of sequence b is inside it, [B, T]."""
    if lens is None:
        return None
    t = torch.arange(T, device=like.device)
    return (t[None, :] < lens[:, None]).float()


def _conv_pre(s, first):
    """(padded inputs [B,H,K-1+T,d], the convolution before its activation)"""
    x = s["x"].float()
    T, K = x.shape[2], s["w"].shape[2]
    xp = torch.cat([first, x], dim=2)
    pre = s["bias"][None, :, None, :]
    for j in range(K):
        pre = pre + s["w"][None, :, None, :, j] * xp[:, :, j:j + T]
    return xp, pre


def _plain_conv(s):
    c, x = s["case"], s["x"]
    B, H, T, d = x.shape
    K = c["K"]
    first = torch.zeros_like(s["state"]).float() if c["fresh"] else s["state"].float()
    xp, pre = _conv_pre(s, first)
    y = pre * _sigmoid(pre)
    ok = _valid(s["lens"], T, x)
    if ok is not None:
        y = y * ok[:, None, :, None]
        at = s["lens"].long()[:, None] + torch.arange(K - 1, device=x.device)[None, :]
        last = torch.gather(xp, 2, at[:, None, :, None].expand(B, H, K - 1, d))
    else:
        last = xp[:, :, T:]
    s["state"].copy_(last)
    return {"y": y.to(x.dtype), "state": s["state"]}


def _plain_conv_bwd(s):
    x = s["x"]
    T, K = x.shape[2], s["w"].shape[2]
    xp, pre = _conv_pre(s, s["state"].float())
    g = s["dy"].float() * _dsilu(pre)
    ok = _valid(s["lens"], T, x)
    if ok is not None:
        g = torch.where(ok[:, None, :, None] > 0, g, torch.zeros_like(g))
    dxp = torch.zeros_like(xp)
    dw = []
    for j in range(K):
        dxp[:, :, j:j + T] += s["w"][None, :, None, :, j] * g
        dw.append((g * xp[:, :, j:j + T]).sum(dim=(0, 2)))
    return {"dx": dxp[:, :, K - 1:].to(x.dtype), "dw": torch.stack(dw, dim=-1),
            "dbias": g.sum(dim=(0, 2)), "dstate": dxp[:, :, :K - 1].contiguous()}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 with h_{-1} = 0, by doubling."""
    T, k = a.shape[1], 1
    while k < T:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], dim=1)
        if 2 * k < T:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], dim=1)
        k *= 2
    return b


def _per_channel(m, D):
    """[B,T,G,N] -> [B,T,D,N]: the group's row for each of its channels."""
    B, T, G, N = m.shape
    return m.float()[:, :, :, None, :].expand(B, T, G, D // G, N).reshape(B, T, D, N)


def _states(s, h0, ok):
    """(step, decay, step * input, states) of every token; a token behind its sequence changes
    nothing: step 0, decay 1."""
    u = s["u"].float()
    step = _softplus(s["delta"].float() + s["dt_bias"])
    if ok is not None:
        step = torch.where(ok[:, :, None] > 0, step, torch.zeros_like(step))
        u = torch.where(ok[:, :, None] > 0, u, torch.zeros_like(u))
    a = torch.exp(step[..., None] * s["A"])
    b = (step * u)[..., None] * _per_channel(s["Bm"], u.shape[2])
    b[:, 0] += a[:, 0] * h0
    return u, step, a, _scan(a, b)


def _plain_scan(s):
    c = s["case"]
    T, D = s["u"].shape[1:]
    h0 = torch.zeros_like(s["state"]) if c["fresh"] else s["state"]
    ok = _valid(s["lens"], T, s["u"])
    u, step, a, h = _states(s, h0, ok)
    del a
    y = (_per_channel(s["Cm"], D) * h).sum(-1) + s["Dskip"] * u
    z = s["z"].float()
    y = y * (z * _sigmoid(z))
    if ok is not None:
        y = y * ok[:, :, None]
    s["state"].copy_(h[:, -1])
    return {"y": y.to(s["u"].dtype), "state": s["state"]}


def _plain_scan_bwd(s):
    dt = s["u"].dtype
    B, T, D = s["u"].shape
    G, N = s["Bm"].shape[2:]
    ok = _valid(s["lens"], T, s["u"])
    u, step, a, h = _states(s, s["state"], ok)
    Bc, Cc = _per_channel(s["Bm"], D), _per_channel(s["Cm"], D)
    z, dy = s["z"].float(), s["dy"].float()
    if ok is not None:
        dy = torch.where(ok[:, :, None] > 0, dy, torch.zeros_like(dy))
    y = (Cc * h).sum(-1) + s["Dskip"] * u
    dz = dy * y * _dsilu(z)
    dy = dy * (z * _sigmoid(z))
    # dh_t = C_t dy_t + a_{t+1} dh_{t+1}: the same scan, backwards
    an = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    dh = _scan(an.flip(1), (dy[..., None] * Cc).flip(1)).flip(1)
    hp = torch.cat([s["state"][:, None], h[:, :-1]], dim=1)
    q = dh * a * hp
    dA = (step[..., None] * q).sum(dim=(0, 1))
    sb = (dh * Bc).sum(-1)
    dstep = (s["A"] * q).sum(-1) + sb * u
    ddelta = dstep * _sigmoid(s["delta"].float() + s["dt_bias"])
    du = s["Dskip"] * dy + step * sb
    dB = (dh * (step * u)[..., None]).reshape(B, T, G, D // G, N).sum(3)
    dC = (h * dy[..., None]).reshape(B, T, G, D // G, N).sum(3)
    if ok is not None:
        ddelta = ddelta * ok[:, :, None]
        dC = dC * ok[:, :, None, None]
    return {"du": du.to(dt), "ddelta": ddelta.to(dt), "dA": dA, "dB": dB.to(dt), "dC": dC.to(dt),
            "dD": (dy * u).sum(dim=(0, 1)), "dz": dz.to(dt), "ddt_bias": ddelta.sum(dim=(0, 1)),
            "dstate": a[:, 0] * dh[:, 0]}


EPS = 1e-6


def _plain_norm(s):
    r, f = s["r"].float(), s["f"].float()
    p = f / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS) * s["w_post"]
    o = r + s["scale"] * _sigmoid(s["gate"].float()) * p
    n = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["w_pre"]
    return {"r_out": o.to(s["r"].dtype), "n": n.to(s["gate"].dtype)}


def _dnorm(x, w, dn):
    """(gradient of x, gradient of w) of x / sqrt(mean x^2 + eps) * w"""
    inv = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh, g = x * inv, dn * w
    return inv * (g - xh * (g * xh).mean(-1, keepdim=True)), (dn * xh).sum(0), xh


def _plain_norm_bwd(s):
    r, f = s["r"].float(), s["f"].float()
    sg = _sigmoid(s["gate"].float())
    fh = f / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
    p = fh * s["w_post"]
    o = r + s["scale"] * sg * p
    d1, dw_pre, _ = _dnorm(o, s["w_pre"], s["dn"].float())
    do = s["dr_out"].float() + d1
    df, dw_post, _ = _dnorm(f, s["w_post"], do * s["scale"] * sg)
    return {"dr": do.to(s["r"].dtype), "df": df.to(s["f"].dtype),
            "dgate": (do * s["scale"] * p * sg * (1.0 - sg)).to(s["gate"].dtype),
            "dscale": (do * sg * p).sum(0), "dw_post": dw_post, "dw_pre": dw_pre}


_PLAIN = {"conv": _plain_conv, "conv_bwd": _plain_conv_bwd, "scan": _plain_scan,
          "scan_bwd": _plain_scan_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        e = case["rows"] * case["D"]
        r, f, x = (4 if case[k] == "f32" else 2 for k in ("rdt", "fdt", "xdt"))
        if op == "norm":
            return {"bytes": e * (2 * r + f + 2 * x) + 12 * case["D"], "flops": 16 * e}
        return {"bytes": e * (3 * r + 2 * f + 3 * x) + 24 * case["D"], "flops": 40 * e}
    B, T = case["B"], case["T"]
    z = 4 if case["dtype"] == "f32" else 2
    # a padded batch: its sequences' lengths are drawn evenly, one of them is T
    tok = T * (1 + (B - 1) / 2) if case["ragged"] else B * T
    if op in ("conv", "conv_bwd"):
        c, K = case["H"] * case["d"], case["K"]
        st = B * c * (K - 1)
        if op == "conv":
            return {"bytes": 2 * tok * c * z + st * z * (1 if case["fresh"] else 2) + 4 * c * (K + 1),
                    "flops": tok * c * (2 * K + 5)}
        return {"bytes": (2 * tok + B * T) * c * z + st * (z + 4) + 8 * c * (K + 1),
                "flops": tok * c * (6 * K + 8)}
    D, N, G = case["D"], case["N"], case["G"]
    st = B * D * N * 4
    if op == "scan":
        return {"bytes": tok * z * (4 * D + 2 * G * N) + st * (1 if case["fresh"] else 2) +
                4 * D * (N + 2), "flops": tok * D * (7 * N + 12)}
    return {"bytes": (tok * (4 * D + 2 * G * N) + B * T * (3 * D + 2 * G * N)) * z + 2 * st +
            8 * D * (N + 2), "flops": tok * D * (21 * N + 30)}


# ---- the definition in 64 bits -------------------------------------------------------------
# Token by token, forwards and backwards; written from the definitions, not from the plain form.

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in s.items()}
    return _EXACT[case["op"]](s)


def _tokens(s, T, B):
    if s["lens"] is None:
        return torch.full((B,), T, device="cuda")
    return s["lens"].long()


def _sig64(x):
    return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), 1 - 1 / (1 + torch.exp(-x.abs())))


def _conv_token(s, win):
    """pre-activation of one token from its window [B,H,K,d] of inputs, oldest first"""
    return (win * s["w"].transpose(1, 2)[None]).sum(2) + s["bias"][None]


def _exact_conv(s):
    x = s["x"]
    B, H, T, d = x.shape
    win = torch.zeros_like(s["state"]) if s["case"]["fresh"] else s["state"].clone()
    n = _tokens(s, T, B)
    y = torch.zeros_like(x)
    for t in range(T):
        full = torch.cat([win, x[:, :, t:t + 1]], dim=2)
        pre = _conv_token(s, full)
        live = (t < n)[:, None, None]
        y[:, :, t] = torch.where(live, pre * _sig64(pre), torch.zeros_like(pre))
        win = torch.where(live[..., None], full[:, :, 1:], win)
    return {"y": y, "state": win}


def _exact_conv_bwd(s):
    x, dy = s["x"], s["dy"]
    B, H, T, d = x.shape
    K = s["w"].shape[2]
    n = _tokens(s, T, B)
    wins = torch.cat([s["state"], x], dim=2).unfold(2, K, 1).transpose(3, 4)  # [B,H,T,K,d]
    pre = (wins * s["w"].transpose(1, 2)[None, :, None]).sum(3) + s["bias"][None, :, None]
    sg = _sig64(pre)
    g = dy * (sg + pre * sg * (1 - sg))
    g = g * (torch.arange(T, device="cuda")[None] < n[:, None])[:, None, :, None]
    dwin = g[:, :, :, None] * s["w"].transpose(1, 2)[None, :, None]
    dxp = torch.zeros(B, H, T + K - 1, d, dtype=torch.float64, device="cuda")
    at = torch.arange(T, device="cuda")
    for j in range(K):
        dxp.index_add_(2, at + j, dwin[:, :, :, j])
    dw = (wins * g[:, :, :, None]).sum(dim=(0, 2)).transpose(1, 2)
    return {"dx": dxp[:, :, K - 1:], "dw": dw, "dbias": g.sum(dim=(0, 2)),
            "dstate": dxp[:, :, :K - 1]}


def _softplus64(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _exact_scan(s):
    u = s["u"]
    B, T, D = u.shape
    rep = D // s["Bm"].shape[2]
    n = _tokens(s, T, B)
    h = torch.zeros_like(s["state"]) if s["case"]["fresh"] else s["state"].clone()
    y = torch.zeros_like(u)
    for t in range(T):
        step = _softplus64(s["delta"][:, t] + s["dt_bias"])[..., None]
        Bt = s["Bm"][:, t].repeat_interleave(rep, dim=1)
        Ct = s["Cm"][:, t].repeat_interleave(rep, dim=1)
        new = torch.exp(step * s["A"]) * h + step * Bt * u[:, t, :, None]
        live = (t < n)[:, None]
        h = torch.where(live[..., None], new, h)
        zt = s["z"][:, t]
        out = ((h * Ct).sum(-1) + s["Dskip"] * u[:, t]) * zt * _sig64(zt)
        y[:, t] = torch.where(live, out, torch.zeros_like(out))
    return {"y": y, "state": h}


def _exact_scan_bwd(s):
    u = s["u"]
    B, T, D = u.shape
    G, N = s["Bm"].shape[2:]
    rep = D // G
    n = _tokens(s, T, B)
    h = s["state"].clone()
    before = torch.empty(B, T, D, N, dtype=torch.float64, device="cuda")
    raw = s["delta"] + s["dt_bias"]
    step = _softplus64(raw)

    def onward(h, t):
        return (torch.exp(step[:, t, :, None] * s["A"]) * h +
                (step[:, t] * u[:, t])[..., None] * s["Bm"][:, t].repeat_interleave(rep, dim=1))

    for t in range(T):
        before[:, t] = h
        h = torch.where((t < n)[:, None, None], onward(h, t), h)
    gr = {k: torch.zeros_like(s[v]) for k, v in (("du", "u"), ("ddelta", "delta"), ("dA", "A"),
                                                 ("dB", "Bm"), ("dC", "Cm"), ("dD", "Dskip"),
                                                 ("dz", "z"), ("ddt_bias", "dt_bias"))}
    dh = torch.zeros_like(h)
    for t in range(T - 1, -1, -1):
        live = (t < n)[:, None]
        zt, ut = s["z"][:, t], u[:, t]
        Bt = s["Bm"][:, t].repeat_interleave(rep, dim=1)
        Ct = s["Cm"][:, t].repeat_interleave(rep, dim=1)
        ht, st = onward(before[:, t], t), step[:, t]
        yt = (ht * Ct).sum(-1) + s["Dskip"] * ut
        sg = _sig64(zt)
        dout = torch.where(live, s["dy"][:, t], torch.zeros_like(zt))
        gr["dz"][:, t] = dout * yt * sg * (1 + zt * (1 - sg))
        dp = dout * zt * sg
        gr["dD"] += (dp * ut).sum(0)
        gr["dC"][:, t] = (dp[..., None] * ht).reshape(B, G, rep, N).sum(2)
        cur = torch.where(live[..., None], dh + dp[..., None] * Ct, torch.zeros_like(dh))
        decay = torch.exp(st[..., None] * s["A"])
        back = cur * decay * before[:, t]
        gr["dA"] += (back * st[..., None]).sum(0)
        gr["dB"][:, t] = (cur * (st * ut)[..., None]).reshape(B, G, rep, N).sum(2)
        along = (cur * Bt).sum(-1)
        gr["du"][:, t] = dp * s["Dskip"] + along * st
        draw_ = ((back * s["A"]).sum(-1) + along * ut) * _sig64(raw[:, t])
        gr["ddelta"][:, t] = draw_
        gr["ddt_bias"] += draw_.sum(0)
        dh = torch.where(live[..., None], cur * decay, dh)
    gr["dstate"] = dh
    return gr


def _rms64(x):
    return torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _exact_norm(s):
    o = s["r"] + s["scale"] * _sig64(s["gate"]) * (s["w_post"] * s["f"] / _rms64(s["f"]))
    return {"r_out": o, "n": s["w_pre"] * o / _rms64(o)}


def _exact_norm_bwd(s):
    D = s["f"].shape[1]
    sg, rf = _sig64(s["gate"]), _rms64(s["f"])
    p = s["w_post"] * s["f"] / rf
    o = s["r"] + s["scale"] * sg * p
    ro = _rms64(o)
    gn = s["dn"] * s["w_pre"]
    do = s["dr_out"] + gn / ro - o * (gn * o).sum(-1, keepdim=True) / (D * ro ** 3)
    dp = do * s["scale"] * sg
    gp = dp * s["w_post"]
    df = gp / rf - s["f"] * (gp * s["f"]).sum(-1, keepdim=True) / (D * rf ** 3)
    return {"dr": do, "df": df, "dgate": do * s["scale"] * p * sg * (1 - sg),
            "dscale": (do * sg * p).sum(0), "dw_post": (dp * s["f"] / rf).sum(0),
            "dw_pre": (s["dn"] * o / ro).sum(0)}


_EXACT = {"conv": _exact_conv, "conv_bwd": _exact_conv_bwd, "scan": _exact_scan,
          "scan_bwd": _exact_scan_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd}
