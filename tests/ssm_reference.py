"""The state-space block's operators written out in fp64 (torch, on the CPU), token by token, with
their gradients, and bounds for the fp32 kernels.

Every function has a form `mag=True` that replaces each term by its absolute value.  A sum of
products computed in fp32 with n roundings is off by at most about n * U times that magnitude
(U = 2^-24), whatever the order of the sum, which is how the tests derive their tolerances:

  - a step of the scan costs 6 roundings: exp2 of a rounded product (ex2.approx: 2^-22 = 4 U; its
    argument x is off by 2 U |x| ln 2, and e^-x x < 0.37) and one multiply-add;
  - sigmoid, its derivative and softplus are within 64 U for the arguments drawn here (|x| < 8:
    __expf is within 2 + 1.2 |x| steps of 2 U, the division within 4 U, log1p within 2 U);
  - a sum of m terms adds m U.

An output is then rounded once to its type: half a step, finfo(type).eps / 2 of its value.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def _ab(x, mag):
    return x.abs() if mag and x is not None else x


def sigmoid(x):
    return torch.sigmoid(x)


def silu(x, mag=False):
    return _ab(x, mag) * sigmoid(x)


def dsilu(x, mag=False):
    s = sigmoid(x)
    return s * (1 + (x.abs() if mag else x) * (1 - s))


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _lens(lens, B, T):
    if lens is None:
        return [T] * B
    return [max(0, min(T, int(n))) for n in lens]


# ---- short convolution ---------------------------------------------------------------------

def conv(x, w, bias, act, state, lens, mag=False):
    """x [B,H,T,d], w [H,d,K] -> (y (zero behind lens), state after the call)"""
    B, H, T, d = x.shape
    K = w.shape[2]
    if state is None:
        state = torch.zeros(B, H, K - 1, d, dtype=x.dtype)
    y = torch.zeros_like(x)
    out = state.clone()
    for b, n in enumerate(_lens(lens, B, T)):
        xp = torch.cat([state[b], x[b, :, :n]], dim=1)  # [H, K-1+n, d]
        for t in range(n):
            win = xp[:, t:t + K].transpose(1, 2)
            p = (win * w).sum(-1) + (0 if bias is None else bias)
            if mag:
                p = (win.abs() * w.abs()).sum(-1) + (0 if bias is None else bias.abs())
            # |d silu| < 1.1, so p's error carries over times 1.1
            y[b, :, t] = 1.1 * p if mag else (silu(p) if act else p)
        out[b] = xp[:, xp.shape[1] - (K - 1):] if K > 1 else out[b]
    return y, out


def conv_bwd(x, w, bias, act, state, lens, dy, dstate_end, mag=False):
    B, H, T, d = x.shape
    K = w.shape[2]
    if state is None:
        state = torch.zeros(B, H, K - 1, d, dtype=x.dtype)
    dx, dst = torch.zeros_like(x), torch.zeros_like(state)
    dw, db = torch.zeros_like(w), torch.zeros(H, d, dtype=x.dtype)
    wa = _ab(w, mag)
    for b, n in enumerate(_lens(lens, B, T)):
        xp = torch.cat([state[b], x[b, :, :n]], dim=1)
        dxp = torch.zeros_like(xp)
        if dstate_end is not None and K > 1:
            dxp[:, xp.shape[1] - (K - 1):] += _ab(dstate_end[b], mag)
        for t in range(n):
            win = xp[:, t:t + K].transpose(1, 2)
            p = (win * w).sum(-1) + (0 if bias is None else bias)
            g = _ab(dy[b, :, t], mag)
            if act:
                if mag:  # |dsilu| and, for p's own error, |d2 silu| < 0.5
                    pa = (win.abs() * w.abs()).sum(-1) + (0 if bias is None else bias.abs())
                    g = g * (dsilu(p, True) + 0.5 * pa)
                else:
                    g = g * dsilu(p)
            dxp[:, t:t + K] += (g[..., None] * wa).transpose(1, 2)
            dw += g[..., None] * _ab(win, mag)
            db += g
        dx[b, :, :n] = dxp[:, K - 1:]
        dst[b] = dxp[:, :K - 1]
    return {"dx": dx, "dw": dw, "dbias": db, "dstate": dst}


def conv_all(x, w, bias, act, state, lens, dy, dstate_end):
    """conv and conv_bwd for calls of many tokens, on x's device, all tokens at once -> (values,
    magnitudes): dicts of y, state, dx, dw, dbias, dstate."""
    B, H, T, d = x.shape
    K = w.shape[2]
    n = torch.tensor(_lens(lens, B, T), device=x.device)
    m = (torch.arange(T, device=x.device) < n[:, None])[:, None, :, None]
    x, dy = x.masked_fill(~m, 0), dy.masked_fill(~m, 0)
    xp = torch.cat([state, x], dim=2)
    at = (n[:, None, None, None] + torch.arange(K - 1, device=x.device)[:, None]).expand(B, H, K - 1, d)
    tap = lambda v, j: v[:, :, j:j + T]  # noqa: E731
    b = 0 if bias is None else bias[None, :, None]
    p = sum(tap(xp, j) * w[None, :, None, :, j] for j in range(K)) + b
    pa = sum(tap(xp, j).abs() * w[None, :, None, :, j].abs() for j in range(K)) + abs(b)
    out = []
    for mag in (False, True):
        v = {"y": (1.1 * pa if mag else silu(p) if act else p) * m, "state": xp.gather(2, at)}
        g = _ab(dy, mag)
        if act:
            g = g * (dsilu(p, True) + 0.5 * pa if mag else dsilu(p))
        g = g * m
        dxp = torch.zeros_like(xp).scatter_add_(2, at, _ab(dstate_end, mag))
        for j in range(K):
            tap(dxp, j).add_(g * _ab(w, mag)[None, :, None, :, j])
        v["dx"], v["dstate"] = dxp[:, :, K - 1:] * m, dxp[:, :, :K - 1]
        v["dw"] = torch.stack([(g * tap(_ab(xp, mag), j)).sum((0, 2)) for j in range(K)], dim=-1)
        v["dbias"] = g.sum((0, 2))
        out.append(v)
    return out


# ---- selective scan ------------------------------------------------------------------------

def _rep(m, D):
    """[G,N] -> [D,N]"""
    return m.repeat_interleave(D // m.shape[0], dim=0)


def scan(u, delta, A, Bm, Cm, D=None, z=None, dt_bias=None, state=None, lens=None, sp=True,
         mag=False):
    """-> (y (zero behind lens), state after the call)"""
    B, T, Dn = u.shape
    N = A.shape[1]
    y = torch.zeros_like(u)
    out = torch.zeros(B, Dn, N, dtype=u.dtype)
    for b, n in enumerate(_lens(lens, B, T)):
        h = torch.zeros(Dn, N, dtype=u.dtype) if state is None else _ab(state[b], mag).clone()
        for t in range(n):
            raw = delta[b, t] + (0 if dt_bias is None else dt_bias)
            s = softplus(raw) if sp else raw
            h = torch.exp(s[:, None] * A) * h + \
                _ab((s * u[b, t])[:, None] * _rep(Bm[b, t], Dn), mag)
            v = (_ab(_rep(Cm[b, t], Dn), mag) * h).sum(-1)
            if D is not None:
                v = v + _ab(D * u[b, t], mag)
            if z is not None:
                v = v * silu(z[b, t], mag)
            y[b, t] = v
        out[b] = h
    return y, out


def scan_bwd(u, delta, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, state=None, lens=None, sp=True,
             dstate_end=None, mag=False):
    B, T, Dn = u.shape
    G, N = Bm.shape[2:]
    f = dict(dtype=u.dtype)
    g = {"du": torch.zeros_like(u), "ddelta": torch.zeros_like(u), "dz": torch.zeros_like(u),
         "dA": torch.zeros_like(A), "dB": torch.zeros_like(Bm), "dC": torch.zeros_like(Cm),
         "dD": torch.zeros(Dn, **f), "ddt_bias": torch.zeros(Dn, **f),
         "dstate": torch.zeros(B, Dn, N, **f)}
    fold = lambda x: x.reshape(G, Dn // G, N).sum(1)  # noqa: E731
    for b, n in enumerate(_lens(lens, B, T)):
        h = torch.zeros(Dn, N, **f) if state is None else _ab(state[b], mag).clone()
        raw = delta[b] + (0 if dt_bias is None else dt_bias)
        s = softplus(raw) if sp else raw
        hs = [h]
        for t in range(n):
            h = torch.exp(s[t][:, None] * A) * h + \
                _ab((s[t] * u[b, t])[:, None] * _rep(Bm[b, t], Dn), mag)
            hs.append(h)
        c = torch.zeros(Dn, N, **f) if dstate_end is None else _ab(dstate_end[b], mag).clone()
        for t in range(n - 1, -1, -1):
            Bt, Ct = _ab(_rep(Bm[b, t], Dn), mag), _ab(_rep(Cm[b, t], Dn), mag)
            ut, st, dyt = _ab(u[b, t], mag), _ab(s[t], mag), _ab(dy[b, t], mag)
            dp = dyt
            if z is not None:
                yt = (Ct * hs[t + 1]).sum(-1) + (0 if D is None else _ab(D, mag) * ut)
                g["dz"][b, t] = dyt * yt * _ab(dsilu(z[b, t], mag), mag)
                dp = dyt * silu(z[b, t], mag)
            dh = Ct * dp[:, None] + c
            w = dh * torch.exp(s[t][:, None] * A)
            q = w * hs[t]
            along = (dh * Bt).sum(-1)
            g["dA"] += st[:, None] * q
            g["dB"][b, t] = fold(dh * (st * ut)[:, None])
            g["dC"][b, t] = fold(dp[:, None] * hs[t + 1])
            g["du"][b, t] = (0 if D is None else _ab(D, mag) * dp) + st * along
            dd = (_ab(A, mag) * q).sum(-1) + along * ut
            if sp:
                dd = dd * sigmoid(raw[t])
            g["ddelta"][b, t] = dd
            g["ddt_bias"] += dd
            g["dD"] += dp * ut
            c = w
        g["dstate"][b] = c
    return g


# ---- block norms ---------------------------------------------------------------------------

def norm(r, f, w_post=None, gate=None, scale=None, w_pre=None, eps=1e-6):
    p = f
    if w_post is not None:
        p = f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps) * w_post
    if gate is not None:
        p = p * sigmoid(gate)
    if scale is not None:
        p = p * scale
    o = r + p
    n = o / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    return o, n if w_pre is None else n * w_pre


def norm_bwd(r, f, dr_out, dn, w_post=None, gate=None, scale=None, w_pre=None, eps=1e-6):
    """The formulas, and for each output a magnitude (row by row, terms in absolute value)."""
    one = torch.ones(f.shape[-1], dtype=f.dtype)
    D = f.shape[-1]
    wp, sc, wq = (one if v is None else v for v in (w_post, scale, w_pre))
    s = torch.ones_like(f) if gate is None else sigmoid(gate)
    rf = torch.ones_like(f[..., :1])
    if w_post is not None:
        rf = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + eps)
    fh = f * rf
    p = fh * wp
    o = r + sc * s * p
    ro = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + eps)
    oh = o * ro
    dn0 = torch.zeros_like(f) if dn is None else dn
    dr0 = torch.zeros_like(f) if dr_out is None else dr_out
    m = dn0 * wq
    do = dr0 + ro * (m - oh * (m * oh).mean(-1, keepdim=True))
    dom = dr0.abs() + ro * (m.abs() + oh.abs() * (m * oh).abs().mean(-1, keepdim=True))
    # o cancels where r and the block's share do: its error against its own size
    blow = 1 + (r.abs() + (sc * s * p).abs()).max() / o.abs().mean(-1, keepdim=True)
    dom = dom * blow
    dp, dpm = do * sc * s, dom * (sc * s).abs()
    q, qm = dp * wp, dpm * wp.abs()
    df = q if w_post is None else rf * (q - fh * (q * fh).mean(-1, keepdim=True))
    dfm = qm if w_post is None else rf * (qm + fh.abs() * (qm * fh.abs()).mean(-1, keepdim=True))
    v = {"dr": do, "df": df, "dgate": do * sc * p * s * (1 - s), "dscale": (do * s * p), "dw_post": dp * fh,
         "dw_pre": dn0 * oh}
    mag = {"dr": dom, "df": dfm, "dgate": dom * (sc * p).abs(), "dscale": dom * (s * p).abs(),
           "dw_post": dpm * fh.abs(), "dw_pre": dn0.abs() * (1 + oh.abs()) * blow}
    for k in ("dscale", "dw_post", "dw_pre"):
        v[k], mag[k] = v[k].reshape(-1, D).sum(0), mag[k].reshape(-1, D).sum(0)
    return v, mag


def along(rows, D, r, f, x, has, g, eps=1e-6, std=1.0):
    """Inputs of a norm whose gradients lie along its rows, dn along o^ and dr_out along f^, so that
    the means which the gradient takes off are of its own size (of independent ones they are
    D^-1/2 of it, and a gradient without them would pass)."""
    rnd = lambda dt, s=1.0: (torch.randn(rows, D, generator=g) * s).to(dt)  # noqa: E731
    vec = [torch.rand(D, generator=g) + 0.5 for _ in range(3)]
    rr, ff = rnd(r, std), rnd(f, std)
    opt = {"w_post": vec[0] if has[0] else None, "gate": rnd(x) if has[1] else None,
           "scale": vec[1] if has[2] else None, "w_pre": vec[2] if has[3] else None}
    o, n = norm(rr.double(), ff.double(), **{k: None if v is None else v.double() for k, v in opt.items()},
                eps=eps)
    oh = n if opt["w_pre"] is None else n / opt["w_pre"].double()
    dn = rnd(x).double() + oh / (1 if opt["w_pre"] is None else opt["w_pre"].double())
    dr = rnd(r).double() + ff.double() / std
    return rr, ff, opt, dr.to(r), dn.to(x)


# ---- checks --------------------------------------------------------------------------------

def within(got, ref, mag, roundings, what):
    """|got - ref| <= roundings * U * mag + half a step of got's type, element by element."""
    got64 = got.detach().double().cpu()
    assert got64.shape == ref.shape, (what, got64.shape, ref.shape)
    step = torch.finfo(got.dtype).eps / 2
    tol = roundings * U * mag
    tol = tol * (1 + step) + step * ref.abs() + 1e-37
    err = (got64 - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / tol).nan_to_num(float('inf')).max()):.3g} of its bound")


def off(got, ref):
    """|got - ref| / |ref|, of the whole tensors."""
    got, ref = got.detach().double(), ref.to(got.device)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    return float((got - ref).norm() / ref.norm())
