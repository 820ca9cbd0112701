"""The fp64 forms of the state-space block's operators against autograd and differences (CPU)."""
import pytest
import torch

from tests import ssm_reference as R


def _leaf(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).requires_grad_()


def _close(a, b, what):
    assert torch.allclose(a, b, rtol=1e-10, atol=1e-12), what


@pytest.mark.parametrize("K,act,lens", [(1, True, None), (3, True, [5, 2, 0]), (4, False, [6, 1, 3]),
                                        (8, True, [6, 6, 2])])
def test_conv_formulas(K, act, lens):
    g = torch.Generator().manual_seed(K)
    B, H, T, d = 3, 2, 6, 3
    x, w, bias = _leaf(g, B, H, T, d), _leaf(g, H, d, K), _leaf(g, H, d)
    st = _leaf(g, B, H, K - 1, d)
    y, end = R.conv(x, w, bias, act, st, lens)
    dy, de = torch.randn(y.shape, generator=g, dtype=y.dtype), torch.randn(end.shape, generator=g,
                                                                         dtype=y.dtype)
    grads = torch.autograd.grad((y * dy).sum() + (end * de).sum(), (x, w, bias, st),
                                allow_unused=True)
    got = R.conv_bwd(x, w, bias, act, st, lens, dy, de)
    for k, a in zip(("dx", "dw", "dbias", "dstate"), grads):
        if a is not None:
            _close(got[k], a, k)


@pytest.mark.parametrize("sp,opt,lens,G", [(True, True, None, 1), (True, True, [5, 0, 1], 2),
                                           (False, False, [3, 5, 4], 2)])
def test_scan_formulas(sp, opt, lens, G):
    g = torch.Generator().manual_seed(G)
    B, T, D, N = 3, 5, 4, 3
    u, de = _leaf(g, B, T, D), _leaf(g, B, T, D)
    A = (-torch.rand(D, N, generator=g, dtype=torch.float64) - 0.1).requires_grad_()
    Bm, Cm, st = _leaf(g, B, T, G, N), _leaf(g, B, T, G, N), _leaf(g, B, D, N)
    Ds, z, db = (_leaf(g, D), _leaf(g, B, T, D), _leaf(g, D)) if opt else (None, None, None)
    y, end = R.scan(u, de, A, Bm, Cm, Ds, z, db, st, lens, sp)
    dy = torch.randn(y.shape, generator=g, dtype=y.dtype)
    dend = torch.randn(end.shape, generator=g, dtype=y.dtype)
    names = ["du", "ddelta", "dA", "dB", "dC", "dstate"] + (["dD", "dz", "ddt_bias"] if opt else [])
    leaves = [u, de, A, Bm, Cm, st] + ([Ds, z, db] if opt else [])
    grads = torch.autograd.grad((y * dy).sum() + (end * dend).sum(), leaves)
    got = R.scan_bwd(u, de, A, Bm, Cm, dy, Ds, z, db, st, lens, sp, dend)
    for k, a in zip(names, grads):
        _close(got[k], a, k)
    # and one direction by central differences
    with torch.no_grad():
        dirs = [torch.randn(v.shape, generator=g, dtype=v.dtype) for v in leaves]

        def loss(e):
            v = [a + e * b for a, b in zip(leaves, dirs)]
            o = (v[6], v[7], v[8]) if opt else (None, None, None)
            yy, ee = R.scan(v[0], v[1], v[2], v[3], v[4], *o, v[5], lens, sp)
            return float((yy * dy).sum() + (ee * dend).sum())
        num = (loss(1e-5) - loss(-1e-5)) / 2e-5
        ana = sum(float((got[k] * b).sum()) for k, b in zip(names, dirs))
        assert abs(num - ana) <= 1e-6 * (1 + abs(ana))


@pytest.mark.parametrize("full", [True, False])
def test_norm_formulas(full):
    g = torch.Generator().manual_seed(7)
    r, f = _leaf(g, 4, 9), _leaf(g, 4, 9)
    opt = [_leaf(g, 9), _leaf(g, 4, 9), _leaf(g, 9), _leaf(g, 9)] if full else [None] * 4
    o, n = R.norm(r, f, *opt)
    dro, dn = torch.randn(4, 9, generator=g, dtype=o.dtype), torch.randn(4, 9, generator=g,
                                                                       dtype=o.dtype)
    names = ["dr", "df"] + (["dw_post", "dgate", "dscale", "dw_pre"] if full else [])
    grads = torch.autograd.grad((o * dro).sum() + (n * dn).sum(), [r, f] + [x for x in opt if x is not None])
    got, mag = R.norm_bwd(r, f, dro, dn, *opt)
    for k, a in zip(names, grads):
        _close(got[k], a, k)
        assert (mag[k] >= got[k].abs() * (1 - 1e-12)).all(), k


@pytest.mark.parametrize("K,act,lens,bias", [(1, True, None, True), (4, False, [5, 2, 0], True),
                                             (8, True, [6, 1, 6], False)])
def test_conv_of_all_tokens_at_once(K, act, lens, bias):
    g = torch.Generator().manual_seed(K)
    r = lambda *n: torch.randn(n, generator=g, dtype=torch.float64)  # noqa: E731
    B, H, T, d = 3, 2, 6, 3
    x, w, b, st = r(B, H, T, d), r(H, d, K), r(H, d) if bias else None, r(B, H, K - 1, d)
    dy, de = r(B, H, T, d), r(B, H, K - 1, d)
    for mag, got in zip((False, True), R.conv_all(x, w, b, act, st, lens, dy, de)):
        y, end = R.conv(x, w, b, act, st, lens, mag)
        want = dict(R.conv_bwd(x, w, b, act, st, lens, dy, de, mag), y=y)
        if not mag:
            want["state"] = end
        for k in want:
            _close(got[k], want[k], (k, mag))


@pytest.mark.parametrize("rows,D,dt", [(3, 16384, torch.bfloat16), (2, 16383, torch.float32),
                                       (2, 8191, torch.float32), (5, 64, torch.float32)])
def test_norm_gradients_without_a_mean_are_told_apart(rows, D, dt):
    """The check that the kernels' gradients pass on R.along's inputs rejects a gradient that leaves
    out mean(m o^) in dr, or mean(q f^) in df."""
    rr, ff, opt, dro, dn = R.along(rows, D, dt, dt, dt, (1, 1, 1, 1), torch.Generator().manual_seed(D))
    r, f, dr0, m0 = (v.double() for v in (rr, ff, dro, dn))
    o64 = {k: v.double() for k, v in opt.items()}
    ref, _ = R.norm_bwd(r, f, dr0, m0, **o64)
    o, _ = R.norm(r, f, **o64)
    ro = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6)
    rf = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + 1e-6)
    share = o64["scale"] * R.sigmoid(o64["gate"]) * o64["w_post"]
    for name, do in (("dr", dr0 + ro * m0 * o64["w_pre"]), ("df", ref["dr"])):
        bad = do if name == "dr" else rf * do * share
        assert R.off(ref[name].to(dt), ref[name]) <= 2.0 ** -8
        assert R.off(bad.to(dt), ref[name]) > 0.05, name
