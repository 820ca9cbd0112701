"""GPU parity of the state-space block: short convolution, selective scan, block norms, their
gradients, their forms for single tokens and padded batches, against the fp64 definitions of
tests/ssm_reference.py (which also derives the tolerances)."""
from __future__ import annotations

import threading

import pytest
import torch

import oracle
from tests import ssm_reference as R
from tests.parity import f64, normwise_rel_err

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sdm():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_state_linear_score_b200 as m
    m.device_error(clear=True)
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dt=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dt)


def up(x):
    return None if x is None else x.cuda()


def d64(x):
    return None if x is None else x.double()


def poison(x, lens, axis):
    """NaN and infinities behind the sequences: they must not be read."""
    x = x.clone()
    for b, n in enumerate(lens):
        v = x[b].movedim(axis - 1, 0)
        v[n:] = float("nan")
        if n + 1 < v.shape[0]:
            v[n + 1:] = float("inf")
    return x


def strided(x, pad, off=0):
    """x on the GPU as a column slice of a wider tensor."""
    w = torch.full((*x.shape[:-1], x.shape[-1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    v = w[..., off:off + x.shape[-1]]
    v.copy_(x)
    return v


# ---- short convolution ---------------------------------------------------------------------

CONV = [  # B, H, T, d, K, dtype, act, bias, lens, view (pad, off)
    (2, 3, 37, 16, 4, "f32", "silu", True, None, None),
    (2, 3, 300, 32, 4, "bf16", "silu", True, None, None),
    (3, 1, 70, 50, 3, "bf16", "silu", True, [70, 0, 33], None),
    (3, 2, 9, 7, 2, "f32", None, False, [1, 9, 2], None),
    (2, 2, 33, 8, 8, "bf16", "silu", False, None, (24, 8)),
    (2, 2, 40, 12, 5, "f32", "silu", True, [40, 3], (5, 3)),
    (4, 2, 1, 64, 4, "bf16", "silu", True, None, None),
    (4, 2, 1, 64, 4, "f32", "silu", True, [1, 0, 1, 0], None),
    (2, 1, 2, 20, 6, "f32", "silu", True, None, None),
    (1, 2, 65, 24, 1, "f32", "silu", True, None, None),
    (2, 2, 129, 36, 7, "f32", "silu", True, [100, 129], None),
    (1, 16, 1111, 64, 4, "bf16", "silu", True, None, None),
]


def conv_case(B, H, T, d, K, dtype, act, bias, lens, seed=0):
    g = gen(1000 * K + T + seed)
    dt = DT[dtype]
    x, w = rnd(g, B, H, T, d, dt=dt), rnd(g, H, d, K, std=0.6)
    return x, w, (rnd(g, H, d, std=0.3) if bias else None), rnd(g, B, H, K - 1, d, dt=dt), \
        rnd(g, B, H, T, d, dt=dt), rnd(g, B, H, K - 1, d), act


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("B,H,T,d,K,dtype,act,bias,lens,view", CONV)
def test_conv(sdm, B, H, T, d, K, dtype, act, bias, lens, view, fresh):
    x, w, b, st, _, _, act = conv_case(B, H, T, d, K, dtype, act, bias, lens)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    xp = x if lens is None else poison(x, lens, 2)
    xg = up(xp) if view is None else strided(xp, *view)
    stg = st.cuda()
    y = torch.full((B, H, T, d), 77.0, dtype=x.dtype, device="cuda")
    yv = y if view is None else strided(y, *view)
    sdm.short_conv(xg, up(w), up(b), act=act, state=stg, lens=up(ln), fresh=fresh, y=yv)
    s64 = None if fresh else st.double()
    ref, end = R.conv(x.double(), w.double(), d64(b), act, s64, lens)
    mag, _ = R.conv(x.double(), w.double(), d64(b), act, s64, lens, mag=True)
    for q, n in enumerate(lens or [T] * B):
        # K multiply-adds and the bias, then the sigmoid
        R.within(yv[q, :, :n], ref[q, :, :n], mag[q, :, :n], K + 1 + (64 if act else 0), "y")
        assert (yv[q, :, n:] == 77.0).all(), "rows behind the sequence are left as they were"
    assert torch.equal(stg.cpu().double(), end), "the state holds the inputs themselves"


@pytest.mark.parametrize("ends", [False, True])
@pytest.mark.parametrize("B,H,T,d,K,dtype,act,bias,lens,view", CONV)
def test_conv_backward(sdm, B, H, T, d, K, dtype, act, bias, lens, view, ends):
    x, w, b, st, dy, de, act = conv_case(B, H, T, d, K, dtype, act, bias, lens)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    xp, dyp = (x, dy) if lens is None else (poison(x, lens, 2), poison(dy, lens, 2))
    put = up if view is None else (lambda v: strided(v, *view))
    g = sdm.short_conv_backward(put(xp), up(w), put(dyp), up(b), act=act, state=up(st) if ends else None,
                                lens=up(ln), dstate_end=up(de) if ends else None)
    a = (x.double(), w.double(), d64(b), act, st.double() if ends else None, lens, dy.double(),
         de.double() if ends else None)
    ref, mag = R.conv_bwd(*a), R.conv_bwd(*a, mag=True)
    n = K + 1 + (128 if act else 0)  # p, dsilu and the products
    R.within(g["dx"], ref["dx"], mag["dx"], n + K + 1, "dx")
    R.within(g["dw"], ref["dw"], mag["dw"], n + B * T, "dw")
    assert ("dbias" in g) == bias and ("dstate" in g) == ends
    if bias:
        R.within(g["dbias"], ref["dbias"], mag["dbias"], n + B * T, "dbias")
    if ends:
        R.within(g["dstate"], ref["dstate"], mag["dstate"], n + K + 1, "dstate")


@pytest.mark.parametrize("cuts", [[1] * 6, [3, 2, 1], [4, 0, 2]])
def test_conv_calls_chain(sdm, cuts):
    """A sequence in several calls, single tokens among them, equals one call bit for bit."""
    x, w, b, st, _, _, _ = conv_case(2, 2, 6, 16, 4, "bf16", "silu", True, None)
    s1, s2 = st.cuda(), st.cuda()
    whole = sdm.short_conv(up(x), up(w), up(b), state=s1)
    parts, t = [], 0
    for n in cuts:
        parts.append(sdm.short_conv(x[:, :, t:t + n].contiguous().cuda(), up(w), up(b), state=s2))
        t += n
    assert torch.equal(torch.cat(parts, dim=2), whole) and torch.equal(s1, s2)


@pytest.mark.parametrize("K,d,dtype", [(2, 7, "f32"), (4, 8, "bf16"), (4, 8, "f32"), (8, 12, "bf16")])
def test_conv_backward_of_sequences_without_tokens(sdm, K, d, dtype):
    """What an empty sequence's state holds, and the gradient that comes to it, are its own: the
    filters' gradients are those of the others.  Behind a sequence dx is zero whatever the filters."""
    B, H, T, lens = 3, 2, 40, [5, 0, 33]
    x, w, b, st, dy, de, act = conv_case(B, H, T, d, K, dtype, "silu", True, lens)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    xg, dyg = poison(x, lens, 2).cuda(), poison(dy, lens, 2).cuda()
    st[1], de[1] = 0, 0
    want = sdm.short_conv_backward(xg, up(w), dyg, up(b), state=up(st), lens=ln, dstate_end=up(de))
    for bad in (float("nan"), float("inf")):
        st[1], de[1] = bad, bad
        g = sdm.short_conv_backward(xg, up(w), dyg, up(b), state=up(st), lens=ln, dstate_end=up(de))
        for k in ("dx", "dw", "dbias"):
            assert torch.equal(g[k], want[k]), (k, bad)
        assert torch.equal(g["dstate"][::2], want["dstate"][::2])
        assert torch.equal(g["dstate"][1].cpu().nan_to_num(7, 8), de[1].nan_to_num(7, 8))
    w[0, 1], w[1, 3, 0] = float("nan"), float("inf")
    g = sdm.short_conv_backward(xg, up(w), dyg, up(b), lens=ln)
    for q, n in enumerate(lens):
        assert (g["dx"][q, :, n:] == 0).all()


# ---- selective scan ------------------------------------------------------------------------

SCAN = [  # B, T, D, N, G, dtype, softplus, opt (z, D, dt_bias), lens, view
    (2, 37, 24, 16, 1, "f32", True, True, None, None),
    (2, 50, 40, 16, 2, "bf16", True, True, None, None),
    (3, 70, 33, 16, 1, "f32", True, True, [70, 0, 33], None),
    (3, 65, 30, 7, 3, "f32", True, True, [64, 65, 1], (6, 1)),
    (1, 200, 20, 4, 1, "f32", False, False, None, None),
    (2, 130, 12, 32, 1, "bf16", True, True, [130, 65], None),
    (1, 129, 10, 64, 2, "f32", True, True, None, (10, 2)),
    (2, 40, 9, 45, 1, "f32", True, False, None, None),
    (2, 30, 150, 8, 1, "bf16", True, True, None, None),
    (1, 700, 16, 16, 1, "f32", True, True, None, None),
    (3, 2, 140, 16, 1, "f32", True, True, [2, 1, 0], None),
    (4, 1, 70, 16, 2, "f32", True, True, [1, 0, 1, 0], None),
    (4, 1, 70, 16, 1, "bf16", True, True, None, (3, 0)),
    (2, 1, 33, 5, 1, "f32", True, False, None, None),
    (2, 1, 20, 33, 2, "f32", True, True, None, None),
    (1, 1, 20, 64, 1, "f32", False, True, None, None),
    # four sequences a thread, the last ones missing
    (13, 1, 9600, 16, 1, "bf16", True, True, [1, 0, 1, 1, 1, 1, 0, 0, 1, 1, 1, 1, 0], None),
    (14, 1, 20000, 7, 2, "f32", True, True, None, None),
    # split over time, sequences that end in the first and in a middle chunk; rows at odd addresses
    (3, 900, 24, 16, 1, "f32", True, True, [900, 333, 20], None),
    (2, 700, 9, 11, 1, "bf16", True, True, [95, 700], None),
    (2, 300, 33, 3, 1, "bf16", True, True, [300, 161], (1, 1)),
    (1, 260, 6, 1, 3, "bf16", True, False, None, None),
    (2, 90, 5, 2, 1, "f32", True, True, [64, 32], None),
    (1, 150, 300, 16, 3, "bf16", True, True, None, (4, 4)),
]


def scan_case(B, T, D, N, G, dtype, sp, opt, seed=0):
    g = gen(100 * N + T + seed)
    dt = DT[dtype]
    c = {"u": rnd(g, B, T, D, dt=dt), "delta": rnd(g, B, T, D, dt=dt, std=0.7),
         "A": -(torch.rand(D, N, generator=g) * 4 + 0.05),
         "B": rnd(g, B, T, G, N, dt=dt), "C": rnd(g, B, T, G, N, dt=dt)}
    if not sp:
        c["delta"] = (torch.rand(B, T, D, generator=g) * 0.5).to(dt)
    o = {"D": rnd(g, D), "z": rnd(g, B, T, D, dt=dt), "dt_bias": rnd(g, D, std=1.0) - 2}
    return c, o if opt else {}, rnd(g, B, D, N, std=0.5), rnd(g, B, T, D, dt=dt), \
        rnd(g, B, D, N, std=0.5)


def scan_ref(c, o, st, lens, sp, mag=False):
    return R.scan(*(c[k].double() for k in ("u", "delta", "A", "B", "C")), d64(o.get("D")),
                  d64(o.get("z")), d64(o.get("dt_bias")), d64(st), lens, sp, mag)


def put_scan(c, o, lens, view):
    rows = ("u", "delta", "z", "B", "C")
    out = []
    for part in (c, o):
        r = {}
        for k, v in part.items():
            if k in rows and lens is not None:
                v = poison(v, lens, 1)
            r[k] = strided(v, *view) if k in rows and view is not None else up(v)
        out.append(r)
    return out


@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("B,T,D,N,G,dtype,sp,opt,lens,view", SCAN)
def test_scan(sdm, B, T, D, N, G, dtype, sp, opt, lens, view, fresh):
    c, o, st, _, _ = scan_case(B, T, D, N, G, dtype, sp, opt)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    cg, og = put_scan(c, o, lens, view)
    stg = st.cuda()
    if fresh:
        stg.fill_(float("nan"))  # not read
    y = torch.full((B, T, D), 77.0, dtype=DT[dtype], device="cuda")
    if view is not None:
        y = strided(y, *view)
    sdm.selective_scan(*cg.values(), **og, state=stg, lens=up(ln), softplus=sp, fresh=fresh, y=y)
    s0 = None if fresh else st
    (ref, end), (mag, mend) = scan_ref(c, o, s0, lens, sp), scan_ref(c, o, s0, lens, sp, True)
    n = 6 * T + 64 + N  # the steps behind a state, softplus, the sum over the states
    R.within(stg, end, mend + 1e-30, n, "state")
    for q, m in enumerate(lens or [T] * B):
        R.within(y[q, :m], ref[q, :m], mag[q, :m], n + 64, "y")
        assert (y[q, m:] == 77.0).all(), "rows behind the sequence are left as they were"


@pytest.mark.parametrize("ends", [False, True])
@pytest.mark.parametrize("B,T,D,N,G,dtype,sp,opt,lens,view", SCAN)
def test_scan_backward(sdm, B, T, D, N, G, dtype, sp, opt, lens, view, ends):
    c, o, st, dy, de = scan_case(B, T, D, N, G, dtype, sp, opt)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    cg, og = put_scan(c, o, lens, view)
    dyg = up(dy if lens is None else poison(dy, lens, 1))
    g = sdm.selective_scan_backward(*cg.values(), dyg, **og, state=up(st) if ends else None,
                                    lens=up(ln), softplus=sp, dstate_end=up(de) if ends else None)
    a = [c[k].double() for k in ("u", "delta", "A", "B", "C")] + [dy.double()] + \
        [d64(o.get(k)) for k in ("D", "z", "dt_bias")] + \
        [st.double() if ends else None, lens, sp, de.double() if ends else None]
    ref, mag = R.scan_bwd(*a), R.scan_bwd(*a, mag=True)
    want = {"du", "ddelta", "dA", "dB", "dC"} | ({"dD", "dz", "ddt_bias"} if opt else set()) | \
        ({"dstate"} if ends else set())
    assert set(g) == want
    n = 12 * T + 200 + N + D // G  # both scans, softplus and gates, the sums
    for k in sorted(want):
        m = n + (B * T if k in ("dA", "dD", "ddt_bias") else 0)
        R.within(g[k], ref[k], mag[k], m, k)


@pytest.mark.parametrize("cuts", [[1] * 5 + [60], [17, 1, 47], [0, 65]])
def test_scan_calls_chain(sdm, cuts):
    """A sequence in several calls, single tokens among them, against one call: the same sums in
    another order."""
    c, o, st, _, _ = scan_case(2, 65, 24, 16, 1, "f32", True, True)
    cg, og = put_scan(c, o, None, None)
    s1, s2 = st.cuda(), st.cuda()
    whole = sdm.selective_scan(*cg.values(), **og, state=s1)
    parts, t = [], 0
    for n in cuts:
        cut = {k: (v if k == "A" else v[:, t:t + n]) for k, v in cg.items()}
        oc = dict(og, z=og["z"][:, t:t + n])
        parts.append(sdm.selective_scan(*cut.values(), **oc, state=s2))
        t += n
    mag, mend = scan_ref(c, o, st, None, True, True)
    R.within(torch.cat(parts, dim=1), whole.double().cpu(), mag, 12 * 65 + 256, "y")
    R.within(s2, s1.double().cpu(), mend, 12 * 65 + 256, "state")


def test_scan_long_is_split_and_matches(sdm):
    """Few channels and many tokens: the tokens are split over the GPU (the workspace shows it)."""
    B, T, D, N = 1, 2500, 40, 16
    c, o, st, _, _ = scan_case(B, T, D, N, 1, "f32", True, True)
    cg, og = put_scan(c, o, None, None)
    stg = st.cuda()
    d = sdm._ScanDims(B, T, D, N, 1, 0, 1, 0)
    assert sdm._lib.sdm_selective_scan_workspace_bytes(d) > 0
    y = sdm.selective_scan(*cg.values(), **og, state=stg)
    (ref, end), (mag, mend) = scan_ref(c, o, st, None, True), scan_ref(c, o, st, None, True, True)
    R.within(stg, end, mend + 1e-30, 6 * T + 128, "state")
    R.within(y, ref, mag, 6 * T + 128, "y")
    # far tighter than the worst case: the errors of the steps do not add up
    assert normwise_rel_err(f64(y), ref.numpy()) < 1e-5


def test_scan_extreme_steps(sdm):
    """Steps of zero keep the state, large ones forget it; a decay of zero integrates."""
    B, T, D, N = 1, 20, 8, 16
    c, o, st, _, _ = scan_case(B, T, D, N, 1, "f32", False, False)
    c["delta"] = torch.zeros(B, T, D)
    c["delta"][:, :, 1] = 200.0
    c["delta"][:, :, 2] = 1.0
    c["A"][2] = 0.0
    cg, og = put_scan(c, o, None, None)
    stg = st.cuda()
    y = sdm.selective_scan(*cg.values(), state=stg, softplus=False)
    (ref, end), (mag, mend) = scan_ref(c, o, st, None, False), scan_ref(c, o, st, None, False, True)
    assert torch.equal(stg[:, 0].cpu(), st[:, 0])
    R.within(stg, end, mend + 1e-30, 6 * T + 64, "state")
    R.within(y, ref, mag + 1e-30, 6 * T + 128, "y")


@pytest.mark.parametrize("B,T,lens", [(3, 37, [37, 20, 0]), (2, 300, [300, 161]), (3, 1, [1, 0, 1])])
def test_scan_infinite_rates_and_masked_tokens(sdm, B, T, lens):
    """A of -inf or of the type's lowest value forgets at every token, and rows behind a sequence
    still leave its state; tokens masked by a delta of -inf or of the lowest value are passed over."""
    D, N, low = 8, 16, torch.finfo(torch.float32).min
    c, o, st, dy, de = scan_case(B, T, D, N, 1, "f32", True, True)
    c["A"][1], c["A"][2], c["A"][3, ::2] = -float("inf"), low, -float("inf")
    c["delta"][:, ::3, 4], c["delta"][:, ::4, 5] = -float("inf"), low
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    cg, og = put_scan(c, o, lens, None)
    stg = st.cuda()
    y = sdm.selective_scan(*cg.values(), **og, state=stg, lens=ln)
    (ref, end), (mag, mend) = scan_ref(c, o, st, lens, True), scan_ref(c, o, st, lens, True, True)
    n = 6 * T + 64 + N
    R.within(stg, end, mend + 1e-30, n, "state")
    R.within(y, ref, mag + 1e-30, n + 64, "y")
    # the gradient's formula has A q: finite for the lowest value, 0 * inf for -inf
    c["A"].clamp_(min=low)
    cg["A"] = c["A"].cuda()
    g = sdm.selective_scan_backward(*cg.values(), poison(dy, lens, 1).cuda(), **og, state=up(st),
                                    lens=ln, dstate_end=up(de))
    a = [c[k].double() for k in ("u", "delta", "A", "B", "C")] + [dy.double()] + \
        [d64(o[k]) for k in ("D", "z", "dt_bias")] + [st.double(), lens, True, de.double()]
    ref, mag = R.scan_bwd(*a), R.scan_bwd(*a, mag=True)
    for k in sorted(ref):
        m = 12 * T + 200 + N + D + (B * T if k in ("dA", "dD", "ddt_bias") else 0)
        R.within(g[k], ref[k], mag[k] + 1e-30, m, k)


def test_scan_outputs_are_reproducible(sdm):
    c, o, st, dy, de = scan_case(2, 300, 200, 16, 2, "bf16", True, True)
    cg, og = put_scan(c, o, None, None)
    runs = []
    for _ in range(2):
        s = st.cuda()
        y = sdm.selective_scan(*cg.values(), **og, state=s)
        g = sdm.selective_scan_backward(*cg.values(), up(dy), **og, state=up(st), dstate_end=up(de))
        runs.append([y, s] + [g[k] for k in sorted(g)])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N", [(20, 16), (90, 16), (90, 5)])
def test_scan_backward_of_sequences_without_tokens(sdm, T, N, dtype):
    """What an empty sequence's state holds, and the gradient that comes to it, are its own: the
    sums over the batch are those of the others.  Behind a sequence every gradient is zero, whatever
    comes to the state at its end."""
    B, D, G, lens = 3, 12, 2, [T, 0, 5]
    c, o, st, dy, de = scan_case(B, T, D, N, G, dtype, True, True)
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    cg, og = put_scan(c, o, lens, None)
    dyg = poison(dy, lens, 1).cuda()

    def run(**kw):
        return sdm.selective_scan_backward(*cg.values(), dyg, **{**og, **kw}, state=up(st), lens=ln,
                                           dstate_end=up(de))
    st[1], de[1] = 0, 0
    want = run()
    for bad in (float("nan"), float("inf")):
        st[1], de[1] = bad, bad
        g = run()
        for k in g:
            if k != "dstate":
                assert torch.equal(g[k], want[k]), (k, bad)
        assert torch.equal(g["dstate"][::2], want["dstate"][::2])
        assert torch.equal(g["dstate"][1].cpu().nan_to_num(7, 8), de[1].nan_to_num(7, 8))
    de[2] = float("inf")
    g = run(D=torch.full((D,), float("inf"), device="cuda"))
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        for q, n in enumerate(lens):
            assert (g[k][q, n:] == 0).all(), k


# ---- block norms ---------------------------------------------------------------------------

NORM = [  # rows, D, r, f, x, (w_post, gate, scale, w_pre)
    (5, 64, "f32", "f32", "f32", (1, 1, 1, 1)),
    (7, 100, "bf16", "f32", "bf16", (1, 1, 1, 1)),
    (300, 256, "f32", "bf16", "bf16", (1, 0, 1, 1)),
    (3, 33, "bf16", "bf16", "bf16", (1, 1, 1, 1)),
    (3, 1, "f32", "f32", "f32", (1, 1, 1, 1)),
    (2, 4096, "bf16", "f32", "bf16", (1, 1, 1, 1)),
    (2, 4100, "f32", "f32", "f32", (0, 1, 0, 1)),
    (2, 8191, "f32", "f32", "bf16", (1, 1, 1, 0)),
    (3, 16384, "bf16", "bf16", "bf16", (1, 1, 1, 1)),
    (2, 16383, "f32", "f32", "f32", (1, 1, 1, 1)),
    (1000, 72, "f32", "f32", "f32", (0, 0, 0, 0)),
    (700, 12, "bf16", "bf16", "f32", (1, 0, 0, 1)),
    (400, 6001, "bf16", "f32", "bf16", (1, 1, 1, 1)),
    (200, 12000, "f32", "bf16", "f32", (1, 1, 1, 1)),
    # more wide rows than blocks
    (700, 4104, "bf16", "f32", "bf16", (1, 1, 1, 1)),
    (650, 4099, "f32", "f32", "f32", (0, 1, 1, 0)),
    (601, 5001, "f32", "bf16", "f32", (1, 1, 1, 1)),
]


def norm_case(rows, D, r, f, x, has, seed=0):
    g = gen(rows + D + seed)
    vec = [torch.rand(D, generator=g) + 0.5 for _ in range(3)]
    opt = {"w_post": vec[0] if has[0] else None,
           "gate": rnd(g, rows, D, dt=DT[x]) if has[1] else None,
           "scale": vec[1] * 0.3 if has[2] else None, "w_pre": vec[2] if has[3] else None}
    return rnd(g, rows, D, dt=DT[r], std=2.0), rnd(g, rows, D, dt=DT[f]), opt, \
        rnd(g, rows, D, dt=DT[r]), rnd(g, rows, D, dt=DT[x])


@pytest.mark.parametrize("rows,D,r,f,x,has", NORM)
def test_norm(sdm, rows, D, r, f, x, has):
    rr, ff, opt, _, _ = norm_case(rows, D, r, f, x, has)
    og = {k: up(v) for k, v in opt.items()}
    o, n = sdm.block_norm(up(rr), up(ff), **og, x_dtype=DT[x])
    ref_o, ref_n = R.norm(rr.double(), ff.double(), **{k: d64(v) for k, v in opt.items()})
    # the block's share: D squares, rsqrt (4), sigmoid (64), products; the sum's cancellation is
    # against the sizes of its two terms, and reaches n through o over its root mean square
    a = rr.double().abs() + (ref_o - rr.double()).abs()
    R.within(o, ref_o, a, D / 2 + 80, "r_out")
    big = a.amax(-1, keepdim=True) / torch.sqrt((ref_o ** 2).mean(-1, keepdim=True) + 1e-6)
    w = 1.0 if opt["w_pre"] is None else opt["w_pre"].double()
    R.within(n, ref_n, (big + 2 * (ref_n / w).abs()) * w * torch.ones_like(ref_n), D + 100, "n")
    # in place, and without n
    r2 = up(rr)
    o2, n2 = sdm.block_norm(r2, up(ff), **og, x_dtype=DT[x], r_out=r2)
    assert o2 is r2 and torch.equal(r2, o) and torch.equal(n2, n)


@pytest.mark.parametrize("zero", [None, "dr_out", "dn"])
@pytest.mark.parametrize("rows,D,r,f,x,has", NORM)
def test_norm_backward(sdm, rows, D, r, f, x, has, zero):
    rr, ff, opt, dro, dn = norm_case(rows, D, r, f, x, has)
    dro, dn = (None if zero == "dr_out" else dro), (None if zero == "dn" else dn)
    g = sdm.block_norm_backward(up(rr), up(ff), up(dro), up(dn), **{k: up(v) for k, v in opt.items()})
    ref, mag = R.norm_bwd(rr.double(), ff.double(), d64(dro), d64(dn),
                          **{k: d64(v) for k, v in opt.items()})
    names = {"dr", "df"} | {n for n, k in (("dgate", "gate"), ("dscale", "scale"),
                                           ("dw_post", "w_post"), ("dw_pre", "w_pre"))
                            if opt[k] is not None}
    assert set(g) == names
    for k in sorted(names):
        m = 4 * D + 300 + (rows if k in ("dscale", "dw_post", "dw_pre") else 0)
        R.within(g[k], ref[k], mag[k] + 1e-30, m, k)


@pytest.mark.parametrize("D", [33, 72, 100, 1000, 4100])
def test_norm_rows_do_not_mix(sdm, D):
    """A row of NaN leaves the rows that the same block takes after it as they are, at widths that
    do not fill the block's threads."""
    rows = 1500
    rr, ff, opt, dro, dn = norm_case(rows, D, "f32", "f32", "f32", (1, 1, 1, 1))
    og = {k: up(v) for k, v in opt.items()}
    for k in ("gate",):
        og[k][:600] = float("nan")
    rg, fg, drog, dng = up(rr), up(ff), up(dro), up(dn)
    want_o, want_n = sdm.block_norm(rg, fg, **og)
    want = sdm.block_norm_backward(rg, fg, drog, dng, **og)
    ref, _ = R.norm_bwd(rr[600:].double(), ff[600:].double(), dro[600:].double(), dn[600:].double(),
                        **{k: (d64(v[600:]) if k == "gate" else d64(v)) for k, v in opt.items()})
    assert want_o[:600].isnan().all() and want_n[:600].isnan().all()
    assert want_o[600:].isfinite().all() and want_n[600:].isfinite().all()
    for k in ("dr", "df", "dgate"):
        assert normwise_rel_err(f64(want[k][600:]), ref[k].numpy()) < 1e-5, k


@pytest.mark.parametrize("back", [False, True])
def test_wide_norms_from_two_host_threads(sdm, back):
    """Calls of different widths from two host threads: a kernel's shared memory is not allowed less
    by one call than the other needs."""
    status = {}

    def calls(D):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        d = sdm._NormDims(1, D, 0, 0, 0, 1e-6)
        r, f, o, n, dr, df = (torch.ones(1, D, device="cuda") for _ in range(6))
        ws = torch.empty(sdm._lib.sdm_block_norm_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        p = [t.data_ptr() for t in (r, f, o, n, dr, df, ws)]
        bad = 0
        for i in range(4000):
            if back:
                bad += sdm._lib.sdm_block_norm_backward(
                    d, p[0], p[1], None, None, None, None, p[2], p[3], p[4], p[5], None, None, None, None,
                    p[6], ws.numel(), s.cuda_stream) != 0
            else:
                bad += sdm._lib.sdm_block_norm(d, p[0], p[1], None, None, None, None, p[2], p[3],
                                               s.cuda_stream) != 0
            if i % 500 == 0:
                s.synchronize()
        s.synchronize()
        status[D] = bad

    threads = [threading.Thread(target=calls, args=(D,)) for D in (16384, 8192)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert status == {16384: 0, 8192: 0}


# ---- as they are used ----------------------------------------------------------------------

def test_block_around_the_scan(sdm):
    """One state-space block: norm -> projection -> convolution -> projection -> scan ->
    projection -> norm with gate and residual, each stage against fp64 from the GPU's previous
    stage; u and z are column slices of one projection."""
    B, T, dm, D, N = 2, 90, 64, 128, 16
    g = gen(42)
    r, f0 = rnd(g, B, T, dm, std=2.0).cuda(), rnd(g, B, T, dm).cuda()
    ones = torch.ones(dm, device="cuda")
    gate = rnd(g, B, T, dm, dt=torch.bfloat16).cuda()
    Win = (rnd(g, 2 * D, dm) / 8).to(torch.bfloat16).cuda()
    Wx = (rnd(g, D + 2 * N, D) / 11).to(torch.bfloat16).cuda()
    Wo = (rnd(g, dm, D) / 11).to(torch.bfloat16).cuda()
    wc, bc = rnd(g, 1, D, 4, std=0.5).cuda(), rnd(g, 1, D, std=0.1).cuda()
    A, Ds = -(torch.rand(D, N, generator=g) * 4 + 0.1).cuda(), rnd(g, D).cuda()
    dtb = (rnd(g, D) - 3).cuda()
    cs = torch.zeros(B, 1, 3, D, dtype=torch.bfloat16, device="cuda")
    hs = torch.zeros(B, D, N, device="cuda")

    r1, n1 = sdm.block_norm(r, f0, w_post=ones, gate=gate, w_pre=ones)
    xz = sdm.gemm_bf16(n1.view(B * T, dm), Win).view(B, T, 2 * D).to(torch.bfloat16)
    u = sdm.short_conv(xz[..., :D].unsqueeze(1), wc, bc, state=cs, fresh=True)[:, 0]
    p = sdm.gemm_bf16(u.reshape(B * T, D), Wx).view(B, T, D + 2 * N).to(torch.bfloat16)
    delta, Bm, Cm = p[..., :D], p[..., D:D + N].unsqueeze(2), p[..., D + N:].unsqueeze(2)
    y = sdm.selective_scan(u, delta, A, Bm, Cm, D=Ds, z=xz[..., D:], dt_bias=dtb, state=hs,
                           fresh=True)
    f1 = sdm.gemm_bf16(y.view(B * T, D), Wo).view(B, T, dm)
    r2, n2 = sdm.block_norm(r1, f1, w_post=ones, gate=gate, w_pre=ones, r_out=r1.clone())
    torch.cuda.synchronize()

    c64 = lambda t: t.detach().double().cpu()  # noqa: E731
    ref_u, ref_cs = R.conv(c64(xz[..., :D]).unsqueeze(1), c64(wc), c64(bc), True, None, None)
    assert normwise_rel_err(f64(u), ref_u[:, 0].numpy()) <= 2.0 ** -8 * 1.01
    assert torch.equal(c64(cs), ref_cs)
    ref_y, ref_h = R.scan(c64(u), c64(delta), c64(A), c64(Bm), c64(Cm), c64(Ds), c64(xz[..., D:]),
                          c64(dtb))
    assert normwise_rel_err(f64(y), ref_y.numpy()) <= 2.0 ** -8 * 1.01
    assert normwise_rel_err(f64(hs), ref_h.numpy()) <= 1e-5
    ref_r, ref_n = R.norm(c64(r1), c64(f1), c64(ones), c64(gate), None, c64(ones))
    assert normwise_rel_err(f64(r2), ref_r.numpy()) <= 1e-5
    assert normwise_rel_err(f64(n2), ref_n.numpy()) <= 2.0 ** -8 * 1.01

    # the next token, from the states the prompt left
    nt = rnd(g, B, 1, 2 * D, dt=torch.bfloat16).cuda()
    u1 = sdm.short_conv(nt[..., :D].unsqueeze(1), wc, bc, state=cs)[:, 0]
    p1 = sdm.gemm_bf16(u1.reshape(B, D), Wx).view(B, 1, D + 2 * N).to(torch.bfloat16)
    y1 = sdm.selective_scan(u1, p1[..., :D], A, p1[..., D:D + N].unsqueeze(2),
                            p1[..., D + N:].unsqueeze(2), D=Ds, z=nt[..., D:], dt_bias=dtb, state=hs)
    ref_u1, _ = R.conv(c64(nt[..., :D]).unsqueeze(1), c64(wc), c64(bc), True, ref_cs, None)
    assert normwise_rel_err(f64(u1), ref_u1[:, 0].numpy()) <= 2.0 ** -8 * 1.01
    ref_y1, ref_h1 = R.scan(c64(u1), c64(p1[..., :D]), c64(A), c64(p1[..., D:D + N]).unsqueeze(2),
                            c64(p1[..., D + N:]).unsqueeze(2), c64(Ds), c64(nt[..., D:]), c64(dtb),
                            ref_h)
    assert normwise_rel_err(f64(y1), ref_y1.numpy()) <= 2.0 ** -8 * 1.01
    assert normwise_rel_err(f64(hs), ref_h1.numpy()) <= 1e-5


def test_convolutions_and_norm_around_a_memory_layer(sdm):
    """layer_in -> short convolutions of q, k and v -> prefill -> layer_out -> block norm, whose n
    is the next layer's input."""
    B, H, T, dk, dv, n, k = 1, 2, 80, 128, 64, 16, 8
    dm = 64
    g = gen(9)
    d = sdm.Dims(B, H, T, dk, n, dv, k, 8, 8, "bf16", "bf16")
    x = rnd(g, B, T, dm, dt=torch.bfloat16).cuda()
    Win = (rnd(g, H * (2 * dk + 2 * dv + 2), dm) / 8).to(torch.bfloat16).cuda()
    p = sdm.layer_in(d, x, Win, rnd(g, H).cuda(), rnd(g, H).cuda())
    conv = {}
    for name, w in (("q", dk), ("k", dk), ("v", dv)):
        wt = rnd(g, H, w, 4, std=0.5).cuda()
        conv[name] = sdm.short_conv(p[name], wt)
        ref, _ = R.conv(p[name].double().cpu(), wt.double().cpu(), None, True, None, None)
        assert normwise_rel_err(f64(conv[name]), ref.numpy()) <= 2.0 ** -8 * 1.01
    skw = (rnd(g, H, 2, n, dk // 2) / 8).to(torch.bfloat16).cuda()
    st = sdm.State(d, (rnd(g, H, n * n, dv) * 0.02).cuda())
    sdm.state_reset(d, st)
    o, (widx, ww, ridx, rw) = sdm.prefill(d, conv["q"], conv["k"], conv["v"], p["alpha"], p["beta"],
                                          skw, skw, st)
    wn, Wo = torch.ones(dv, device="cuda"), (rnd(g, dm, H * dv) / 11).to(torch.bfloat16).cuda()
    f = sdm.layer_out(d, o, p["g"], wn, Wo)
    ones = torch.ones(dm, device="cuda")
    res, nxt = sdm.block_norm(x, f, w_post=ones, w_pre=ones)
    torch.cuda.synchronize()
    orc = oracle.default()
    for h in range(H):
        s = orc.fresh_lazy_state(f64(st.M0[h]))
        ref = orc.recur_lazy(f64(conv["v"][0, h]), f64(p["alpha"][0, h]), f64(p["beta"][0, h]),
                             widx[0, h].cpu().numpy(), f64(ww[0, h]), ridx[0, h].cpu().numpy(),
                             f64(rw[0, h]), s)
        assert normwise_rel_err(f64(o[0, h]), ref) <= 2e-2
    ref_r, ref_n = R.norm(x.double().cpu(), f.double().cpu(), ones.double().cpu(), None, None,
                          ones.double().cpu())
    assert normwise_rel_err(f64(res), ref_r.numpy()) <= 2.0 ** -8 * 1.01
    assert normwise_rel_err(f64(nxt), ref_n.numpy()) <= 2.0 ** -8 * 1.01
    assert nxt.dtype == torch.bfloat16 and sdm.layer_in(d, nxt, Win, rnd(g, H).cuda(),
                                                        rnd(g, H).cuda())["q"].isfinite().all()
    assert sdm.device_error() == 0


def test_streams_and_graphs(sdm):
    """On a side stream, and captured: two graphs with workspaces of their own, replayed in turn,
    give the eager results; decode steps in a graph move the states on in place."""
    c, o, st, dy, _ = scan_case(1, 600, 40, 16, 1, "f32", True, True)
    cg, og = put_scan(c, o, None, None)
    x, w, b, cst, cdy, _, _ = conv_case(1, 2, 30, 16, 4, "f32", "silu", True, None)
    rr, ff, opt, dro, dn = norm_case(50, 5000, "f32", "f32", "f32", (1, 1, 1, 1))
    xg, wg, bg, cdyg, dyg = up(x), up(w), up(b), up(cdy), up(dy)
    rg, fg, drog, dng = up(rr), up(ff), up(dro), up(dn)
    optg = {k: up(v) for k, v in opt.items()}

    def everything(hs, cs):
        out = [sdm.selective_scan(*cg.values(), **og, state=hs),
               sdm.short_conv(xg, wg, bg, state=cs), *sdm.block_norm(rg, fg, **optg)]
        for d in (sdm.selective_scan_backward(*cg.values(), dyg, **og),
                  sdm.short_conv_backward(xg, wg, cdyg, bg),
                  sdm.block_norm_backward(rg, fg, drog, dng, **optg)):
            out += [d[k] for k in sorted(d)]
        return out + [hs, cs]

    want = everything(st.cuda(), cst.cuda())
    side = torch.cuda.Stream()
    hs, cs = st.cuda(), cst.cuda()
    side.wait_stream(torch.cuda.current_stream())
    y = sdm.selective_scan(*cg.values(), **og, state=hs, stream=side)
    yc = sdm.short_conv(xg, wg, bg, state=cs, stream=side)
    no, nn = sdm.block_norm(rg, fg, **optg, stream=side)
    back = [sdm.selective_scan_backward(*cg.values(), dyg, **og, stream=side),
            sdm.short_conv_backward(xg, wg, cdyg, bg, stream=side),
            sdm.block_norm_backward(rg, fg, drog, dng, **optg, stream=side)]
    side.synchronize()
    got = [y, yc, no, nn] + [d[k] for d in back for k in sorted(d)] + [hs, cs]
    assert len(got) == len(want) and all(torch.equal(a, b2) for a, b2 in zip(got, want))

    states = [(st.cuda(), cst.cuda()) for _ in range(2)]
    graphs, outs = [], []
    for s in states:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(everything(*s))
        graphs.append(gr)
    for gr in graphs + graphs[:1]:
        for a, b2 in states:
            a.copy_(st), b2.copy_(cst)
        gr.replay()
    torch.cuda.synchronize()
    for s, got in ((states[0], outs[0]),):
        assert all(torch.equal(a, b2) for a, b2 in zip(got, want))
    for t in outs[1][:-2]:
        t.fill_(0)
    for a, b2 in states:
        a.copy_(st), b2.copy_(cst)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b2) for a, b2 in zip(outs[1], want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 90])
def test_layouts(sdm, T, dtype):
    """Token-major and sequence-minor views, and inputs that are broadcast over sequences, heads or
    tokens, give what contiguous copies give; gradients of broadcast inputs are of the whole view."""
    g, dt, B, H, d, D, G, N = gen(5), DT[dtype], 3, 2, 8, 24, 2, 16
    w = rnd(g, H, d, 4).cuda()
    A = -(torch.rand(D, N, generator=g) + 0.1).cuda()

    def same(f, views):
        got, want = f(*views), f(*(v.contiguous() for v in views))
        for a, b in zip(*((r if isinstance(r, tuple) else [r[k] for k in sorted(r)])
                          for r in (got, want))):
            assert torch.equal(a, b)

    def conv(x, dy):
        st = torch.ones(B, H, 3, d, dtype=dt, device="cuda")
        return sdm.short_conv(x, w, state=st), st, *sdm.short_conv_backward(x, w, dy).values()

    def scan(u, de, Bm, Cm, dy):
        h = torch.ones(B, D, N, device="cuda")
        y = sdm.selective_scan(u, de, A, Bm, Cm, z=u, state=h)
        r = sdm.selective_scan_backward(u, de, A, Bm, Cm, dy, z=u)
        return y, h, *(r[k] for k in sorted(r))

    x = rnd(g, B, T, H, d, dt=dt).cuda().transpose(1, 2)
    xs = rnd(g, H, T, B, d, dt=dt).cuda().permute(2, 0, 1, 3)
    for views in ((x, xs), (xs, x), (x[:1].expand(B, H, T, d), xs[:, :1].expand(B, H, T, d)),
                  (x[:, :, :1].expand(B, H, T, d), x)):
        same(conv, views)
    u = rnd(g, T, B, D, dt=dt).cuda().transpose(0, 1)
    de = rnd(g, 1, T, D, dt=dt).cuda().expand(B, T, D)
    Bm = rnd(g, B, G, T, N, dt=dt).cuda().transpose(1, 2)
    Cm = rnd(g, 1, T, 1, N, dt=dt).cuda().expand(B, T, G, N)
    same(scan, (u, de, Bm, Cm, de))
    same(scan, (de, u, Cm, Bm, u[:, :1].expand(B, T, D)))


def test_lengths_are_clamped(sdm):
    """Lengths below zero and beyond the call are taken as 0 and T."""
    B, T = 3, 20
    raw, ln = (torch.tensor(v, dtype=torch.int32, device="cuda")
               for v in ([-7, T + 5, 1 << 30], [0, T, T]))
    c, o, st, dy, _ = scan_case(B, T, 12, 16, 1, "f32", True, True)
    cg, og = put_scan(c, o, None, None)
    x, w, b, cst, cdy, _, _ = conv_case(B, 2, T, 16, 4, "f32", "silu", True, None)
    out = []
    for v in (raw, ln):
        h, s = st.cuda(), cst.cuda()
        r = [sdm.selective_scan(*cg.values(), **og, state=h, lens=v), h,
             sdm.short_conv(up(x), up(w), up(b), state=s, lens=v), s]
        for q in (sdm.selective_scan_backward(*cg.values(), up(dy), **og, lens=v),
                  sdm.short_conv_backward(up(x), up(w), up(cdy), up(b), lens=v)):
            r += [q[k] for k in sorted(q)]
        t = [a[:, :1].contiguous() for a in (cg["u"], cg["delta"], cg["B"], cg["C"])]
        r.append(sdm.selective_scan(t[0], t[1], cg["A"], *t[2:], state=h, lens=v))
        out.append(r + [h])
    assert all(torch.equal(a, b2) for a, b2 in zip(*out))


def test_long_offsets(sdm):
    """Offsets beyond 2^31 elements: two sequences far apart in one buffer, and a state behind
    them."""
    far = (1 << 31) + 64
    buf = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda")
    g = gen(3)
    x = rnd(g, 2, 1, 20, 32, dt=torch.bfloat16).cuda()
    xv = buf.as_strided((2, 1, 20, 32), (far, 32, 32, 1))
    xv.copy_(x)
    w = rnd(g, 1, 32, 4).cuda()
    yv = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda").as_strided(
        (2, 1, 20, 32), (far, 32, 32, 1))
    sdm.short_conv(xv, w, y=yv)
    assert torch.equal(yv, sdm.short_conv(x, w))
    A = -(torch.rand(32, 16, generator=g) + 0.1).cuda()
    Bm, Cm = (rnd(g, 2, 20, 1, 16, dt=torch.bfloat16).cuda() for _ in range(2))
    u = x[:, 0].contiguous()
    want = sdm.selective_scan(u, u, A, Bm, Cm)
    sdm.selective_scan(xv[:, 0], xv[:, 0], A, Bm, Cm, y=yv[:, 0])
    assert torch.equal(yv[:, 0], want)


# ---- refusals of the binding ---------------------------------------------------------------

def test_binding_refuses(sdm):
    x, w, b, st, dy, _, _ = (v.cuda() if isinstance(v, torch.Tensor) else v for v in
                             conv_case(2, 2, 8, 16, 4, "bf16", "silu", True, None))
    bad = [lambda: sdm.short_conv(x.cpu(), w), lambda: sdm.short_conv(x.half(), w),
           lambda: sdm.short_conv(x, w.double()), lambda: sdm.short_conv(x, w[:, :8].contiguous()),
           lambda: sdm.short_conv(x, w, state=st.float()),
           lambda: sdm.short_conv(x, w, state=st[:1].contiguous()),
           lambda: sdm.short_conv(x, w, lens=torch.ones(2, dtype=torch.int64, device="cuda")),
           lambda: sdm.short_conv(x[..., ::2], w[:, ::2].contiguous()),
           lambda: sdm.short_conv(x, w, y=x), lambda: sdm.short_conv(x, w, y=x.clone()[:, :1].expand(2, 2, 8, 16)),
           lambda: sdm.short_conv(x, torch.zeros(2, 16, 9, device="cuda")),
           lambda: sdm.short_conv(x, w, act="relu"),
           lambda: sdm.short_conv_backward(x, w, dy.float())]
    for f in bad:
        with pytest.raises((TypeError, ValueError, KeyError, sdm.SdmError)):
            f()
    c, o, s, dy2, _ = scan_case(2, 10, 12, 16, 2, "f32", True, True)
    (cg, og), s = put_scan(c, o, None, None), s.cuda()
    a = list(cg.values())
    bad = [lambda: sdm.selective_scan(a[0], a[1][:, :5], *a[2:]),
           lambda: sdm.selective_scan(*a[:3], a[3][:, :, :1], a[4]),
           lambda: sdm.selective_scan(*a, state=s[:, :, :8].contiguous()),
           lambda: sdm.selective_scan(*a, z=og["z"].bfloat16()),
           lambda: sdm.selective_scan(*a, y=a[0]),
           lambda: sdm.selective_scan(a[0], a[1], torch.zeros(12, 65, device="cuda"),
                                      *(torch.zeros(2, 10, 2, 65, device="cuda") for _ in range(2))),
           lambda: sdm.selective_scan(*a[:3], *(torch.zeros(2, 10, 5, 16, device="cuda") for _ in range(2))),
           lambda: sdm.selective_scan_backward(*a, dy2.cuda(),
                                               ws=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for f in bad:
        with pytest.raises((TypeError, ValueError, sdm.SdmError)):
            f()
    r = torch.zeros(4, 16, device="cuda")
    bad = [lambda: sdm.block_norm(r, r[:2]), lambda: sdm.block_norm(r, r, gate=r.half()),
           lambda: sdm.block_norm(r, r, w_post=torch.ones(8, device="cuda")),
           lambda: sdm.block_norm(r, r, eps=-1.0), lambda: sdm.block_norm(r, r, eps=float("nan")),
           lambda: sdm.block_norm(*(torch.zeros(1, 16388, device="cuda") for _ in range(2))),
           lambda: sdm.block_norm_backward(r, r, None, None)]
    for f in bad:
        with pytest.raises((TypeError, ValueError, sdm.SdmError)):
            f()


def test_norm_refuses_scalars(sdm):
    """A tensor without dimensions has no last one: it is no row of one value, nor an empty call."""
    s, m = torch.ones((), device="cuda"), torch.ones(2, 1, device="cuda")
    for f in (lambda: sdm.block_norm(s, s), lambda: sdm.block_norm(s, m), lambda: sdm.block_norm(m, s),
              lambda: sdm.block_norm_backward(s, s, s, None)):
        with pytest.raises(ValueError):
            f()


def test_binding_refuses_sizes_beyond_its_fields(sdm):
    """2^32 + 4 tokens or columns are not taken for 4."""
    big, z = (1 << 32) + 4, torch.zeros(1, device="cuda")
    x, w = z.expand(1, 1, big, 4), z.expand(1, 4, 4).contiguous()
    u, A, Bm = z.expand(1, big, 4), z.expand(4, 16).contiguous(), z.expand(1, big, 1, 16)
    r = z.expand(2, big)
    for f in (lambda: sdm.short_conv(x, w), lambda: sdm.short_conv_backward(x, w, x),
              lambda: sdm.selective_scan(u, u, A, Bm, Bm),
              lambda: sdm.selective_scan_backward(u, u, A, Bm, Bm, u),
              lambda: sdm.block_norm(r, r), lambda: sdm.block_norm_backward(r, r, r, None)):
        with pytest.raises(ValueError, match="too large"):
            f()


def test_empty_calls(sdm):
    """No tokens: states stay (or start at zero when fresh), gradients pass through."""
    w, st = torch.ones(1, 8, 4, device="cuda"), torch.ones(2, 1, 3, 8, device="cuda")
    x = torch.zeros(2, 1, 0, 8, device="cuda")
    assert sdm.short_conv(x, w, state=st).shape == x.shape and (st == 1).all()
    g = sdm.short_conv_backward(x, w, x, state=st, dstate_end=st * 3)
    assert (g["dstate"] == 3).all() and (g["dw"] == 0).all()
    sdm.short_conv(x, w, state=st, fresh=True)
    assert (st == 0).all()
    u, A = torch.zeros(2, 0, 8, device="cuda"), -torch.ones(8, 16, device="cuda")
    B, h = torch.zeros(2, 0, 1, 16, device="cuda"), torch.ones(2, 8, 16, device="cuda")
    sdm.selective_scan(u, u, A, B, B, state=h)
    assert (h == 1).all()
    g = sdm.selective_scan_backward(u, u, A, B, B, u, state=h, dstate_end=h * 2)
    assert (g["dstate"] == 2).all() and (g["dA"] == 0).all()
    sdm.selective_scan(u, u, A, B, B, state=h, fresh=True)
    assert (h == 0).all()
    r = torch.zeros(0, 16, device="cuda")
    o, n = sdm.block_norm(r, r)
    assert o.shape == (0, 16) == tuple(n.shape)
    g = sdm.block_norm_backward(r, r, r, None, scale=torch.ones(16, device="cuda"))
    assert (g["dscale"] == 0).all()
