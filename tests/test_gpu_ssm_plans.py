"""The state-space block at sizes that take the kernels' longer paths, as real prompts do: rings and
stages that are filled again, several runs, chunks and channel tiles a warp, several rows a block.
The sizes are the smallest that the launch rules give these plans; what a workspace shows of a plan is
checked.

Besides the bounds of tests/ssm_reference.py element by element, which grow with the number of
tokens, whole tensors are compared: |got - ref| <= rel |ref|.  For bf16 rel is the half step of its
rounding, 2^-8, and a hundredth.  For fp32 it is 2e-5 for values and 5e-5 for gradients (U = 2^-24):
  - a term carries the 64 U (value) or 128 U (gradient: two of them) of its activations against its
    size without signs, some three times the signed one: 1.2e-5, 2.4e-5 in two;
  - a scan's contribution of age n carries 6 n roundings of either sign, and ages beyond 200 count for
    little at the rates drawn here: 6 * 200^0.5 U = 5e-6, twice in a gradient;
  - a sum over the tokens is made of runs of some hundred, of either sign: 100^0.5 U."""
from __future__ import annotations

import pytest
import torch

from tests import ssm_reference as R
from tests.test_gpu_ssm import (DT, conv_case, d64, gen, norm_case, poison, put_scan, scan_case, scan_ref,
                                sdm, up)  # noqa: F401 (sdm: the fixture)

pytestmark = pytest.mark.gpu

REL = {torch.bfloat16: 2.0 ** -8 * 1.01}


def close(got, ref, what, rel=2e-5):
    rel = REL.get(got.dtype, rel)
    e = R.off(got, ref)
    assert e <= rel, f"{what}: {e:.3g} of its size off, at most {rel:.3g}"


def near(got, ref, mag, roundings, what):
    """R.within where the tensors lie."""
    step = torch.finfo(got.dtype).eps / 2
    tol = roundings * R.U * mag * (1 + step) + step * ref.abs() + 1e-37
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off"


# ---- short convolution ---------------------------------------------------------------------

CONV = [  # B, H, T, d, K, dtype, act, lens
    # runs of 32 tokens, eight groups through a ring of four
    (8, 16, 900, 128, 4, "bf16", "silu", None),
    (8, 16, 900, 128, 8, "f32", "silu", None),
    # runs of 12, as many as the ring holds; the gradient in two runs of 16 a warp
    (4, 16, 750, 128, 4, "bf16", "silu", None),
    (4, 16, 750, 128, 3, "f32", None, [750, 3, 0, 400]),
    # single channels: runs of 16 and more, the gradient in two runs a warp
    (5, 1, 900, 1001, 4, "bf16", "silu", None),
    (5, 1, 900, 1001, 4, "f32", "silu", [900, 1, 500, 0, 333]),
    # the gradient in two runs of 128 a warp, sequences that end within the runs
    (8, 16, 2400, 128, 4, "bf16", "silu", [2400, 2399, 0, 130, 2400, 1024, 2400, 7]),
]


@pytest.mark.parametrize("B,H,T,d,K,dtype,act,lens", CONV)
def test_conv_of_long_runs(sdm, B, H, T, d, K, dtype, act, lens):
    x, w, b, st, dy, de, _ = conv_case(B, H, T, d, K, dtype, act, True, lens)
    w, b, st, de = up(w), up(b), up(st), up(de)
    xg, dyg = (up(v if lens is None else poison(v, lens, 2)) for v in (x, dy))
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    ref, mag = R.conv_all(up(x).double(), w.double(), b.double(), act, st.double(), lens, up(dy).double(),
                          de.double())
    sg, y = st.clone(), torch.full((B, H, T, d), 77.0, dtype=DT[dtype], device="cuda")
    sdm.short_conv(xg, w, b, act=act, state=sg, lens=ln, y=y)
    for q, m in enumerate(lens or []):
        assert (y[q, :, m:] == 77.0).all()
        y[q, :, m:] = 0
    near(y, ref["y"], mag["y"], K + 1 + (64 if act else 0), "y")
    close(y, ref["y"], "y")
    assert torch.equal(sg.double(), ref["state"])
    g = sdm.short_conv_backward(xg, w, dyg, b, act=act, state=st, lens=ln, dstate_end=de)
    n = 2 * K + 2 + (128 if act else 0)
    for k in ("dx", "dw", "dbias", "dstate"):
        near(g[k], ref[k], mag[k], n + (B * T if k in ("dw", "dbias") else 0), k)
        close(g[k], ref[k], k, 5e-5)


def test_conv_in_runs_of_128_equals_short_calls(sdm):
    """Runs of 128 tokens give bit for bit what calls of at most 512 tokens give, which take runs of
    12 and less."""
    x, w, b, st, _, _, _ = conv_case(8, 16, 7500, 64, 4, "bf16", "silu", True, None)
    x, w, b, s1, s2 = up(x), up(w), up(b), up(st), up(st)
    whole = sdm.short_conv(x, w, b, state=s1)
    t = 0
    for n in [512, 1, 511, 2, 77] + 14 * [457]:
        part = x[:, :, t:t + n]
        if part.shape[2]:
            assert torch.equal(sdm.short_conv(part, w, b, state=s2), whole[:, :, t:t + n]), t
        t += n
    assert t >= x.shape[2] and torch.equal(s1, s2)


# ---- selective scan ------------------------------------------------------------------------

SCAN = [  # B, T, D, N, G, dtype, lens, split over time
    # four states a lane
    (4, 400, 640, 16, 1, "bf16", None, False),
    (4, 400, 640, 16, 1, "f32", [400, 0, 77, 161], False),
    (4, 400, 641, 16, 1, "bf16", [400, 399, 0, 33], False),       # rows at odd addresses
    # eight; in the gradient two channel tiles a warp and walks over two chunks
    (4, 200, 2400, 16, 1, "bf16", [200, 0, 77, 161], False),
    (4, 200, 2400, 16, 1, "f32", None, False),
    (4, 200, 2401, 16, 1, "bf16", None, False),
    (2, 200, 2400, 32, 2, "bf16", None, False),
    (4, 200, 600, 64, 1, "f32", None, False),
    (4, 200, 4800, 8, 1, "bf16", None, False),
    # chunks of twelve tiles
    (2, 1500, 1000, 16, 1, "f32", [1500, 700], True),
    (2, 1500, 1000, 16, 1, "bf16", None, True),
    (2, 1500, 1001, 16, 1, "bf16", [1111, 1500], True),
]


@pytest.mark.parametrize("B,T,D,N,G,dtype,lens,split", SCAN)
def test_scan_of_many_tiles(sdm, B, T, D, N, G, dtype, lens, split):
    c, o, st, _, _ = scan_case(B, T, D, N, G, dtype, True, True)
    xdt = 1 if dtype == "bf16" else 0
    ws = sdm._lib.sdm_selective_scan_workspace_bytes(sdm._ScanDims(B, T, D, N, G, xdt, 1, 0))
    # a chunk leaves a state; a ring has at most six stages of 16 tokens or four of 32
    assert (0 < ws < T * B * D * N * 4 / (6 * 16)) if split else (ws == 0 and T > 4 * 32), "another plan"
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    cg, og = put_scan(c, o, lens, None)
    sg, y = st.cuda(), torch.full((B, T, D), 77.0, dtype=DT[dtype], device="cuda")
    sdm.selective_scan(*cg.values(), **og, state=sg, lens=ln, y=y)
    for q, m in enumerate(lens or []):
        assert (y[q, m:] == 77.0).all()
        y[q, m:] = 0
    (ref, end), (mag, mend) = scan_ref(c, o, st, lens, True), scan_ref(c, o, st, lens, True, True)
    n = 6 * T + 64 + N
    R.within(sg, end, mend + 1e-30, n, "state")
    R.within(y, ref, mag, n + 64, "y")
    close(sg, end, "state")
    close(y, ref, "y")


@pytest.mark.parametrize("B,T,D,N,G,dtype,lens,split", SCAN)
def test_scan_backward_of_many_tiles(sdm, B, T, D, N, G, dtype, lens, split):
    c, o, st, dy, de = scan_case(B, T, D, N, G, dtype, True, True)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    cg, og = put_scan(c, o, lens, None)
    dyg = up(dy if lens is None else poison(dy, lens, 1))
    g = sdm.selective_scan_backward(*cg.values(), dyg, **og, state=up(st), lens=ln, dstate_end=up(de))
    a = [c[k].double() for k in ("u", "delta", "A", "B", "C")] + [dy.double()] + \
        [d64(o[k]) for k in ("D", "z", "dt_bias")] + [st.double(), lens, True, de.double()]
    ref, mag = R.scan_bwd(*a), R.scan_bwd(*a, mag=True)
    assert set(g) == set(ref)
    for k in sorted(ref):
        n = 12 * T + 200 + N + D // G + (B * T if k in ("dA", "dD", "ddt_bias") else 0)
        R.within(g[k], ref[k], mag[k] + 1e-30, n, k)
        close(g[k], ref[k], k, 5e-5)


# ---- block norms ---------------------------------------------------------------------------

def norm_refs(rr, ff, opt, dro, dn, eps):
    o64 = {k: d64(v) for k, v in opt.items()}
    return R.norm(rr.double(), ff.double(), **o64, eps=eps), \
        R.norm_bwd(rr.double(), ff.double(), d64(dro), d64(dn), **o64, eps=eps)[0]


def check_norm(sdm, rr, ff, opt, dro, dn, eps=1e-6):
    a = {k: up(v) for k, v in opt.items()}
    o, n = sdm.block_norm(up(rr), up(ff), **a, x_dtype=dn.dtype, eps=eps)
    g = sdm.block_norm_backward(up(rr), up(ff), up(dro), up(dn), **a, eps=eps)
    (ro, rn), ref = norm_refs(rr, ff, opt, dro, dn, eps)
    close(o, ro, "r_out")
    close(n, rn, "n")
    for k in g:
        close(g[k], ref[k], k, 5e-5)


@pytest.mark.parametrize("has", [(1, 1, 1, 1), (1, 0, 1, 1), (0, 1, 0, 0)])
@pytest.mark.parametrize("rows,D,r,f,x", [
    # more rows than blocks: four and eight a block of 512 threads
    (1300, 4096, "bf16", "bf16", "bf16"), (1300, 4096, "f32", "bf16", "bf16"), (700, 2560, "f32", "f32", "f32"),
    # up to sixteen blocks an SM
    (5000, 72, "bf16", "bf16", "bf16"), (5000, 33, "bf16", "bf16", "bf16"), (5000, 100, "f32", "f32", "bf16"),
    (3000, 1000, "bf16", "f32", "bf16"), (3000, 1001, "bf16", "bf16", "bf16"),
    # wide
    (1300, 4100, "bf16", "bf16", "bf16"), (3, 16384, "bf16", "bf16", "bf16"), (2, 16383, "f32", "f32", "f32"),
    (2, 8191, "f32", "f32", "bf16"), (300, 12000, "f32", "f32", "f32"), (500, 9001, "bf16", "bf16", "bf16"),
])
def test_norm_of_many_rows_and_gradients_along_them(sdm, rows, D, r, f, x, has):
    check_norm(sdm, *R.along(rows, D, DT[r], DT[f], DT[x], has, gen(rows + D)))


@pytest.mark.parametrize("eps", [0.1, 3e-3])
@pytest.mark.parametrize("D", [64, 33, 4096, 4100, 5001, 16384])
def test_norm_uses_its_eps(sdm, D, eps):
    """Rows of the size of eps's root, one of them zero (its o^ and f^ are zero, its gradients not)."""
    rr, ff, opt, dro, dn = R.along(40, D, *3 * (torch.float32,), (1, 1, 1, 1), gen(D), eps, eps ** 0.5)
    rr[7] = ff[7] = 0
    check_norm(sdm, rr, ff, opt, dro, dn, eps)
    _, ref = norm_refs(rr, ff, opt, dro, dn, eps)
    assert R.off(norm_refs(rr, ff, opt, dro, dn, 1e-6)[1]["dr"][:7], ref["dr"][:7]) > 0.05
    g = sdm.block_norm_backward(up(rr[7:8]), up(ff[7:8]), up(dro[7:8]), up(dn[7:8]),
                                **{k: up(v[7:8] if k == "gate" else v) for k, v in opt.items()}, eps=eps)
    for k in ("dr", "df"):
        close(g[k], ref[k][7:8], k, 5e-5)


@pytest.mark.parametrize("D", [33, 72, 100, 1000, 4100])
def test_norm_rows_of_a_block_do_not_mix(sdm, D):
    """A row of NaN leaves the rows that the same block takes after it as they are: 5000 rows are more
    than two a block at every width."""
    rr, ff, opt, dro, dn = norm_case(5000, D, "f32", "f32", "f32", (1, 1, 1, 1))
    bad = {k: (v.clone() if k == "gate" else v) for k, v in opt.items()}
    bad["gate"][:2500] = float("nan")
    rg, fg, drog, dng = up(rr), up(ff), up(dro), up(dn)
    got, want = ([*sdm.block_norm(rg, fg, **a), *(sdm.block_norm_backward(rg, fg, drog, dng, **a)[k]
                                                  for k in ("dr", "df", "dgate"))]
                 for a in ({k: up(v) for k, v in q.items()} for q in (bad, opt)))
    for a, b in zip(got, want):
        assert a[:2500].isnan().all() and torch.equal(a[2500:], b[2500:])


# ---- calls that start their sequences ---------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [20, 150])
def test_backward_of_fresh_calls(sdm, T, dtype):
    """fresh: the state's contents are not read, and its gradient is that of a start at zero."""
    x, w, b, st, dy, de, _ = conv_case(2, 2, T, 16, 4, dtype, "silu", True, None)
    a = (up(x), up(w), up(dy), up(b))
    got = sdm.short_conv_backward(*a, state=up(st).fill_(float("nan")), fresh=True, dstate_end=up(de))
    want = sdm.short_conv_backward(*a, state=up(st).zero_(), dstate_end=up(de))
    assert got.keys() == want.keys() and all(torch.equal(got[k], want[k]) for k in want)
    c, o, st, dy, de = scan_case(2, T, 24, 16, 1, dtype, True, True)
    cg, og = put_scan(c, o, None, None)
    f = lambda s, fresh: sdm.selective_scan_backward(*cg.values(), up(dy), **og, state=s, fresh=fresh,  # noqa: E731
                                                     dstate_end=up(de))
    got, want = f(up(st).fill_(float("nan")), True), f(up(st).zero_(), False)
    assert got.keys() == want.keys() and all(torch.equal(got[k], want[k]) for k in want)


# ---- the ends of the ranges ------------------------------------------------------------------

@pytest.mark.parametrize("B,H,T,d,dtype,cut", [
    (65535, 1, 1100, 4, "bf16", 7),        # runs as long as the grid's second axis asks for
    (2, 3, 45, 100001, "bf16", 1),         # more columns of blocks than the gradient wants blocks
    (3, 1, 70, 80000, "f32", 2),
    (1, 1, 5_000_001, 4, "bf16", None),
])
def test_conv_of_many_sequences_channels_or_tokens(sdm, B, H, T, d, dtype, cut):
    """The batch's parts give bit for bit what the whole gives, and the filters' gradients add up."""
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *n, dt=torch.float32: torch.randn(n, generator=g, device="cuda").to(dt)  # noqa: E731
    x, dy = r(B, H, T, d, dt=DT[dtype]), r(B, H, T, d, dt=DT[dtype])
    w, st = r(H, d, 4), r(B, H, 3, d, dt=DT[dtype])
    s1, s2 = st.clone(), st.clone()
    y, got = sdm.short_conv(x, w, state=s1), sdm.short_conv_backward(x, w, dy, state=st)
    if cut is None:  # tokens instead of sequences
        t = T // 3
        parts = [sdm.short_conv(v, w, state=s2) for v in (x[:, :, :t], x[:, :, t:])]
        assert torch.equal(torch.cat(parts, 2), y) and torch.equal(s1, s2)
        for a in (0, T - 2000):  # dx of the last tokens of a part needs the tokens behind it
            before = st if a == 0 else x[:, :, a - 3:a]
            p, q = (v[:, :, a:a + 2000].double() for v in (x, dy))
            ref, mag = R.conv_all(p, w.double(), None, True, before.double(), None, q, torch.zeros_like(st).double())
            n = 2000 if a else 1997
            near(got["dx"][:, :, a:a + n], ref["dx"][:, :, :n], mag["dx"][:, :, :n], 2 * 4 + 2 + 128, "dx")
        return
    s2 = [s2[:cut].clone(), s2[cut:].clone()]  # starts at 16 bytes
    cuts = ((0, cut), (cut, B))
    parts = [sdm.short_conv(x[a:b], w, state=v) for (a, b), v in zip(cuts, s2)]
    assert torch.equal(torch.cat(parts), y) and torch.equal(s1, torch.cat(s2))
    p = [sdm.short_conv_backward(x[a:b], w, dy[a:b], state=st[a:b].clone()) for a, b in cuts]
    for k in ("dx", "dstate"):
        assert torch.equal(torch.cat([v[k] for v in p]), got[k])
    close(got["dw"], p[0]["dw"].double() + p[1]["dw"].double(), "dw", 5e-5)


@pytest.mark.parametrize("B,T,D,N,G,dtype", [
    (65535, 3, 4, 8, 1, "bf16"), (65535, 1, 4, 8, 1, "f32"), (2, 90, 300, 16, 300, "bf16"),
    (3, 40, 21000, 1, 21000, "f32"), (3, 100, 70001, 3, 1, "bf16"),
])
def test_scan_of_many_sequences_groups_or_channels(sdm, B, T, D, N, G, dtype):
    g = torch.Generator("cuda").manual_seed(2)
    r = lambda *n, dt=DT[dtype]: torch.randn(n, generator=g, device="cuda").to(dt)  # noqa: E731
    u, de, z, dy, Bm, Cm = r(B, T, D), r(B, T, D), r(B, T, D), r(B, T, D), r(B, T, G, N), r(B, T, G, N)
    A, st = -torch.rand(D, N, generator=g, device="cuda") - 0.05, r(B, D, N, dt=torch.float32)
    s1, s2 = st.clone(), st.clone()
    y = sdm.selective_scan(u, de, A, Bm, Cm, z=z, state=s1)
    got = sdm.selective_scan_backward(u, de, A, Bm, Cm, dy, z=z, state=st)
    c = B // 2
    cuts = ((0, c), (c, B))
    s2 = [s2[:c].clone(), s2[c:].clone()]  # starts at 16 bytes
    parts = [sdm.selective_scan(u[a:b], de[a:b], A, Bm[a:b], Cm[a:b], z=z[a:b], state=v)
             for (a, b), v in zip(cuts, s2)]
    back = [sdm.selective_scan_backward(u[a:b], de[a:b], A, Bm[a:b], Cm[a:b], dy[a:b], z=z[a:b],
                                        state=st[a:b].clone()) for a, b in cuts]
    close(torch.cat(parts), y.double(), "y")
    close(torch.cat(s2), s1.double(), "state")
    for k in ("du", "ddelta", "dz", "dB", "dC", "dstate"):
        close(torch.cat([v[k] for v in back]), got[k].double(), k, 5e-5)
    close(got["dA"], back[0]["dA"].double() + back[1]["dA"].double(), "dA", 5e-5)


def test_scan_of_the_most_tokens(sdm):
    """2,097,120 tokens, 65,535 chunks of the gradient, against calls of a part of them."""
    B, T, D, N = 1, 2_097_120, 2, 2
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    u, de, dy, Bm, Cm = r(B, T, D), r(B, T, D), r(B, T, D), r(B, T, 1, N), r(B, T, 1, N)
    A = -torch.rand(D, N, generator=g, device="cuda") - 0.05
    s1, s2 = torch.zeros(B, D, N, device="cuda"), torch.zeros(B, D, N, device="cuda")
    y = sdm.selective_scan(u, de, A, Bm, Cm, state=s1)
    got = sdm.selective_scan_backward(u, de, A, Bm, Cm, dy)
    c = T // 3 + 5
    cut = lambda v: (v[:, :c], v[:, c:])  # noqa: E731
    parts, mid = [], None
    for q in range(2):
        if q:
            mid = s2.clone()
        parts.append(sdm.selective_scan(cut(u)[q], cut(de)[q], A, cut(Bm)[q], cut(Cm)[q], state=s2))
    close(torch.cat(parts, 1), y.double(), "y")
    close(s2, s1.double(), "state")
    late = sdm.selective_scan_backward(cut(u)[1], cut(de)[1], A, cut(Bm)[1], cut(Cm)[1], cut(dy)[1], state=mid)
    early = sdm.selective_scan_backward(cut(u)[0], cut(de)[0], A, cut(Bm)[0], cut(Cm)[0], cut(dy)[0],
                                        state=torch.zeros_like(mid), dstate_end=late["dstate"])
    for k in ("du", "ddelta", "dB", "dC"):
        close(torch.cat([early[k], late[k]], 1), got[k].double(), k, 5e-5)
    close(got["dA"], early["dA"].double() + late["dA"].double(), "dA", 5e-5)


def test_norm_of_more_than_2_31_values(sdm):
    rows, D = 530_000, 4096  # 2.17e9 values
    r, f = (torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    w = torch.rand(D, device="cuda") + 0.5
    o, n = sdm.block_norm(r, f, w_post=w, w_pre=w)
    g = sdm.block_norm_backward(r, f, r, f, w_post=w, w_pre=w)
    for a, b in ((0, 300), (rows - 300, rows), (rows // 2, rows // 2 + 300)):
        o2, n2 = sdm.block_norm(r[a:b].contiguous(), f[a:b].contiguous(), w_post=w, w_pre=w)
        g2 = sdm.block_norm_backward(r[a:b].contiguous(), f[a:b].contiguous(), r[a:b].contiguous(),
                                     f[a:b].contiguous(), w_post=w, w_pre=w)
        assert torch.equal(o[a:b], o2) and torch.equal(n[a:b], n2)
        for k in ("dr", "df"):  # a block's first row sums f^2 in another order: a step of bf16 at most
            d = (g[k][a:b].float() - g2[k].float()).abs()
            assert (d <= 2.0 ** -7 * g2[k].float().abs() + 1e-5).all(), k
