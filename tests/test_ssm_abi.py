"""The state-space block's entry points on the CPU: every refusal is made on the host, before
anything is enqueued, and the workspace queries answer without a GPU."""
import ctypes

import pytest


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_int64), ("sh", ctypes.c_int64),
                ("st", ctypes.c_int64)]


def _struct(names, more=()):
    return type("S", (ctypes.Structure,), {"_fields_": [(n, ctypes.c_int32) for n in names] + list(more)})


Conv = _struct(("B", "H", "T", "d", "K", "x_dtype", "act", "fresh"))
Scan = _struct(("B", "T", "D", "N", "G", "x_dtype", "softplus", "fresh"))


class Norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in
                                             ("D", "r_dtype", "f_dtype", "x_dtype")] + \
               [("eps", ctypes.c_float)]


@pytest.fixture(scope="module")
def lib():
    from sparse_state_linear_score_b200 import build
    lib = ctypes.CDLL(build.build())
    for n in ("sdm_short_conv_backward", "sdm_selective_scan", "sdm_selective_scan_backward",
              "sdm_block_norm_backward"):
        getattr(lib, n + "_workspace_bytes").restype = ctypes.c_size_t
    return lib


P = 0x1000  # pointers are looked at, never followed
BIG = ctypes.c_size_t(1 << 44)
V = lambda p, *s: ctypes.byref(View(p, *s))  # noqa: E731
p = ctypes.c_void_p


def conv_dims(**kw):
    d = dict(B=2, H=4, T=64, d=128, K=4, x_dtype=1, act=1, fresh=0)
    d.update(kw)
    return Conv(*d.values())


def scan_dims(**kw):
    d = dict(B=2, T=64, D=128, N=16, G=2, x_dtype=1, softplus=1, fresh=0)
    d.update(kw)
    return Scan(*d.values())


def norm_dims(**kw):
    d = dict(rows=10, D=64, r_dtype=0, f_dtype=0, x_dtype=1, eps=1e-6)
    d.update(kw)
    return Norm(*d.values())


CS = (4 * 64 * 128, 64 * 128, 128)


def conv(lib, d=None, x=None, w=p(P), bias=None, state=None, lens=None, y=None):
    d = conv_dims() if d is None else d
    return lib.sdm_short_conv(ctypes.byref(d), x or V(P, *CS), w, bias, state, lens,
                              y or V(2 * P, *CS), None)


@pytest.mark.parametrize("field,value,code", [
    ("x_dtype", 2, 3), ("act", 2, 1), ("fresh", 2, 1), ("B", 0, 2), ("H", 0, 2), ("d", 0, 2),
    ("T", -1, 2), ("K", 0, 2), ("K", 9, 2), ("B", 20000, 2)])
def test_conv_dims(lib, field, value, code):
    assert conv(lib, conv_dims(**{field: value})) == code
    assert lib.sdm_short_conv_backward_workspace_bytes(ctypes.byref(conv_dims(**{field: value}))) == 0


def test_conv_arguments(lib):
    assert lib.sdm_short_conv(None, V(P, *CS), p(P), None, None, None, V(2 * P, *CS), None) == 1
    assert conv(lib, x=V(None, *CS)) == 1 and conv(lib, y=V(None, *CS)) == 1
    assert conv(lib, w=None) == 1
    assert conv(lib, y=V(P, *CS)) == 1                       # in place
    assert conv(lib, x=V(P + 1, *CS)) == 4 and conv(lib, y=V(2 * P + 1, *CS)) == 4
    assert conv(lib, w=p(P + 4)) == 4 and conv(lib, bias=p(P + 8)) == 4
    assert conv(lib, state=p(P + 2)) == 4 and conv(lib, lens=p(P + 2)) == 4
    assert conv(lib, x=V(P, -1, CS[1], CS[2])) == 1          # negative stride
    assert conv(lib, y=V(2 * P, CS[0], CS[1], 127)) == 1     # rows overlap
    assert conv(lib, y=V(2 * P, 128, CS[1], 128)) == 1       # sequences overlap
    assert conv(lib, y=V(2 * P, 0, CS[1], 128)) == 1
    assert conv(lib, y=V(2 * P, CS[0], 1 << 61, 1 << 62)) == 1  # sizes that pass 64 bits
    d = conv_dims()
    need = lib.sdm_short_conv_backward_workspace_bytes(ctypes.byref(d))
    assert need >= 5 * 4 * 128 * 4

    def bwd(dy=V(2 * P, *CS), dx=V(3 * P, *CS), dw=p(P), ws=p(P), n=BIG, dse=None, ds=None):
        return lib.sdm_short_conv_backward(ctypes.byref(d), V(P, *CS), p(P), None, None, None, dy, dse,
                                           dx, dw, None, ds, ws, n, None)
    assert bwd(dx=V(P, *CS)) == 1 and bwd(dx=V(2 * P, *CS)) == 1 and bwd(dw=None) == 1
    assert bwd(ws=None) == 7 and bwd(n=ctypes.c_size_t(need - 1)) == 7 and bwd(ws=p(P + 8)) == 4
    assert bwd(dse=p(P + 4)) == 4 and bwd(ds=p(P + 4)) == 4


SS = (64 * 128, 0, 128)
GS = (64 * 32, 16, 32)


def scan(lib, d=None, u=None, A=p(P), B=None, y=None, z=None, state=None, lens=None, ws=p(P), n=BIG):
    d = scan_dims() if d is None else d
    return lib.sdm_selective_scan(ctypes.byref(d), u or V(P, *SS), V(P, *SS), A, B or V(P, *GS),
                                  V(P, *GS), None, z, None, state, lens, y or V(2 * P, *SS), ws, n,
                                  None)


@pytest.mark.parametrize("field,value,code", [
    ("x_dtype", -1, 3), ("softplus", 2, 1), ("fresh", -1, 1), ("B", 0, 2), ("D", 0, 2),
    ("G", 0, 2), ("G", 3, 2), ("N", 0, 2), ("N", 65, 2), ("T", -1, 2), ("T", (1 << 21) + 1, 2),
    ("B", 40000, 2)])
def test_scan_dims(lib, field, value, code):
    d = scan_dims(**{field: value})
    assert scan(lib, d) == code
    assert lib.sdm_selective_scan_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.sdm_selective_scan_backward_workspace_bytes(ctypes.byref(d)) == 0


def test_scan_arguments(lib):
    assert scan(lib, A=None) == 1 and scan(lib, u=V(None, *SS)) == 1
    assert scan(lib, y=V(P, *SS)) == 1
    assert scan(lib, u=V(P + 1, *SS)) == 4 and scan(lib, z=V(P + 1, *SS)) == 4
    assert scan(lib, B=V(P, -5, 16, 32)) == 1
    assert scan(lib, A=p(P + 4)) == 4 and scan(lib, state=p(P + 4)) == 4 and scan(lib, lens=p(P + 1)) == 4
    assert scan(lib, y=V(2 * P, SS[0], 0, 100)) == 1
    long = scan_dims(B=1, T=4096, D=64, G=1)
    need = lib.sdm_selective_scan_workspace_bytes(ctypes.byref(long))
    assert need > 0  # few channels, many tokens: split over time
    ls = (4096 * 64, 0, 64)
    a = dict(d=long, u=V(P, *ls), y=V(2 * P, *ls))
    assert scan(lib, **a, ws=None) == 7 and scan(lib, **a, n=ctypes.c_size_t(need - 1)) == 7
    assert scan(lib, **a, ws=p(P + 4)) == 4
    assert lib.sdm_selective_scan_workspace_bytes(ctypes.byref(scan_dims(T=1))) == 0
    assert lib.sdm_selective_scan_workspace_bytes(ctypes.byref(scan_dims(B=64, D=4096))) == 0

    d = scan_dims()
    need = lib.sdm_selective_scan_backward_workspace_bytes(ctypes.byref(d))
    assert need >= 2 * 64 * 2 * 2 * 16 * 4  # the shares of dB and dC

    def bwd(z=None, dz=None, du=V(3 * P, *SS), dd=V(4 * P, *SS), dA=p(P), dB=p(P), ws=p(P), n=BIG):
        return lib.sdm_selective_scan_backward(
            ctypes.byref(d), V(P, *SS), V(P, *SS), p(P), V(P, *GS), V(P, *GS), None, z, None, None, None,
            V(2 * P, *SS), None, du, dd, dA, dB, p(P), None, dz, None, None, ws, n, None)
    assert bwd(z=V(P, *SS)) == 1 and bwd(dz=V(5 * P, *SS)) == 1   # z and dz come together
    assert bwd(dA=None) == 1 and bwd(dB=None) == 1 and bwd(dB=p(P + 2)) == 4
    assert bwd(du=V(2 * P, *SS)) == 1 and bwd(dd=V(3 * P, *SS)) == 1
    assert bwd(ws=None) == 7 and bwd(n=ctypes.c_size_t(need - 1)) == 7


@pytest.mark.parametrize("field,value,code", [
    ("r_dtype", 2, 3), ("f_dtype", -1, 3), ("x_dtype", 3, 3), ("rows", -1, 2), ("D", 0, 2),
    ("D", 16385, 2), ("eps", -1.0, 1), ("eps", float("nan"), 1)])
def test_norm_dims(lib, field, value, code):
    d = norm_dims(**{field: value})
    assert lib.sdm_block_norm(ctypes.byref(d), p(P), p(P), None, None, None, None, p(P), p(P), None) == code
    assert lib.sdm_block_norm_backward_workspace_bytes(ctypes.byref(d)) == 0


def test_norm_arguments(lib):
    d = norm_dims()

    def fwd(r=p(P), f=p(P), w=None, r_out=p(P), n=p(P)):
        return lib.sdm_block_norm(ctypes.byref(d), r, f, w, None, None, None, r_out, n, None)
    assert fwd(r=None) == 1 and fwd(f=None) == 1 and fwd(r_out=None, n=None) == 1
    assert fwd(w=p(P + 4)) == 4 and fwd(n=p(P + 8)) == 4
    need = lib.sdm_block_norm_backward_workspace_bytes(ctypes.byref(d))
    assert need >= 10 * 3 * 64 * 4

    def bwd(gate=None, dgate=None, w=None, dw=None, ws=p(P), n=BIG):
        return lib.sdm_block_norm_backward(ctypes.byref(d), p(P), p(P), w, gate, None, None, p(P), p(P),
                                           p(P), p(P), dgate, None, dw, None, ws, n, None)
    assert bwd(dgate=p(P)) == 1 and bwd(dw=p(P)) == 1
    assert bwd(ws=None) == 7 and bwd(n=ctypes.c_size_t(need - 1)) == 7 and bwd(ws=p(P + 4)) == 4


@pytest.mark.parametrize("dims,sizes", [
    ("_conv_dims", (2, 4, 64, 128, 4, 1, 1, 0)), ("_scan_dims", (2, 64, 128, 16, 2, 1, 1, 0)),
    ("_norm_dims", (10, 64, 0, 0, 1, 1e-6))])
def test_binding_sizes(dims, sizes):
    """The binding's dims structures hold what they are given or refuse it."""
    import sparse_state_linear_score_b200 as m
    f = getattr(m, dims)
    f(*sizes)
    for i, v in enumerate(sizes):
        if isinstance(v, int) and not (dims == "_norm_dims" and i == 0):
            with pytest.raises(ValueError, match="too large"):
                f(*sizes[:i], (1 << 32) + v, *sizes[i + 1:])


def test_binding_refuses_norms_of_scalars(monkeypatch):
    """A tensor without dimensions is not taken for an empty call, whose outputs nothing writes."""
    import torch

    import sparse_state_linear_score_b200 as m
    monkeypatch.setattr(m, "_act_dtype", lambda t, what: 0)
    s, r = torch.ones(()), torch.ones(2, 8)
    with pytest.raises(ValueError, match="dimensions"):
        m._norm_setup(s, s, torch.float32, 1e-6)
    for t in (r, r[:0]):
        assert m._norm_setup(t, t, torch.float32, 1e-6)[0].rows == len(t)
