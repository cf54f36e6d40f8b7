"""Refusals of the feed-forward operators, on the host (no GPU needed): every
documented error comes back before anything is launched, so the fake device
addresses are never touched; and the binding's own checks."""
import contextlib
import ctypes

import pytest
import torch

import semi_structured_sparse_nm_amd as nm
from tests.test_abi_host import FAKE, _desc

P = [FAKE + (i << 28) for i in range(1, 12)]
EINVAL, EUNSUP = nm.NM_EINVAL, nm.NM_EUNSUPPORTED


def _w(**kw):
    return _desc(R=kw.pop("R", 48), K=kw.pop("K", 128), dt=kw.pop("dt", nm.NM_F16), **kw)


def _glu(g=None, u=None, X=P[0], ldx=128, T=5, H=P[1], ldh=48, act=2, G=None, U=None, ldp=0, ws=P[2], wsb=1 << 30):
    g, u = g or _w(), u or _w()
    return nm.lib().nm_glu(ctypes.byref(g), ctypes.byref(u), X, ldx, T, H, ldh, act, G, U, ldp, ws, wsb, None)


def test_glu_refusals():
    L = nm.lib()
    # a 4:8 weight and many tokens: dense copies in the workspace
    dense = dict(T=1100, g=_w(N=4, M=8), u=_w(N=4, M=8))
    assert L.nm_glu(None, None, P[0], 128, 5, P[1], 48, 2, None, None, 0, None, 0, None) == EINVAL
    for kw in (dict(X=None), dict(H=None), dict(T=0), dict(T=-3), dict(ldx=127), dict(ldh=47), dict(G=P[3], ldp=48),
               dict(U=P[3], ldp=48), dict(G=P[3], U=P[4], ldp=47), dict(u=_w(R=49)), dict(u=_w(K=132)),
               dict(u=_w(N=1)), dict(u=_w(N=4, M=8)), dict(u=_w(dt=nm.NM_BF16)), dict(g=_w(format_version=0)),
               dict(u=_w(format_version=9)), dict(g=_w(values_bytes=7)), dict(u=_w(meta=None)),
               dict(**dense, ws=None), dict(**dense, wsb=1000), dict(T=1100, X=P[0] + 2, ws=None)):
        assert _glu(**kw) == EINVAL, kw
    i8 = dict(dt=nm.NM_I8)
    for kw in (dict(g=_w(**i8), u=_w(**i8)), dict(act=0), dict(act=3), dict(X=P[0] + 1), dict(H=P[1] + 1),
               dict(G=P[3] + 1, U=P[4], ldp=48), dict(**dense, ws=P[2] + 16), dict(T=(1 << 30) + 1)):
        assert _glu(**kw) == EUNSUP, kw
    big = dict(R=(1 << 22) + 16, K=8)
    assert _glu(g=_w(**big), u=_w(**big), ldx=8, ldh=big["R"]) == EUNSUP
    big = dict(R=16, K=1 << 22)
    assert _glu(g=_w(**big), u=_w(**big), ldx=1 << 22) == EUNSUP


def test_glu_workspace():
    n = ctypes.c_size_t()
    f = nm.lib().nm_glu_workspace_size
    g, u = _w(R=50, K=100), _w(R=50, K=100)
    assert f(ctypes.byref(g), ctypes.byref(u), None, 0, 1100, ctypes.byref(n)) == nm.NM_OK and n.value == 1100 * 256
    assert f(ctypes.byref(g), ctypes.byref(u), None, 0, 0, ctypes.byref(n)) == EINVAL
    assert f(ctypes.byref(g), ctypes.byref(u), None, 0, 5, None) == EINVAL
    assert f(ctypes.byref(g), ctypes.byref(u), P[0], 99, 5, ctypes.byref(n)) == EINVAL
    assert f(ctypes.byref(g), ctypes.byref(_w(R=51, K=100)), None, 0, 5, ctypes.byref(n)) == EINVAL
    # rows the kernels read as they are, and not: tiles, then streamed weights
    d, short = _w(R=50, K=104), _w(R=50, K=4)
    for X, ldx, want in ((P[0], 104, 0), (P[0] + 16, 112, 0), (P[0] + 2, 104, 1100 * 256), (P[0], 105, 1100 * 256)):
        assert f(ctypes.byref(d), ctypes.byref(d), X, ldx, 1100, ctypes.byref(n)) == nm.NM_OK and n.value == want
        assert f(ctypes.byref(d), ctypes.byref(d), X, ldx, 5, ctypes.byref(n)) == nm.NM_OK and n.value == 0
    assert f(ctypes.byref(short), ctypes.byref(short), P[0], 4, 5, ctypes.byref(n)) == nm.NM_OK and n.value == 1280 // 2 + 128
    b = nm.lib().nm_glu_backward_workspace_size
    assert b(ctypes.byref(g), ctypes.byref(u), 5, ctypes.byref(n)) == nm.NM_OK and n.value > 0
    assert b(ctypes.byref(g), ctypes.byref(u), 1 << 22, ctypes.byref(n)) == EUNSUP
    assert b(ctypes.byref(g), ctypes.byref(u), 0, ctypes.byref(n)) == EINVAL


def _bwd(g=None, u=None, X=P[0], ldx=128, T=5, G=P[1], U=P[2], ldp=48, dH=P[3], lddh=48, act=2, dX=P[4], lddx=128,
         dWg=P[5], dWu=P[6], lddw=128, ws=P[7], wsb=1 << 27):
    g, u = g or _w(), u or _w()
    return nm.lib().nm_glu_backward(ctypes.byref(g), ctypes.byref(u), X, ldx, T, G, U, ldp, dH, lddh, act, dX, lddx,
                                    dWg, dWu, lddw, ws, wsb, None)


def test_glu_backward_refusals():
    for kw in (dict(X=None), dict(G=None), dict(U=None), dict(dH=None), dict(T=0), dict(ldx=127), dict(ldp=47),
               dict(lddh=47), dict(lddx=127), dict(lddw=127), dict(dWg=None), dict(dWu=None),
               dict(dX=None, dWg=None, dWu=None), dict(ws=None), dict(wsb=100), dict(u=_w(R=64)),
               dict(g=_w(format_version=0))):
        assert _bwd(**kw) == EINVAL, kw
    for kw in (dict(act=0), dict(act=7), dict(ws=P[7] + 16), dict(dH=P[3] + 1), dict(dWu=P[6] + 1), dict(dX=P[4] + 1),
               dict(T=1 << 22)):
        assert _bwd(**kw) == EUNSUP, kw
    long = dict(R=1 << 21, K=8)
    assert _bwd(g=_w(**long), u=_w(**long), T=1, ldx=8, ldp=1 << 21, lddh=1 << 21, lddx=8, lddw=8) == EUNSUP
    # operands' tiles past one launch
    wide = dict(R=1 << 20, K=1 << 12)
    assert _bwd(g=_w(**wide), u=_w(**wide), T=1 << 21, ldx=1 << 12, ldp=1 << 20, lddh=1 << 20, lddx=1 << 12,
                lddw=1 << 12, wsb=1 << 62) == EUNSUP


def test_kept_products_type():
    """G and U in the weights' type or binary32, aligned to their element."""
    L = nm.lib()

    def fwd(pdt, G=P[3], U=P[4], ldp=47):
        g, u = _w(), _w()
        return L.nm_glu_kept(ctypes.byref(g), ctypes.byref(u), P[0], 128, 5, P[1], 48, 2, G, U, ldp, pdt, P[2], 1 << 30,
                             None)

    def bwd(pdt, G=P[1], U=P[2], wsb=100):
        g, u = _w(), _w()
        return L.nm_glu_backward_kept(ctypes.byref(g), ctypes.byref(u), P[0], 128, 5, G, U, 48, pdt, P[3], 48, 2, P[4],
                                      128, P[5], P[6], 128, P[7], wsb, None)

    for pdt in (nm.NM_F16, nm.NM_F32):                    # (as far as the row pitch and the workspace, which are refused)
        assert fwd(pdt) == EINVAL and bwd(pdt) == EINVAL
    for pdt in (nm.NM_BF16, nm.NM_I8, nm.NM_I32, 9):
        assert fwd(pdt, ldp=48) == EUNSUP and bwd(pdt) == EUNSUP
    assert fwd(nm.NM_F32, G=P[3] + 2, ldp=48) == EUNSUP and fwd(nm.NM_F32, U=P[4] + 2, ldp=48) == EUNSUP
    assert bwd(nm.NM_F32, G=P[1] + 2) == EUNSUP and bwd(nm.NM_F32, U=P[2] + 2) == EUNSUP
    p = _packed()
    X = torch.zeros(3, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="pre has dtype torch.bfloat16, expected torch.float16 or torch.float32"):
        nm.glu(p, p, X, pre=torch.zeros(2, 3, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.glu(p, p, X, pre=torch.zeros(2, 3, 16))


def test_mx_workspace():
    n = ctypes.c_size_t()
    f = nm.lib().nm_mx_workspace_size
    w, x = _mx(40, 304), _mx(17, 304)
    b, nb = ctypes.byref(w), ctypes.byref(n)
    for xq, T, want in ((None, 16, 0), (None, 17, 17 * 256 + 2 * 256), (ctypes.byref(x), 17, 0)):
        assert f(b, xq, T, 0, nb) == nm.NM_OK and n.value == want
    narrow = _mx(40, 7)
    assert f(ctypes.byref(narrow), None, 1, 0, nb) == nm.NM_OK and n.value == 2 * 256
    assert f(b, None, 0, 0, nb) == EINVAL and f(None, None, 5, 0, nb) == EINVAL and f(b, None, 5, 0, None) == EINVAL


@pytest.mark.parametrize("shape", [0, 1, 2, 3])
@pytest.mark.parametrize("asked,slabs,split", [(1, 33, 1), (2, 33, 2), (7, 33, 7), (16, 33, 11), (16, 32, 16), (5, 6, 3),
                                               (5, 10, 5), (5, 1, 1), (16, 3, 3)])
def test_forced_splits(monkeypatch, shape, asked, slabs, split):
    """A forced split is taken, or the most slices up to it that the reduction
    divides into: seen by the partial sums' workspace."""
    monkeypatch.setenv("NM_FFN_TILE", f"tile:{shape}:{asked}")
    n = ctypes.c_size_t()
    T, R = 70, 333
    w, x = _mx(R, 256 * slabs), _mx(T, 256 * slabs)
    assert nm.lib().nm_mx_workspace_size(ctypes.byref(w), ctypes.byref(x), T, 0, ctypes.byref(n)) == nm.NM_OK
    assert n.value == (-(-split * T * R * 4 // 256) * 256 if split > 1 else 0)
    # the input's gradient: a reduction over both weights' rows, 64 a slab, in two
    # parts at this size (the most a call can need)
    sps = -(-2 * slabs // min(asked, 2 * slabs, 16))
    split = -(-2 * slabs // sps)
    if slabs % 2 == 0:
        g = _w(R=32 * slabs - 5, K=128)
        f = nm.lib().nm_glu_backward_workspace_size
        assert f(ctypes.byref(g), ctypes.byref(g), T, ctypes.byref(n)) == nm.NM_OK
        got = n.value
        monkeypatch.setenv("NM_FFN_TILE", f"tile:{shape}:1")
        assert f(ctypes.byref(g), ctypes.byref(g), T, ctypes.byref(n)) == nm.NM_OK
        assert got - n.value == (-(-split * T * 128 * 4 // 256) * 256 if split > 1 else 0)


def test_lengths_past_one_launch():
    """Sizes whose launch would pass 2^32 threads are refused."""
    c = ctypes.c_size_t()
    assert nm.lib().nm_mx_size(1 << 26, 8, ctypes.byref(c), ctypes.byref(c)) == EUNSUP
    assert nm.lib().nm_mx_size(8, 1 << 26, ctypes.byref(c), ctypes.byref(c)) == EUNSUP
    m = _mx(1 << 24, 1 << 13)
    assert nm.lib().nm_mx_quantize(P[0], 1 << 13, nm.NM_F16, ctypes.byref(m), None) == EUNSUP
    w = _mx(16, 1 << 13)
    f = nm.lib().nm_mx_workspace_size
    assert f(ctypes.byref(w), None, 1 << 24, 0, ctypes.byref(c)) == EUNSUP
    assert f(ctypes.byref(w), None, 1 << 20, 0, ctypes.byref(c)) == nm.NM_OK
    assert nm.lib().nm_mx_linear(ctypes.byref(w), None, P[0], 1 << 13, nm.NM_F16, 1 << 24, P[1], 16, nm.NM_F16, None,
                                 0, P[2], 1 << 62, None) == EUNSUP
    g = _w(R=8, K=8)
    assert nm.lib().nm_glu_workspace_size(ctypes.byref(g), ctypes.byref(g), None, 0, (1 << 25) + 1, ctypes.byref(c)) == EUNSUP


def _mx(rows=40, K=300, **kw):
    c, s = nm.mx_size(rows, K)
    d = nm.NmMx(rows, K, nm.FORMAT_VERSION, 0, P[8], c, P[9], s)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_mx_size():
    assert nm.mx_size(1, 1) == (128, 256)
    assert nm.mx_size(33, 257) == (33 * 256, 2 * 2 * 256)
    c = ctypes.c_size_t()
    f = nm.lib().nm_mx_size
    assert f(0, 4, ctypes.byref(c), ctypes.byref(c)) == EINVAL
    assert f(4, 0, ctypes.byref(c), ctypes.byref(c)) == EINVAL
    assert f(4, 4, None, ctypes.byref(c)) == EINVAL
    assert f(1 << 31, 4, ctypes.byref(c), ctypes.byref(c)) == EUNSUP


def test_mx_quantize_refusals():
    L = nm.lib()

    def q(m, X=P[0], ldx=300, dt=nm.NM_F16):
        return L.nm_mx_quantize(X, ldx, dt, ctypes.byref(m), None)

    def d(m, Y=P[0], ldy=300, dt=nm.NM_F16):
        return L.nm_mx_dequantize(ctypes.byref(m), Y, ldy, dt, None)

    assert L.nm_mx_quantize(P[0], 300, nm.NM_F16, None, None) == EINVAL
    for f in (q, d):
        assert f(_mx(), None) == EINVAL
        assert f(_mx(), P[0], 299) == EINVAL
        assert f(_mx(codes_bytes=3)) == EINVAL and f(_mx(scales_bytes=3)) == EINVAL and f(_mx(codes=None)) == EINVAL
        assert f(_mx(), P[0] + 1) == EUNSUP and f(_mx(), P[0], 300, nm.NM_I8) == EUNSUP
        assert f(_mx(codes=P[8] + 4)) == EUNSUP
    assert d(_mx(format_version=0)) == EINVAL


def _lin(w=None, xq=None, X=P[0], ldx=300, xdt=nm.NM_BF16, T=20, Y=P[1], ldy=40, ydt=nm.NM_BF16, bias=None, act=0,
         ws=P[2], wsb=1 << 28):
    w = w or _mx()
    return nm.lib().nm_mx_linear(ctypes.byref(w), None if xq is None else ctypes.byref(xq), X, ldx, xdt, T, Y, ldy,
                                 ydt, bias, act, ws, wsb, None)


def test_mx_product_refusals():
    for kw in (dict(X=None), dict(Y=None), dict(T=0), dict(ldx=299), dict(ldy=39), dict(w=_mx(format_version=0)),
               dict(xq=_mx(21, 300)), dict(xq=_mx(20, 301)), dict(xq=_mx(20, 300, format_version=0)), dict(ws=None),
               dict(wsb=64)):
        assert _lin(**kw) == EINVAL, kw
    for kw in (dict(xdt=nm.NM_I8), dict(ydt=nm.NM_I32), dict(act=2), dict(X=P[0] + 1), dict(Y=P[1] + 1),
               dict(bias=P[3] + 2), dict(ws=P[2] + 32), dict(w=_mx(8, 1 << 24), X=P[0], ldx=1 << 24)):
        assert _lin(**kw) == EUNSUP, kw
    L = nm.lib()
    g, u = _mx(), _mx()

    def glu(u, act=2, H=P[1]):
        return L.nm_mx_glu(ctypes.byref(g), u, None, P[0], 300, nm.NM_BF16, 20, H, 40, nm.NM_BF16, act, P[2],
                           1 << 28, None)

    assert glu(None) == EINVAL and glu(ctypes.byref(_mx(41))) == EINVAL and glu(ctypes.byref(_mx(40, 301))) == EINVAL
    assert glu(ctypes.byref(u), act=0) == EUNSUP and glu(ctypes.byref(u), H=None) == EINVAL


# ---------------------------------------------------------------- binding
def _packed(R=16, K=64, N=2, M=4, dt=nm.NM_F16):
    v, m = nm.pack_size(R, K, N, M, dt)
    return nm.Packed(R, K, N, M, dt, torch.empty(v, dtype=torch.uint8), torch.empty(m, dtype=torch.uint8) if m else None)


def test_binding_refuses_before_the_library():
    p = _packed()
    X = torch.zeros(3, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.glu(p, p, X)
    with pytest.raises(ValueError, match="act must be"):
        nm.glu(p, p, X, act="relu")
    with pytest.raises(ValueError, match="differ in rows"):
        nm.glu(p, _packed(R=17), X)
    with pytest.raises(ValueError, match="differ in N"):
        nm.glu(p, _packed(N=1), X)
    with pytest.raises(TypeError, match="gated block takes"):
        nm.glu(_packed(dt=nm.NM_I8), _packed(dt=nm.NM_I8), X)
    with pytest.raises(TypeError, match="Xt has dtype"):
        nm.glu(p, p, X.bfloat16())
    with pytest.raises(ValueError, match="Xt must be"):
        nm.glu(p, p, X[:, :63])
    with pytest.raises(ValueError, match="unit stride"):
        nm.glu(p, p, torch.zeros(64, 3, dtype=torch.float16).t())
    with pytest.raises(ValueError, match="overlapping rows"):
        nm.glu(p, p, X[:1].expand(3, 64))
    with pytest.raises(ValueError, match="out must be"):
        nm.glu(p, p, X, out=torch.zeros(3, 15, dtype=torch.float16))
    with pytest.raises(TypeError, match="out has dtype"):
        nm.glu(p, p, X, out=torch.zeros(3, 16))
    with pytest.raises(ValueError, match="pre must be"):
        nm.glu(p, p, X, pre=torch.zeros(3, 16, dtype=torch.float16))
    with pytest.raises(ValueError, match="halves of pre overlap"):
        nm.glu(p, p, X, pre=torch.zeros(1, 3, 16, dtype=torch.float16).expand(2, 3, 16))
    with pytest.raises(ValueError, match="halves of pre overlap"):
        nm.glu(p, p, X, pre=torch.zeros(4, 40, dtype=torch.float16).as_strided((2, 3, 16), (30, 40, 1)))
    with pytest.raises(ValueError, match="pre has overlapping rows"):
        nm.glu(p, p, X, pre=torch.zeros(2, 1, 16, dtype=torch.float16).expand(2, 3, 16))
    with pytest.raises(ValueError, match="pre must have unit stride"):
        nm.glu(p, p, X, pre=torch.zeros(2, 16, 3, dtype=torch.float16).transpose(1, 2))
    pre, dH = torch.zeros(2, 3, 16, dtype=torch.float16), torch.zeros(3, 16, dtype=torch.float16)
    with pytest.raises(ValueError, match="need_dx or need_dw"):
        nm.glu_backward(p, p, X, pre, dH, need_dx=False, need_dw=False)
    with pytest.raises(TypeError, match="dH has dtype"):
        nm.glu_backward(p, p, X, pre, dH.float())
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.glu_backward(p, p, X, pre, dH)


def test_binding_refuses_mx_operands():
    c, s = nm.mx_size(16, 64)
    w = nm.Mx(16, 64, torch.empty(c, dtype=torch.uint8), torch.empty(s, dtype=torch.uint8))
    X = torch.zeros(3, 64)
    with pytest.raises(TypeError, match="X must be float16"):
        nm.mx_quantize(X.double())
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.mx_quantize(X)
    with pytest.raises(ValueError, match="2-D"):
        nm.mx_quantize(X[0])
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.mx_dequantize(w)
    with pytest.raises(ValueError, match="X must be"):
        nm.mx_linear(w, X[:, :60])
    with pytest.raises(ValueError, match="act must be"):
        nm.mx_linear(w, X, act="silu")
    with pytest.raises(ValueError, match="bias must be"):
        nm.mx_linear(w, X, bias=torch.zeros(15))
    with pytest.raises(TypeError, match="out has dtype"):
        nm.mx_linear(w, X, out=torch.zeros(3, 16), out_dtype=torch.float16)
    with pytest.raises(TypeError, match="out must be float16"):
        nm.mx_linear(w, X, out_dtype=torch.int32)
    with pytest.raises(ValueError, match="has K=32"):
        c2, s2 = nm.mx_size(3, 32)
        nm.mx_linear(w, nm.Mx(3, 32, torch.empty(c2, dtype=torch.uint8), torch.empty(s2, dtype=torch.uint8)))
    with pytest.raises(ValueError, match="gate is 16 x 64, up is 17 x 64"):
        nm.mx_glu(w, nm.Mx(17, 64, w.codes, w.scales), X)
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.mx_glu(w, w, X)


class _On:
    """Stands for a tensor on one device."""

    def __init__(self, i):
        self.i, self.device = i, f"cuda:{i}"

    def get_device(self):
        return self.i


def test_binding_names_the_tensor_on_another_gpu():
    a, b = _On(0), _On(1)
    assert nm._one_gpu("X, gate, out", a, a, None) == 0 and nm._one_gpu("X, gate, out", b, None, b) == 1
    with pytest.raises(ValueError, match="out is on cuda:1, X on cuda:0"):
        nm._one_gpu("X, gate, out", a, None, b)
    with pytest.raises(ValueError, match="gate is on cuda:0, X on cuda:1"):
        nm._one_gpu("X, gate, out", b, a, b)


def test_workspace_sizes_follow_a_forced_path(monkeypatch):
    """A size remembered for one path is not given to a call that the
    environment sends down another."""
    asked = []

    def size(want, out):
        asked.append(want)
        out._obj.value = want
        return nm.NM_OK

    monkeypatch.setattr(torch.cuda, "device", lambda i: contextlib.nullcontext())
    monkeypatch.setattr(nm, "_ws_sizes", {})
    monkeypatch.delenv("NM_FFN_TILE", raising=False)
    key = ("glu", 8, 8, 0)
    assert nm._sized(size, "size", key, 5) == 5 and nm._sized(size, "size", key, 6) == 5 and asked == [5]
    monkeypatch.setenv("NM_FFN_TILE", "stream:0")
    assert nm._sized(size, "size", key, 7) == 7
    monkeypatch.setenv("NM_FFN_TILE", "stream:1")
    assert nm._sized(size, "size", key, 8) == 8
    monkeypatch.delenv("NM_FFN_TILE")
    assert nm._sized(size, "size", key, 9) == 5 and asked == [5, 7, 8]
