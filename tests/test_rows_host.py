"""Refusals of the 8-bit rows and of the products of rows grouped by expert, on
the host (no GPU needed): every documented error comes back before anything is
launched, so the fake device addresses are never touched; and the binding's own
checks, and the 64-bit forms the GPU tests compare with."""
import ctypes

import pytest
import torch

import semi_structured_sparse_nm_amd as nm
from tests._rows import experts_of, i8_64
from tests.test_abi_host import FAKE, _desc

P = [FAKE + (i << 28) for i in range(1, 14)]
EINVAL, EUNSUP = nm.NM_EINVAL, nm.NM_EUNSUPPORTED


def _i8(rows=20, K=300, **kw):
    d = nm.NmI8(rows, K, nm.FORMAT_VERSION, 0, P[8], rows * (-(-K // 128) * 128), P[9], rows * 4)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _experts(E=3, R=40, K=128, N=2, M=4, dt=nm.NM_F16, **kw):
    v, m = ctypes.c_size_t(), ctypes.c_size_t()
    assert nm.lib().nm_experts_size(E, R, K, N, M, dt, ctypes.byref(v), ctypes.byref(m)) == nm.NM_OK
    d = nm.NmExperts(E, R, K, N, M, dt, nm.FORMAT_VERSION, P[10], v.value, P[11] if m.value else None, m.value)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


# ---------------------------------------------------------------- 8-bit rows
def test_i8_sizes():
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    f = nm.lib().nm_i8_size
    for rows, K, want in ((1, 1, 128), (3, 128, 384), (2, 129, 512)):
        assert f(rows, K, ctypes.byref(c), ctypes.byref(s)) == nm.NM_OK and (c.value, s.value) == (want, 4 * rows)
    assert f(0, 4, ctypes.byref(c), ctypes.byref(s)) == EINVAL and f(4, 0, ctypes.byref(c), ctypes.byref(s)) == EINVAL
    assert f(4, 4, None, ctypes.byref(s)) == EINVAL and f(4, 4, ctypes.byref(c), None) == EINVAL
    assert f(1, 131072, ctypes.byref(c), ctypes.byref(s)) == EUNSUP
    assert f(1 << 40, 2, ctypes.byref(c), ctypes.byref(s)) == EUNSUP


def test_i8_quantize_refusals():
    L = nm.lib()

    def q(m, X=P[0], ldx=300, dt=nm.NM_F16):
        return L.nm_i8_quantize(X, ldx, dt, ctypes.byref(m), None)

    def d(m, Y=P[0], ldy=300, dt=nm.NM_F16):
        return L.nm_i8_dequantize(ctypes.byref(m), Y, ldy, dt, None)

    assert L.nm_i8_quantize(P[0], 300, nm.NM_F16, None, None) == EINVAL
    assert L.nm_i8_dequantize(None, P[0], 300, nm.NM_F16, None) == EINVAL
    for f in (q, d):
        assert f(_i8(), None) == EINVAL and f(_i8(), P[0], 299) == EINVAL
        for kw in (dict(codes_bytes=3), dict(scales_bytes=3), dict(codes=None), dict(scales=None)):
            assert f(_i8(**kw)) == EINVAL, kw
        assert f(_i8(), P[0] + 1) == EUNSUP and f(_i8(), P[0] + 2, 300, nm.NM_F32) == EUNSUP
        assert f(_i8(), P[0], 300, nm.NM_I8) == EUNSUP and f(_i8(codes=P[8] + 8)) == EUNSUP
        assert f(_i8(scales=P[9] + 2)) == EUNSUP
    assert d(_i8(format_version=0)) == EINVAL


def _lin(w=None, ws=P[1], xq=None, X=P[0], ldx=300, xdt=nm.NM_BF16, T=20, Y=P[2], ldy=40, ydt=nm.NM_BF16, bias=None,
         act=0, wsp=P[3], wsb=1 << 28):
    w = w or _desc(R=40, K=300)
    return nm.lib().nm_i8_linear(ctypes.byref(w), ws, None if xq is None else ctypes.byref(xq), X, ldx, xdt, T, Y, ldy,
                                 ydt, bias, act, wsp, wsb, None)


def test_i8_linear_refusals(monkeypatch):
    assert nm.lib().nm_i8_linear(None, P[1], None, P[0], 300, nm.NM_F16, 5, P[2], 40, nm.NM_F16, None, 0, P[3], 1 << 28,
                                 None) == EINVAL
    w = dict(R=40, K=300)
    for kw in (dict(X=None), dict(Y=None), dict(ws=None), dict(T=0), dict(ldx=299), dict(ldy=39),
               dict(w=_desc(**w, format_version=0)), dict(w=_desc(**w, values_bytes=7)), dict(w=_desc(**w, meta=None)),
               dict(xq=_i8(21)), dict(xq=_i8(20, 301)), dict(xq=_i8(format_version=0)), dict(xq=_i8(codes=None)),
               dict(wsp=None), dict(wsb=64)):
        assert _lin(**kw) == EINVAL, kw
    for kw in (dict(xdt=nm.NM_I8), dict(ydt=nm.NM_I32), dict(act=2), dict(X=P[0] + 1), dict(Y=P[2] + 1),
               dict(bias=P[4] + 2), dict(ws=P[1] + 1), dict(wsp=P[3] + 32), dict(T=(1 << 25) + 1),
               dict(w=_desc(**w, dt=nm.NM_F16)), dict(w=_desc(R=16, K=131072), ldx=131072), dict(xq=_i8(codes=P[8] + 4)),
               dict(w=_desc(R=(1 << 22) + 16, K=8), ldx=8, ldy=1 << 23)):
        assert _lin(**kw) == EUNSUP, kw
    # dense copies in the workspace
    monkeypatch.setenv("NM_FFN_TILE", "tile:1")
    dense = dict(w=_desc(**w, N=3), xq=_i8(200), T=200)
    assert _lin(**dense, wsp=None) == EINVAL and _lin(**dense, wsb=18000) == EINVAL
    assert _lin(**dense, wsp=P[3] + 16) == EUNSUP


def test_i8_workspace(monkeypatch):
    monkeypatch.setenv("NM_FFN_TILE", "tile:1")           # (streamed or wide products need no copies)
    n = ctypes.c_size_t()
    f = nm.lib().nm_i8_linear_workspace_size
    x = _i8(20)
    for w, xq, T, want in ((_desc(R=40, K=300), None, 20, 20 * 384 + 256), (_desc(R=40, K=300), x, 20, 0),
                           (_desc(R=40, K=300, N=4), None, 500, 500 * 384 + 2048),
                           (_desc(R=40, K=300, N=3), x, 500, 3 * 3 * 2048),
                           (_desc(R=40, K=300, N=1), x, 500, 9 * 1024 + 9 * 256)):
        assert f(ctypes.byref(w), None if xq is None else ctypes.byref(xq), T, ctypes.byref(n)) == nm.NM_OK
        assert n.value == want
    w = _desc(R=40, K=300)
    assert f(ctypes.byref(w), None, 0, ctypes.byref(n)) == EINVAL and f(ctypes.byref(w), None, 5, None) == EINVAL
    assert f(None, None, 5, ctypes.byref(n)) == EINVAL
    assert f(ctypes.byref(_desc(R=40, K=300, dt=nm.NM_BF16)), None, 5, ctypes.byref(n)) == EUNSUP
    for path in ("stream:1", "wide:0", "wide:1"):
        monkeypatch.setenv("NM_FFN_TILE", path)
        assert f(ctypes.byref(_desc(R=40, K=300, N=3)), ctypes.byref(_i8(500)), 500, ctypes.byref(n)) == nm.NM_OK
        assert n.value == 0


# ---------------------------------------------------------------- experts
def test_experts_sizes_and_pack():
    v, m = ctypes.c_size_t(), ctypes.c_size_t()
    L = nm.lib()
    one = nm.pack_size(33, 72, 3, 8, nm.NM_F16)
    assert L.nm_experts_size(5, 33, 72, 3, 8, nm.NM_F16, ctypes.byref(v), ctypes.byref(m)) == nm.NM_OK
    assert (v.value, m.value) == (5 * one[0], 5 * one[1])
    for E, want in ((0, EINVAL), (1024, EUNSUP)):
        assert L.nm_experts_size(E, 33, 72, 3, 8, nm.NM_F16, ctypes.byref(v), ctypes.byref(m)) == want
    assert L.nm_experts_size(2, 33, 71, 3, 8, nm.NM_F16, ctypes.byref(v), ctypes.byref(m)) == EINVAL
    assert L.nm_experts_size(2, 33, 72, 3, 8, nm.NM_F16, None, ctypes.byref(m)) == EINVAL

    def pack(d, W=P[0], lde=40 * 128, ldw=128):
        return L.nm_experts_pack(W, lde, ldw, ctypes.byref(d), None)

    assert L.nm_experts_pack(P[0], 1, 128, None, None) == EINVAL
    for kw in (dict(W=None), dict(ldw=127), dict(lde=-1)):
        assert pack(_experts(), **kw) == EINVAL, kw
    for kw in (dict(values_bytes=7), dict(values=None), dict(meta=None), dict(experts=0), dict(experts=2)):
        assert pack(_experts(**kw)) == EINVAL, kw
    assert pack(_experts(), W=P[0] + 1) == EUNSUP


def _el(w=None, X=P[0], ldx=128, T=5, o=P[1], odt=0, Y=P[2], ldy=40, fill=0, ws=P[3], wsb=1 << 28):
    w = w or _experts()
    return nm.lib().nm_expert_linear(ctypes.byref(w), X, ldx, T, o, odt, Y, ldy, fill, ws, wsb, None)


def test_expert_linear_refusals(monkeypatch):
    assert nm.lib().nm_expert_linear(None, P[0], 128, 5, P[1], 0, P[2], 40, 0, None, 0, None) == EINVAL
    for kw in (dict(X=None), dict(Y=None), dict(o=None), dict(T=0), dict(T=-1), dict(ldx=127), dict(ldy=39),
               dict(w=_experts(format_version=0)), dict(w=_experts(values_bytes=7)), dict(w=_experts(meta=None)),
               dict(w=_experts(experts=0)), dict(w=_experts(K=4), ldx=4, wsb=0)):
        assert _el(**kw) == EINVAL, kw
    for kw in (dict(w=_experts(dt=nm.NM_I8)), dict(odt=2), dict(odt=-1), dict(X=P[0] + 1), dict(Y=P[2] + 1),
               dict(o=P[1] + 2), dict(o=P[1] + 4, odt=1), dict(T=(1 << 25) + 1),
               dict(w=_experts(E=1023, experts=1024, values_bytes=1 << 30, meta_bytes=1 << 30))):
        assert _el(**kw) == EUNSUP, kw
    big = _experts(E=1, R=(1 << 22) + 16, K=8)
    assert _el(w=big, ldx=8, ldy=1 << 23) == EUNSUP
    # more tiles than 32 bits count
    assert _el(w=_experts(E=1, R=1 << 22, K=8), ldx=8, ldy=1 << 22, T=1 << 25) == EUNSUP
    # copies of weights and of rows that the tiles do not read as they are
    monkeypatch.setenv("NM_FFN_TILE", "tile:1")
    dense = dict(T=1100, w=_experts(N=4, M=8))
    assert _el(**dense, ws=None) == EINVAL and _el(**dense, wsb=1000) == EINVAL
    assert _el(**dense, ws=P[3] + 16) == EUNSUP and _el(T=1100, X=P[0] + 2, ws=None) == EINVAL


def _eb(w=None, X=P[0], ldx=128, T=5, o=P[1], odt=0, dY=P[2], lddy=40, dX=P[3], lddx=128, fill=0, dW=P[4], lddw=128,
        ws=P[5], wsb=1 << 28):
    w = w or _experts()
    return nm.lib().nm_expert_linear_backward(ctypes.byref(w), X, ldx, T, o, odt, dY, lddy, dX, lddx, fill, dW, lddw, ws,
                                              wsb, None)


def test_expert_backward_refusals():
    for kw in (dict(X=None), dict(dY=None), dict(o=None), dict(dX=None, dW=None), dict(T=0), dict(ldx=127),
               dict(lddy=39), dict(lddx=127), dict(lddw=127), dict(ws=None), dict(wsb=100),
               dict(w=_experts(format_version=0))):
        assert _eb(**kw) == EINVAL, kw
    for kw in (dict(w=_experts(dt=nm.NM_I8)), dict(odt=5), dict(X=P[0] + 1), dict(dY=P[2] + 1), dict(dX=P[3] + 1),
               dict(dW=P[4] + 1), dict(ws=P[5] + 8), dict(o=P[1] + 1),
               dict(T=(1 << 25) + 1)):
        assert _eb(**kw) == EUNSUP, kw
    wide = _experts(E=64, R=1 << 16, K=1 << 15)
    assert _eb(w=wide, ldx=1 << 15, lddy=1 << 16, lddx=1 << 15, lddw=1 << 15, wsb=1 << 62) == EUNSUP
    n = ctypes.c_size_t()
    f = nm.lib().nm_expert_linear_backward_workspace_size
    w = _experts()
    assert f(ctypes.byref(w), 5, ctypes.byref(n)) == nm.NM_OK and n.value > 0
    assert f(ctypes.byref(w), 0, ctypes.byref(n)) == EINVAL and f(ctypes.byref(w), 5, None) == EINVAL
    assert f(ctypes.byref(_experts(dt=nm.NM_I8)), 5, ctypes.byref(n)) == EUNSUP


def test_i8_expert_refusals():
    def f(w=None, s=P[1], xq=None, X=P[0], ldx=128, xdt=nm.NM_F16, T=50, o=P[2], odt=0, Y=P[3], ldy=40, ydt=nm.NM_F16,
          bias=None, act=0, ws=P[4], wsb=1 << 28):
        w = w or _experts(dt=nm.NM_I8)
        return nm.lib().nm_i8_expert_linear(ctypes.byref(w), s, None if xq is None else ctypes.byref(xq), X, ldx, xdt, T,
                                            o, odt, Y, ldy, ydt, bias, act, 0, ws, wsb, None)

    for kw in (dict(s=None), dict(X=None), dict(o=None), dict(Y=None), dict(T=0), dict(ldx=127), dict(ldy=39),
               dict(ws=None), dict(wsb=10), dict(xq=_i8(49, 128)), dict(xq=_i8(50, 129)),
               dict(w=_experts(dt=nm.NM_I8, format_version=3))):
        assert f(**kw) == EINVAL, kw
    for kw in (dict(w=_experts()), dict(odt=7), dict(o=P[2] + 2), dict(act=2), dict(xdt=nm.NM_I32), dict(ydt=nm.NM_I8),
               dict(ws=P[4] + 128), dict(s=P[1] + 2)):
        assert f(**kw) == EUNSUP, kw
    n = ctypes.c_size_t()
    w = _experts(dt=nm.NM_I8)
    g = nm.lib().nm_i8_expert_linear_workspace_size
    assert g(ctypes.byref(w), None, 50, ctypes.byref(n)) == nm.NM_OK and n.value == 50 * 128 + 256
    # few rows: quantised inside the product
    assert g(ctypes.byref(w), None, 5, ctypes.byref(n)) == nm.NM_OK and n.value == 0
    assert g(ctypes.byref(w), ctypes.byref(_i8(5, 128)), 5, ctypes.byref(n)) == nm.NM_OK and n.value == 0
    assert g(ctypes.byref(_experts()), None, 5, ctypes.byref(n)) == EUNSUP


def _el_size(w, X, ldx, T):
    n = ctypes.c_size_t()
    assert nm.lib().nm_expert_linear_workspace_size(ctypes.byref(w), X, ldx, T, ctypes.byref(n)) == nm.NM_OK
    return n.value


@pytest.mark.parametrize("path", [None, "stream:1", "wide:0", "wide:1", "tile:0", "tile:2", "tile24:1", "tile24:3"])
@pytest.mark.parametrize("K,N,M", [(4, 2, 4), (8, 2, 4), (136, 4, 8), (132, 3, 4), (128, 1, 4), (2048, 4, 4)])
def test_expert_linear_workspace_covers_any_rows(monkeypatch, path, K, N, M):
    """What the query answers without rows is enough for rows of any address and stride."""
    if path:
        monkeypatch.setenv("NM_FFN_TILE", path)
    for E, R, T in ((3, 40, 5), (32, 1536, 4096), (2, 300, 700)):
        w = _experts(E=E, R=R, K=K, N=N, M=M)
        any_rows = _el_size(w, None, 0, T)
        for X in (P[0], P[0] + 2, P[0] + 8):
            for ldx in (K, K + 1, K + 8, 1 << 14, (1 << 22) - 8, 1 << 22, (1 << 22) + 1, 1 << 30):
                assert _el_size(w, X, ldx, T) <= any_rows, (E, R, T, X - P[0], ldx)
        # the stride given beside no rows is not read
        assert _el_size(w, None, 1 << 30, T) == any_rows


def test_backward_workspace_of_a_call():
    """The query for one call is what that call asks for, byte by byte, and no more than
    its parts: one byte less is refused, with all of them the misaligned workspace is."""
    L, n = nm.lib(), ctypes.c_size_t()

    def f(w, X=P[0], ldx=128, T=5, dY=P[2], lddy=40, dx=1, dw=1):
        return L.nm_expert_linear_backward_workspace_size_for(ctypes.byref(w), X, ldx, T, dY, lddy, dx, dw,
                                                              ctypes.byref(n))

    for K, R in ((128, 40), (132, 40), (128, 41), (196, 333)):
        w, T, Kp, Rp = _experts(K=K, R=R), 70, -(-K // 64) * 64, -(-R // 64) * 64
        wt, mask = 3 * -(-K // 16) * 16 * Rp * 2, 3 * -(-R // 128) * (Kp // 64) * 1024
        worst = ctypes.c_size_t()
        assert L.nm_expert_linear_backward_workspace_size(ctypes.byref(w), T, ctypes.byref(worst)) == nm.NM_OK
        for X, ldx in ((P[0], K), (P[0], K + 12), (P[0] + 2, K + 24), (P[0], 1 << 22)):
            for dY, lddy in ((P[2], R), (P[2], R + 15), (P[2] + 8, R)):
                px = (X - P[0]) % 16 or ldx % 8 or K % 8 or ldx >= 1 << 22
                py = (dY - P[2]) % 16 or lddy % 8 or R % 8
                for dx, dw in ((1, 1), (1, 0), (0, 1)):
                    assert f(w, X, ldx, T, dY, lddy, dx, dw) == nm.NM_OK
                    parts = [wt * dx, mask * dw, T * Kp * 2 * bool(dw and px), T * Rp * 2 * bool(py)]
                    assert n.value == sum(-(-v // 256) * 256 for v in parts) <= worst.value
                    call = dict(w=w, X=X, ldx=ldx, T=T, dY=dY, lddy=lddy, dX=P[3] if dx else None, lddx=K,
                                dW=P[4] if dw else None, lddw=K, ws=P[5] + 8)
                    assert _eb(**call, wsb=n.value - 1) == EINVAL and _eb(**call, wsb=n.value) == EUNSUP
    w = _experts()
    for kw in (dict(X=None), dict(dY=None), dict(ldx=127), dict(lddy=39), dict(T=0), dict(dx=0, dw=0)):
        assert f(w, **kw) == EINVAL, kw
    assert L.nm_expert_linear_backward_workspace_size_for(ctypes.byref(w), P[0], 128, 5, P[2], 40, 1, 1, None) == EINVAL
    assert f(_experts(dt=nm.NM_I8)) == EUNSUP and f(_experts(format_version=0)) == EINVAL


# ---------------------------------------------------------------- binding
def _packed_experts(E=2, R=16, K=64, N=2, M=4, dt=nm.NM_F16):
    v, m = nm.pack_size(R, K, N, M, dt)
    return nm.Experts(E, R, K, N, M, dt, torch.empty(E * v, dtype=torch.uint8),
                      torch.empty(E * m, dtype=torch.uint8) if m else None)


def test_binding_refuses_experts_operands():
    w, X, o = _packed_experts(), torch.zeros(3, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    for bad, err, text in ((X.bfloat16(), TypeError, "X has dtype"), (X[:, :63], ValueError, "X must be"),
                           (X[0], ValueError, "2-D"), (X[:1].expand(3, 64), ValueError, "overlapping rows")):
        with pytest.raises(err, match=text):
            nm.expert_linear(w, bad, o)
        with pytest.raises(err, match=text):
            nm.expert_linear_backward(w, bad, o, torch.zeros(3, 16, dtype=torch.float16))
    for bad, err, text in ((o[:2], ValueError, "offsets must be"), (o.short(), TypeError, "offsets must be int32"),
                           (torch.zeros(6, dtype=torch.int32)[::2], ValueError, "offsets must be")):
        with pytest.raises(err, match=text):
            nm.expert_linear(w, X, bad)
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.expert_linear(w, X, o)
    with pytest.raises(ValueError, match="out must be"):
        nm.expert_linear(w, X, o, out=torch.zeros(3, 15, dtype=torch.float16))
    with pytest.raises(TypeError, match="out has dtype"):
        nm.expert_linear(w, X, o, out=torch.zeros(3, 16))
    with pytest.raises(TypeError, match="takes float16 / bfloat16"):
        nm.expert_linear(_packed_experts(dt=nm.NM_I8), X, o)
    dY = torch.zeros(3, 16, dtype=torch.float16)
    with pytest.raises(ValueError, match="need_dx or need_dw"):
        nm.expert_linear_backward(w, X, o, dY, need_dx=False, need_dw=False)
    with pytest.raises(TypeError, match="dY has dtype"):
        nm.expert_linear_backward(w, X, o, dY.float())
    with pytest.raises(ValueError, match="dY must be"):
        nm.expert_linear_backward(w, X, o, dY[:2])
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.expert_linear_backward(w, X, o, dY)
    W = torch.zeros(2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="3-D"):
        nm.pack_experts(W[0], 2, 4)
    with pytest.raises(TypeError, match="unsupported weight dtype"):
        nm.pack_experts(W.float(), 2, 4)
    with pytest.raises(ValueError, match="no expert"):
        nm.pack_experts(W[:0], 2, 4)
    with pytest.raises(ValueError, match="unit stride"):
        nm.pack_experts(W.transpose(1, 2), 2, 4)
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.pack_experts(W, 2, 4)


def test_binding_refuses_i8_operands():
    p = nm.Packed(16, 64, 2, 4, nm.NM_I8, *(torch.empty(n, dtype=torch.uint8) for n in nm.pack_size(16, 64, 2, 4, nm.NM_I8)))
    X, s = torch.zeros(3, 64), torch.ones(16)
    with pytest.raises(TypeError, match="X must be float16"):
        nm.i8_quantize(X.double())
    with pytest.raises(ValueError, match="2-D"):
        nm.i8_quantize(X[0])
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.i8_quantize(X)
    q = nm.I8(3, 64, torch.zeros(3, 128, dtype=torch.int8), torch.ones(3))
    assert q.values.shape == (3, 64) and q.nbytes() == 3 * 132
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.i8_dequantize(q)
    with pytest.raises(TypeError, match="takes int8 weights"):
        nm.i8_linear(nm.Packed(16, 64, 2, 4, nm.NM_F16, p.values, p.meta), s, X)
    for kw, err, text in ((dict(w_scale=s[:15]), ValueError, "w_scale must be"),
                          (dict(w_scale=s.half()), TypeError, "w_scale has dtype"),
                          (dict(w_scale=torch.ones(32)[::2]), ValueError, "w_scale must be"),
                          (dict(bias=s[:15]), ValueError, "bias must be"), (dict(act="silu"), ValueError, "act must be"),
                          (dict(X=X[:, :60]), ValueError, "X must be"),
                          (dict(X=X.to(torch.int8)), TypeError, "X must be float16"),
                          (dict(out_dtype=torch.int32), TypeError, "out must be float16"),
                          (dict(out=torch.zeros(3, 16), out_dtype=torch.float16), TypeError, "out has dtype"),
                          (dict(X=nm.I8(3, 32, q.codes, q.scales)), ValueError, "has K=32"),
                          (dict(), ValueError, "not on a GPU"), (dict(X=q), ValueError, "not on a GPU")):
        with pytest.raises(err, match=text):
            nm.i8_linear(p, **{"w_scale": s, "X": X, **kw})
    w, o = _packed_experts(dt=nm.NM_I8), torch.zeros(3, dtype=torch.int32)
    for kw, err, text in ((dict(w_scale=s), ValueError, "w_scale must be"), (dict(offsets=o[:2]), ValueError, "offsets"),
                          (dict(bias=s), ValueError, "bias must be"), (dict(), ValueError, "not on a GPU")):
        with pytest.raises(err, match=text):
            nm.i8_expert_linear(w, **{"w_scale": torch.ones(2, 16), "X": X, "offsets": o, **kw})


# ---------------------------------------------------------------- the 64-bit forms
def test_i8_definition():
    x = torch.tensor([[127.0, 63.5, -0.5, 1.5, 2.5, -126.5], [0.0] * 6, [float("inf"), 1, 1, 1, 1, 1]])
    q, s = i8_64(x)
    assert s[0] == 1 and s[1] == 2.0 ** -126 and s[2].isnan()
    assert q.tolist() == [[127, 64, 0, 2, 2, -126], [0] * 6, [0] * 6]


def test_offsets_as_read():
    assert experts_of(torch.tensor([-7, 5, 3, 80, 20, 10]), 60) == ([(0, 5), (5, 5), (5, 60), (60, 60), (60, 60)], [])
    assert experts_of(torch.tensor([2, 4, 4, 6]), 8) == ([(2, 4), (4, 4), (4, 6)], [0, 1, 6, 7])


def test_binding_refuses_buffers_of_other_types_and_strides():
    """What an I8 or Experts holds may be replaced by its user; the library gets addresses
    only, so 16-bit scales would be read past their end and strided codes as others."""
    p = nm.Packed(16, 64, 2, 4, nm.NM_I8, *(torch.empty(n, dtype=torch.uint8) for n in nm.pack_size(16, 64, 2, 4, nm.NM_I8)))
    s, codes, scales = torch.ones(16), torch.zeros(3, 128, dtype=torch.int8), torch.ones(3)
    for q, err, text in ((nm.I8(3, 64, codes, scales.half()), TypeError, "scales has dtype"),
                         (nm.I8(3, 64, codes, torch.ones(6)[::2]), ValueError, "scales must be contiguous"),
                         (nm.I8(3, 64, codes.to(torch.int16), scales), TypeError, "codes has dtype"),
                         (nm.I8(3, 64, torch.zeros(6, 128, dtype=torch.int8)[::2], scales), ValueError, "codes must be")):
        with pytest.raises(err, match=text):
            nm.i8_linear(p, s, q)
        with pytest.raises(err, match=text):
            nm.i8_expert_linear(_packed_experts(dt=nm.NM_I8), torch.ones(2, 16), q, torch.zeros(3, dtype=torch.int32))
    # replaced after a call that was fine, the same address and length
    q = nm.I8(3, 64, torch.zeros(6, 128, dtype=torch.int8), scales)
    all6, q.codes = q.codes, q.codes[:3]
    with pytest.raises(ValueError, match="not on a GPU"):
        nm.i8_linear(p, s, q)
    q.codes = all6[::2]
    with pytest.raises(ValueError, match="codes must be contiguous"):
        nm.i8_linear(p, s, q)
    X, o = torch.zeros(3, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    for name in ("values", "meta"):
        w = _packed_experts()
        t = getattr(w, name)
        for bad, err, text in ((t.to(torch.int16), TypeError, f"{name} has dtype"),
                               (torch.empty(2 * t.numel(), dtype=torch.uint8)[::2], ValueError, f"{name} must be contig")):
            setattr(w, name, bad)
            with pytest.raises(err, match=text):
                nm.expert_linear_workspace_size(w, 3)
