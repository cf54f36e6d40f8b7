"""The feed-forward operators on the GPU against their plain 64-bit forms
(tests/_ffn.py, which derives the elementwise bounds): the gated block on N:M
packed weights, its gradients, the microscaled 4-bit format, its product and
its gated block."""
import copy
import pickle
import zlib

import pytest
import torch

import semi_structured_sparse_nm_amd as nm
from tests import _ffn
from tests._ffn import TORCH, check

pytestmark = pytest.mark.gpu


def _gen(*key):
    g = torch.Generator()
    g.manual_seed(zlib.crc32(repr(key).encode()))
    return g


def normal(shape, std, dt, *key):
    return (torch.randn(*shape, generator=_gen(*key)) * std).to(TORCH[dt]).cuda()


def wide(t, pad, fill=0.0):
    """t as a slice of a buffer with `pad` more columns, filled with `fill`."""
    b = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b, b[:, :t.shape[1]]


def weights(R, K, N, M, dt, *key):
    """(packed, masked dense, mask) of one seeded weight."""
    W = normal((R, K), 0.05, dt, "W", R, K, *key)
    k = _ffn.kept(W, N, M)
    return nm.pack(W, N, M), torch.where(k, W, torch.zeros_like(W)), k


# one token to several tiles; rows and columns inside and past 16, 64, 128
SHAPES = [(1, 1, 8), (1, 16, 64), (2, 17, 72), (15, 40, 264), (16, 130, 512), (17, 33, 64), (31, 64, 1032),
          (33, 48, 128), (64, 129, 200), (65, 128, 64), (66, 1, 8), (128, 200, 128), (129, 65, 136), (300, 500, 712)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,R,K", SHAPES)
def test_glu_shapes(T, R, K, dt):
    pg, wg, _ = weights(R, K, 2, 4, dt, "g")
    pu, wu, _ = weights(R, K, 2, 4, dt, "u")
    X = normal((T, K), 1.0, dt, "X", T, K)
    for act in ("silu", "gelu"):
        h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, act)
        pre = torch.full((2, T, R), 7.0, dtype=X.dtype, device="cuda")
        H = nm.glu(pg, pu, X, act=act, pre=pre)
        check(H, h, eh, f"H {act}")
        check(pre[0], g, eg, "G")
        check(pre[1], u, eu, "U")
        assert torch.equal(nm.glu(pg, pu, X, act=act), H), "the call without pre differs"


@pytest.mark.parametrize("N,M", [(1, 4), (3, 4), (4, 4), (1, 8), (2, 8), (3, 8), (4, 8), (5, 8), (6, 8), (7, 8),
                                 (8, 8)])
@pytest.mark.parametrize("T,R,K", [(1, 33, 72), (20, 48, 328), (50, 17, 64), (90, 70, 136)])
def test_glu_patterns(T, R, K, N, M):
    dt = "f16" if N % 2 else "bf16"
    pg, wg, kg = weights(R, K, N, M, dt, "g", N)
    pu, wu, ku = weights(R, K, N, M, dt, "u", N)
    X = normal((T, K), 1.0, dt, "X", T, K, N)
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, "silu")
    pre = torch.empty((2, T, R), dtype=X.dtype, device="cuda")
    check(nm.glu(pg, pu, X, pre=pre), h, eh, "H")
    dH = normal((T, R), 0.1, dt, "dH", T, R, N)
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
    for a, b, e, what in zip(nm.glu_backward(pg, pu, X, pre, dH), want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


@pytest.mark.parametrize("T,R,K", [(5, 20, 12), (70, 40, 100), (3, 64, 64), (80, 64, 64)])
@pytest.mark.parametrize("xpad,ypad", [(0, 3), (5, 0), (8, 4), (1, 1)])
def test_glu_strides(T, R, K, xpad, ypad):
    """Rows whose pitch or length is no multiple of 16 bytes, an activation
    buffer whose other columns hold NaN, outputs inside wider buffers."""
    pg, wg, kg = weights(R, K, 2, 4, "f16", "g")
    pu, wu, ku = weights(R, K, 2, 4, "f16", "u")
    X = normal((T, K), 1.0, "f16", "X", T, K)
    _, xv = wide(X, xpad, float("nan"))
    hb, hv = wide(torch.zeros(T, R, dtype=X.dtype, device="cuda"), ypad, 5.0)
    pb = torch.full((2, T, R + ypad), 5.0, dtype=X.dtype, device="cuda")
    pre = pb[:, :, :R]
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, "silu")
    assert nm.glu(pg, pu, xv, out=hv, pre=pre) is hv
    check(hv, h, eh, "H")
    check(pre[0], g, eg, "G")
    assert bool((hb[:, R:] == 5.0).all()) and bool((pb[:, :, R:] == 5.0).all())
    dH = normal((T, R), 0.1, "f16", "dH", T, R)
    _, dv = wide(dH, ypad, float("nan"))
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
    for a, b, e, what in zip(nm.glu_backward(pg, pu, xv, pre, dv), want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


@pytest.mark.parametrize("T,R,K,dt", [(1, 1, 8, "f16"), (3, 17, 72, "bf16"), (64, 64, 64, "f16"), (65, 130, 200, "bf16"),
                                      (197, 200, 768, "f16"), (300, 520, 264, "bf16")])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_backward_shapes(T, R, K, dt, act):
    pg, wg, kg = weights(R, K, 2, 4, dt, "g")
    pu, wu, ku = weights(R, K, 2, 4, dt, "u")
    X = normal((T, K), 1.0, dt, "X", T, K)
    dH = normal((T, R), 0.1, dt, "dH", T, R)
    pre = torch.empty((2, T, R), dtype=X.dtype, device="cuda")
    nm.glu(pg, pu, X, act=act, pre=pre)
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, act)
    got = nm.glu_backward(pg, pu, X, pre, dH, act=act)
    for a, b, e, k, what in zip(got, want, bound, (None, kg, ku), ("dX", "dWg", "dWu")):
        check(a, b, e, what)
        if k is not None:
            assert bool((a[~k] == 0).all()), f"{what} is not zero where the weight is pruned"
    dx, none_g, none_u = nm.glu_backward(pg, pu, X, pre, dH, act=act, need_dw=False)
    assert none_g is None and none_u is None and torch.equal(dx, got[0])
    no_dx, dwg, dwu = nm.glu_backward(pg, pu, X, pre, dH, act=act, need_dx=False)
    assert no_dx is None and torch.equal(dwg, got[1]) and torch.equal(dwu, got[2])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_backward_against_differences(act):
    """<dX, v> and <dWg, V> against central differences of
    L = sum dH act(G) U, G and U moving linearly from the kept products: the
    difference quotient's own error is below 1e-7 relative at this step."""
    T, R, K, dt = 40, 96, 136, "f16"
    pg, wg, kg = weights(R, K, 2, 4, dt, "g")
    pu, wu, ku = weights(R, K, 2, 4, dt, "u")
    X = normal((T, K), 1.0, dt, "X")
    dH = normal((T, R), 0.1, dt, "dH")
    pre = torch.empty((2, T, R), dtype=X.dtype, device="cuda")
    nm.glu(pg, pu, X, act=act, pre=pre)
    g, u, dh = pre[0].double(), pre[1].double(), dH.double()
    dx, dwg, dwu = nm.glu_backward(pg, pu, X, pre, dH, act=act)
    _, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, act)
    v = normal((T, K), 1.0, "f32", "v").double()
    V = normal((R, K), 1.0, "f32", "V").double()

    def loss(sg, su):
        return float((dh * _ffn.act64(g + sg, act) * (u + su)).sum())

    e = 1e-4
    moves = [(v @ wg.double().t(), v @ wu.double().t(), dx, v, bound[0]),
             (X.double() @ (V * kg).t(), 0.0, dwg, V * kg, bound[1]),
             (0.0, X.double() @ (V * ku).t(), dwu, V * ku, bound[2])]
    for mg, mu, grad, d, b in moves:
        quot = (loss(e * mg, e * mu) - loss(-e * mg, -e * mu)) / (2 * e)
        lim = (d.abs() * (b + _ffn.half_step(grad.dtype) * grad.double().abs() + _ffn.tiny(grad.dtype))).sum()
        scale = (d * grad.double()).abs().sum()
        assert abs(quot - float((grad.double() * d).sum())) <= float(lim) + 1e-6 * float(scale)


@pytest.mark.parametrize("N,M", [(2, 4), (4, 8), (1, 4), (8, 8)])
@pytest.mark.parametrize("T", [3, 40, 90, 300])
@pytest.mark.parametrize("stream", [0, 1])
def test_glu_tokens_are_independent(tile, stream, T, N, M):
    """Infinite and NaN activations change no other token's bits."""
    tile("stream", stream)
    R, K = 150, 200
    pg, pu = weights(R, K, N, M, "bf16", "g")[0], weights(R, K, N, M, "bf16", "u")[0]
    X = normal((T, K), 1.0, "bf16", "X", T)
    pre = torch.empty(2, T, R, dtype=X.dtype, device="cuda")
    clean = nm.glu(pg, pu, X, pre=pre).clone(), pre.clone()
    rows = torch.ones(T, dtype=torch.bool)
    for t, v in ((0, float("inf")), (T - 1, float("nan")), (T // 2, float("-inf"))):
        X[t, (7 * t) % K] = v
        rows[t] = False
    H = nm.glu(pg, pu, X, pre=pre)
    assert torch.equal(H[rows], clean[0][rows]) and torch.equal(pre[:, rows], clean[1][:, rows])
    assert not bool(torch.isfinite(H[T - 1]).all())


@pytest.mark.parametrize("N,M", [(2, 4), (3, 8), (1, 4)])
@pytest.mark.parametrize("T", [1, 33, 130])
def test_glu_layouts(T, N, M):
    """Rows at odd addresses, the two products in turn by token, gradients
    from strided operands, one token in a wide buffer."""
    R, K, dt = 77, 130 if M == 4 else 136, "f16"
    K = K // M * M
    pg, wg, kg = weights(R, K, N, M, dt, "g")
    pu, wu, ku = weights(R, K, N, M, dt, "u")
    X = normal((T, K), 1.0, dt, "X", T, N)
    flat = torch.full((T * (K + 9) + 1,), float("nan"), dtype=X.dtype, device="cuda")
    xv = flat[1:].view(T, K + 9)[:, :K]
    xv.copy_(X)
    both = torch.empty(T, 2, R, dtype=X.dtype, device="cuda")
    pre = both.transpose(0, 1)
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, "silu")
    check(nm.glu(pg, pu, xv, pre=pre), h, eh, "H")
    check(both[:, 0], g, eg, "G")
    check(both[:, 1], u, eu, "U")
    dH = normal((R, T), 0.1, dt, "dH", T, N).t().contiguous()
    db = torch.full((T, R + 3), float("nan"), dtype=X.dtype, device="cuda")
    db[:, 3:] = dH
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
    for a, b, e, what in zip(nm.glu_backward(pg, pu, xv, pre, db[:, 3:]), want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


def test_weights_of_zeros_and_saturated_gates():
    """Products of zero, and gates at the ends of the activation's range."""
    T, R, K = 70, 32, 64
    z = nm.pack(torch.zeros(R, K, dtype=torch.bfloat16, device="cuda"), 2, 4)
    w = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1.0
    p = nm.pack(w, 2, 4)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = torch.linspace(-3e4, 3e4, T)
    for act in ("silu", "gelu"):
        for n in (1, 20, T):
            assert bool((nm.glu(z, p, X[:n], act=act) == 0).all()) and bool((nm.glu(p, z, X[:n], act=act) == 0).all())
            h, _, _, eh, _, _ = _ffn.glu64(X[:n], w, w, act)
            check(nm.glu(p, p, X[:n], act=act), h, eh, act)
        pre = torch.empty(2, T, R, dtype=X.dtype, device="cuda")
        nm.glu(p, p, X, act=act, pre=pre)
        k = torch.zeros_like(w, dtype=torch.bool)
        k[:, 0:2] = True
        k[:, 4::4] = k[:, 5::4] = True
        dH = torch.ones(T, R, dtype=X.dtype, device="cuda")
        want, bound = _ffn.glu_grad64(X, w, w, k, k, pre, dH, act)
        for a, b, e, what in zip(nm.glu_backward(p, p, X, pre, dH, act=act), want, bound, ("dX", "dWg", "dWu")):
            check(a, b, e, what)


@pytest.mark.parametrize("N,M", [(2, 4), (4, 8)])
@pytest.mark.parametrize("T", [1, 20, 70, 193])
def test_silu_of_far_negative_gates(tile, T, N, M):
    """Gates from -80 to -104, where SiLU leaves the normal numbers but not
    the type, times factors from 1 to 2^40; and their gradients."""
    R, K = 20, 64
    wg, wu = torch.zeros(2, R, K, dtype=torch.bfloat16, device="cuda")
    wg[:, 0] = 1.0
    wu[:, 33] = torch.exp2(torch.arange(R, device="cuda") * 2.0)
    kg, ku = _ffn.kept(wg, N, M), _ffn.kept(wu, N, M)
    pg, pu = nm.pack(wg, N, M), nm.pack(wu, N, M)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = torch.linspace(-80, -104, 193)[-T:]
    X[:, 33] = 1.0
    h, _, _, eh, _, _ = _ffn.glu64(X, wg, wu, "silu")
    dH = torch.ones(T, R, dtype=X.dtype, device="cuda")
    for stream in (0, 1):
        tile("stream", stream)
        pre = torch.empty(2, T, R, dtype=X.dtype, device="cuda")
        check(nm.glu(pg, pu, X, pre=pre), h, eh, f"H {stream}")
        want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
        dx, dwg, dwu = nm.glu_backward(pg, pu, X, pre, dH)
        for a, b, e, what in zip((dx, dwg, dwu), want, bound, ("dX", "dWg", "dWu")):
            check(a, b, e, what)
        # dWu's column 33 sums dU = SiLU(G): 2^-9 of it for dU's rounding, 2^-9 for its own, 2^-14 for the rest
        want = _ffn.act64(pre[0].double(), "silu").sum(0)
        assert bool(((dwu[:, 33].double() - want).abs() <= want.abs() * 2.0 ** -7.9 + T * _ffn.tiny(X.dtype)).all())


@pytest.mark.parametrize("T", [1, 16, 40, 100])
def test_mx_silu_of_far_negative_gates(tile, T):
    """The same at 4 bits: gates of -96 and -64, every path."""
    R, K = 20, 64
    W = torch.zeros(2, R, K, dtype=torch.bfloat16, device="cuda")
    W[0, :, 0] = 1.0
    W[1, :, 33] = torch.exp2(torch.arange(R, device="cuda") * 2.0)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = torch.tensor([-96.0, -64.0], device="cuda").repeat(T)[:T]
    X[:, 33] = 1.0
    h, _, _, eh, _, _ = _ffn.glu64(X, W[0], W[1], "silu")
    wg, wu = nm.mx_quantize(W[0]), nm.mx_quantize(W[1])
    for stream in (0, 1):
        tile("stream", stream)
        check(nm.mx_glu(wg, wu, X), h, eh, f"H {stream}")


def test_packed_weights_copy_and_pickle():
    """A weight that has been used copies and pickles like one that has not."""
    pg, pu = weights(16, 64, 2, 4, "f16", "g")[0], weights(16, 64, 2, 4, "f16", "u")[0]
    w = _mx_w(16, 64, "f16")[0]
    X = normal((3, 64), 1.0, "f16", "X")
    H, Y = nm.glu(pg, pu, X), nm.mx_linear(w, X)
    for f in (copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p))):
        assert torch.equal(nm.glu(f(pg), f(pu), X), H) and torch.equal(nm.mx_linear(f(w), X), Y)
    other = weights(16, 64, 2, 4, "f16", "other")[0]
    pg.values, pg.meta = other.values, other.meta             # a field that changes is seen
    assert torch.equal(nm.glu(pg, pu, X), nm.glu(other, pu, X))


def test_workspaces():
    """A workspace that is larger or smaller than needed, shared by calls in
    order, and by two graphs replayed in order."""
    T, R, K, dt = 130, 200, 264, "bf16"
    pg, pu = weights(R, K, 4, 8, dt, "g")[0], weights(R, K, 4, 8, dt, "u")[0]
    w = _mx_w(R, K, dt)[0]
    X, dH = normal((T, K), 1.0, dt, "X"), normal((T, R), 0.1, dt, "dH")
    pre = torch.empty(2, T, R, dtype=X.dtype, device="cuda")

    def forward(ws=None):
        return nm.glu(pg, pu, X, pre=pre, workspace=ws), nm.mx_linear(w, X, workspace=ws)

    def backward(ws=None):
        return nm.glu_backward(pg, pu, X, pre, dH, workspace=ws)

    want = forward(), backward()
    need = max(nm.glu_workspace_size(pg, pu, T), nm.mx_workspace_size(w, T), nm.glu_backward_workspace_size(pg, pu, T))
    big = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    for ws in (big, big[:need], torch.empty(64, dtype=torch.uint8, device="cuda")):
        for got, ref in zip((forward(ws), backward(ws)), want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert bool((big[need:] == 0xAB).all())
    with pytest.raises(nm.NmError):
        backward(big[8:])                                     # not 256-byte aligned
    with pytest.raises(ValueError, match="contiguous"):
        forward(big[::2])
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        fa = forward(big)
    with torch.cuda.graph(gb):
        bb = backward(big)
    for i in range(3):
        X.copy_(normal((T, K), 1.0, dt, "X", i))
        ga.replay()
        gb.replay()
        got = [t.clone() for t in (*fa, *bb)]
        torch.cuda.synchronize()
        for a, b in zip(got, (*forward(), *backward())):
            assert torch.equal(a, b), f"replay {i}"


@pytest.fixture
def tile(monkeypatch):
    """Forces a tile shape (and split) of the feed-forward products."""
    def force(kind, shape, split=0):
        monkeypatch.setenv("NM_FFN_TILE", f"{kind}:{shape}" + (f":{split}" if split else ""))
        nm._ws_sizes.clear()
    yield force
    nm._ws_sizes.clear()


def test_forced_path_after_a_call(monkeypatch):
    """A path forced between calls gets the workspace it needs: dense copies
    (4:8 by tiles) after streamed weights, which need none, and back."""
    T, R, K, dt = 40, 96, 264, "bf16"
    pg, wg, _ = weights(R, K, 4, 8, dt, "g")
    pu, wu, _ = weights(R, K, 4, 8, dt, "u")
    w, W = _mx_w(R, K, dt)
    X = normal((T, K), 1.0, dt, "X")
    h, _, _, eh, _, _ = _ffn.glu64(X, wg, wu, "silu")
    x = _ffn.mx64(X)[0]
    y, e = x @ W.t(), _ffn.sum_err(K, x.abs() @ W.abs().t())
    monkeypatch.delenv("NM_FFN_TILE", raising=False)
    for forced in (None, "stream:0", "stream:1", "tile:3:2", None):
        if forced is None:
            monkeypatch.delenv("NM_FFN_TILE", raising=False)
        else:
            monkeypatch.setenv("NM_FFN_TILE", forced)
        check(nm.glu(pg, pu, X), h, eh, f"H {forced}")
        check(nm.mx_linear(w, X), y, e, f"Y {forced}")


# tokens, rows, columns: several tiles a workgroup, the last ragged both ways
TILES = {0: (2100, 4200), 1: (1100, 3900), 2: (1100, 4300), 3: (700, 3700)}


@pytest.mark.parametrize("N,M", [(2, 4), (4, 8)])
@pytest.mark.parametrize("K", [64, 72, 456])
@pytest.mark.parametrize("shape", [0, 1, 2, 3])
def test_glu_tile_shapes(tile, shape, K, N, M):
    """Every shape of the sparse and the dense tile product with more tiles
    than compute units: one slab, a slab and a piece, several."""
    dt = "bf16" if K == 72 else "f16"
    T, R = TILES[shape] if (N, M) == (4, 8) else {0: (2100, 4200), 1: (1100, 4300), 2: (1100, 2300), 3: (700, 1900)}[shape]
    pg, wg, kg = weights(R, K, N, M, dt, "g")
    pu, wu, ku = weights(R, K, N, M, dt, "u")
    X = normal((T, K), 1.0, dt, "X", T, K)
    tile("tile24" if (N, M) == (2, 4) else "tile", shape)
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, "silu")
    pre = torch.full((2, T, R), 7.0, dtype=X.dtype, device="cuda")
    check(nm.glu(pg, pu, X, pre=pre), h, eh, "H")
    check(pre[0], g, eg, "G")
    check(pre[1], u, eu, "U")


@pytest.mark.parametrize("N,M", [(2, 4), (3, 4), (4, 4), (1, 8), (4, 8), (7, 8)])
@pytest.mark.parametrize("T,R,K", [(1, 300, 1032), (17, 150, 520), (33, 40, 64), (64, 130, 200), (65, 16, 1096),
                                   (130, 333, 584), (1024, 40, 72)])
@pytest.mark.parametrize("stream", [0, 1])
def test_glu_streamed_and_not(tile, stream, T, R, K, N, M):
    """Both ways of every pattern: one to eight groups of tokens, the last short."""
    dt = "f16" if T % 2 else "bf16"
    pg, wg, _ = weights(R, K, N, M, dt, "g", N)
    pu, wu, _ = weights(R, K, N, M, dt, "u", N)
    X = normal((T, K), 1.0, dt, "X", T, K)
    tile("stream", stream)
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, "gelu")
    pre = torch.full((2, T, R), 7.0, dtype=X.dtype, device="cuda")
    check(nm.glu(pg, pu, X, act="gelu", pre=pre), h, eh, "H")
    check(pre[0], g, eg, "G")
    check(pre[1], u, eu, "U")


@pytest.mark.parametrize("N,M", [(2, 4), (3, 4)])
@pytest.mark.parametrize("T,K,xpad", [(1, 4, 0), (1, 12, 0), (20, 60, 0), (33, 68, 1), (70, 100, 3), (100, 516, 0),
                                      (7, 1020, 2), (65, 64, 5)])
def test_glu_streamed_rows_of_any_width(tile, T, K, xpad, N, M):
    """Rows whose last piece is short, at every alignment; the next row and the
    columns between rows hold NaN."""
    R, dt = 50, "bf16"
    pg, wg, _ = weights(R, K, N, M, dt, "g", N)
    pu, wu, _ = weights(R, K, N, M, dt, "u", N)
    X = normal((T, K), 1.0, dt, "X", T, K)
    flat = torch.full((1 + T * (K + xpad) + 9,), float("nan"), dtype=X.dtype, device="cuda")
    xv = flat[1:1 + T * (K + xpad)].view(T, K + xpad)[:, :K]
    xv.copy_(X)
    tile("stream", 1)
    h, _, _, eh, _, _ = _ffn.glu64(X, wg, wu, "silu")
    check(nm.glu(pg, pu, xv), h, eh, "H")


@pytest.mark.parametrize("split", [1, 3])
@pytest.mark.parametrize("shape", [0, 1, 2, 3])
def test_glu_backward_tile_shapes(tile, shape, split):
    T, R, K, dt = 1100, 700, 1032, "bf16"
    if shape == 0:
        R, K = 2300, 2312
    pg, wg, kg = weights(R, K, 2, 4, dt, "g")
    pu, wu, ku = weights(R, K, 2, 4, dt, "u")
    X, dH = normal((T, K), 1.0, dt, "X"), normal((T, R), 0.1, dt, "dH")
    pre = normal((2 * T, R), 1.0, dt, "pre").view(2, T, R)
    tile("tile", shape, split)
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
    for a, b, e, what in zip(nm.glu_backward(pg, pu, X, pre, dH), want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


def test_glu_offsets_past_32_bits():
    """Outputs and activations of more than 2^32 bytes: the last rows."""
    dt = "bf16"
    for T, R, K in ((70000, 32768, 64), (140000, 64, 16384)):
        pg, wg, _ = weights(R, K, 2, 4, dt, "g")
        pu, wu, _ = weights(R, K, 2, 4, dt, "u")
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        X = torch.empty(T, K, dtype=TORCH[dt], device="cuda").normal_(generator=g)
        H = nm.glu(pg, pu, X)
        for rows in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
            h, _, _, eh, _, _ = _ffn.glu64(X[rows], wg, wu, "silu")
            check(H[rows], h, eh, f"H {rows}")
        del X, H


def test_glu_large_tiles():
    """Enough tiles for the largest tile shape, ragged on every side."""
    T, R, K, dt = 1000, 6500, 136, "bf16"
    pg, wg, kg = weights(R, K, 2, 4, dt, "g")
    pu, wu, ku = weights(R, K, 2, 4, dt, "u")
    X = normal((T, K), 1.0, dt, "X")
    h, _, _, eh, _, _ = _ffn.glu64(X, wg, wu, "silu")
    pre = torch.empty((2, T, R), dtype=X.dtype, device="cuda")
    check(nm.glu(pg, pu, X, pre=pre), h, eh, "H")
    dH = normal((T, R), 0.1, dt, "dH")
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
    for a, b, e, what in zip(nm.glu_backward(pg, pu, X, pre, dH), want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


def test_glu_backward_keeps_pruned_gradients_zero():
    """An infinite activation and a NaN in dH reach kept weights' gradients
    only; a kept weight of value zero gets its gradient."""
    T, R, K = 70, 32, 64
    W = normal((R, K), 0.05, "f16", "W")
    W[3] = 0.0                                            # ties: positions 0 and 1 are kept
    pg = pu = nm.pack(W, 2, 4)
    k = _ffn.kept(W, 2, 4)
    X = normal((T, K), 1.0, "f16", "X")
    pre = torch.empty((2, T, R), dtype=X.dtype, device="cuda")
    nm.glu(pg, pu, X, pre=pre)
    dH = normal((T, R), 0.1, "f16", "dH")
    pre[1, :, 3] = 1.0                                    # dG of row 3 is not zero
    _, dwg, _ = nm.glu_backward(pg, pu, X, pre, dH)
    assert bool((dwg[3][k[3]] != 0).all()) and bool((dwg[3][~k[3]] == 0).all())
    X[5, :] = float("inf")
    dH[7, 4] = float("nan")
    _, dwg, dwu = nm.glu_backward(pg, pu, X, pre, dH)
    for d in (dwg, dwu):
        assert bool((d[~k] == 0).all()), "a pruned weight got a gradient"
        assert bool(torch.isnan(d[4][k[4]]).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,R,K,N,M", [(40, 512, 256, 2, 4), (197, 1000, 768, 4, 8), (512, 700, 520, 3, 4)])
def test_training_step_against_unrounded_gradients(T, R, K, N, M, dt, act):
    """Forward and backward against gradients in 64 bits from the inputs alone.
    A rounding is off by at most half a step h of the value, evenly spread: at
    most h / sqrt(3) as a norm.  dWg and dX's gate part have four (U, dG, the
    output, and G through the slope's change, whose norm is below the slope's),
    dWu and dX's up part three (dU, the output, and G, times at most 1.4): less
    than 2 h / sqrt(3) together.  binary32 sums add nothing to that."""
    pg, wg, kg = weights(R, K, N, M, dt, "g")
    pu, wu, ku = weights(R, K, N, M, dt, "u")
    X, dH = normal((T, K), 1.0, dt, "X", T), normal((T, R), 0.1, dt, "dH", T)
    pre = torch.empty((2, T, R), dtype=X.dtype, device="cuda")
    nm.glu(pg, pu, X, act=act, pre=pre)
    got = nm.glu_backward(pg, pu, X, pre, dH, act=act)
    x, g, u, dh = X.double(), X.double() @ wg.double().t(), X.double() @ wu.double().t(), dH.double()
    dg, du = dh * u * _ffn.slope64(g, act), dh * _ffn.act64(g, act)
    want = (dg @ wg.double() + du @ wu.double(), (dg.t() @ x) * kg, (du.t() @ x) * ku)
    lim = 2 * _ffn.half_step(X.dtype) / 3 ** 0.5
    for a, b, what in zip(got, want, ("dX", "dWg", "dWu")):
        off = float((a.double() - b).norm() / b.norm())
        assert off <= lim, f"{what}: {off:.6f} of the norm, at most {lim:.6f}"


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,R,K,N,M", [(40, 512, 256, 2, 4), (197, 1000, 768, 4, 8), (512, 700, 520, 3, 4)])
def test_training_step_with_products_in_float32(T, R, K, N, M, dt, act):
    """The same with G and U kept in float32: two roundings are left (dG or dU,
    and the output), at most h sqrt(2 / 3) together."""
    pg, wg, kg = weights(R, K, N, M, dt, "g")
    pu, wu, ku = weights(R, K, N, M, dt, "u")
    X, dH = normal((T, K), 1.0, dt, "X", T), normal((T, R), 0.1, dt, "dH", T)
    pre = torch.empty((2, T, R), device="cuda")
    H = nm.glu(pg, pu, X, act=act, pre=pre)
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, act)
    check(H, h, eh, "H")
    check(pre[0], g, eg, "G")
    check(pre[1], u, eu, "U")
    got = nm.glu_backward(pg, pu, X, pre, dH, act=act)
    dh = dH.double()
    dg, du = dh * u * _ffn.slope64(g, act), dh * _ffn.act64(g, act)
    want = (dg @ wg.double() + du @ wu.double(), (dg.t() @ X.double()) * kg, (du.t() @ X.double()) * ku)
    lim = _ffn.half_step(X.dtype) * (2 / 3) ** 0.5
    for a, b, what in zip(got, want, ("dX", "dWg", "dWu")):
        off = float((a.double() - b).norm() / b.norm())
        assert off <= lim, f"{what}: {off:.6f} of the norm, at most {lim:.6f}"
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, act)
    for a, b, e, what in zip(got, want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,R,K,N,M", [(1, 200, 136, 2, 4), (6, 92, 592, 2, 4), (24, 149, 72, 4, 8), (65, 130, 264, 3, 4),
                                       (128, 512, 512, 2, 4), (1000, 64, 1048, 1, 8), (1100, 64, 1048, 1, 8)])
def test_small_steps_leave_the_output_rounding_alone(T, R, K, N, M, dt, act):
    """Up to 2^26 multiply-adds and float32 products: dG and dU come in two
    parts, off by h^2 of the value (fp16: h 2^-14 absolutely, where the second
    is below its normal numbers), so what is left is one rounding of exact
    gradients: elementwise half a step and the sums' error."""
    pg, wg, kg = weights(R, K, N, M, dt, "g")
    pu, wu, ku = weights(R, K, N, M, dt, "u")
    X, dH = normal((T, K), 1.0, dt, "X", T), normal((T, R), 0.1, dt, "dH", T)
    pre = torch.empty((2, T, R), device="cuda")
    nm.glu(pg, pu, X, act=act, pre=pre)
    got = nm.glu_backward(pg, pu, X, pre, dH, act=act)
    g, u, dh, x = pre[0].double(), pre[1].double(), dH.double(), X.double()
    dg, du = dh * u * _ffn.slope64(g, act), dh * _ffn.act64(g, act)
    want = (dg @ wg.double() + du @ wu.double(), (dg.t() @ x) * kg, (du.t() @ x) * ku)
    if T * R * K > 2 ** 26:                               # one part: the bound of any other call
        want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, act)
    else:
        h = _ffn.half_step(X.dtype)
        eg = (dh * u).abs() * 2.0 ** -19 * (1 + g.abs()) + h * h * dg.abs() + _ffn.tiny(X.dtype)
        eu = dh.abs() * _ffn.act_err(g, act) + h * h * du.abs() + _ffn.tiny(X.dtype)
        ex = eg @ wg.double().abs() + eu @ wu.double().abs() + _ffn.sum_err(
            4 * R, (dg.abs() + eg) @ wg.double().abs() + (du.abs() + eu) @ wu.double().abs())
        bound = (ex, *((e.t() @ x.abs()) + _ffn.sum_err(2 * T, (d.abs() + e).t() @ x.abs()) for d, e in ((dg, eg), (du, eu))))
        # as a norm: the output's rounding, evenly spread over half a step, and the slope's own 2^-19
        for a, b, what in zip(got, want, ("dX", "dWg", "dWu")):
            off = float((a.double() - b).norm() / b.norm())
            assert off <= h / 3 ** 0.5 + 2.0 ** -17, f"{what}: {off:.6f} of the norm"
    for a, b, e, what in zip(got, want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


@pytest.mark.parametrize("N,M", [(2, 4), (4, 8), (1, 4)])
@pytest.mark.parametrize("T,R,K", [(1, 1, 8), (1, 77, 136), (16, 130, 512), (33, 77, 136), (70, 1, 64), (130, 333, 584),
                                   (300, 500, 712)])
@pytest.mark.parametrize("stream", [0, 1])
def test_glu_float32_products_everywhere(tile, stream, T, R, K, N, M):
    """float32 G and U on every path: contiguous, their rows in turn, inside
    wider buffers at odd elements; H's bits do not change."""
    dt = "bf16" if T % 2 else "f16"
    pg, wg, kg = weights(R, K, N, M, dt, "g")
    pu, wu, ku = weights(R, K, N, M, dt, "u")
    X, dH = normal((T, K), 1.0, dt, "X", T), normal((T, R), 0.1, dt, "dH", T)
    tile("stream", stream)
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, "silu")
    H = nm.glu(pg, pu, X)
    first = None
    for layout in range(3):
        if layout == 0:
            buf = pre = torch.full((2, T, R), 7.0, device="cuda")
        elif layout == 1:
            buf = torch.full((T, 2, R), 7.0, device="cuda")
            pre = buf.transpose(0, 1)
        else:
            buf = torch.full((2, T, R + 6), 7.0, device="cuda")
            pre = buf[:, :, 3:R + 3]
        assert torch.equal(nm.glu(pg, pu, X, pre=pre), H)
        check(pre[0], g, eg, "G")
        check(pre[1], u, eu, "U")
        if layout == 2:
            assert bool((buf[:, :, :3] == 7.0).all()) and bool((buf[:, :, R + 3:] == 7.0).all())
        got = nm.glu_backward(pg, pu, X, pre, dH)
        want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
        for a, b, e, what in zip(got, want, bound, ("dX", "dWg", "dWu")):
            check(a, b, e, what)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("shape", [0, 1, 2, 3])
@pytest.mark.parametrize("N,M", [(2, 4), (4, 8)])
def test_glu_float32_products_in_every_shape(tile, shape, N, M):
    T, R, K, dt = 700, 1900, 136, "bf16"
    pg, wg, _ = weights(R, K, N, M, dt, "g")
    pu, wu, _ = weights(R, K, N, M, dt, "u")
    X = normal((T, K), 1.0, dt, "X")
    tile("tile24" if (N, M) == (2, 4) else "tile", shape)
    h, g, u, eh, eg, eu = _ffn.glu64(X, wg, wu, "gelu")
    pre = torch.full((2, T, R), 7.0, device="cuda")
    check(nm.glu(pg, pu, X, act="gelu", pre=pre), h, eh, "H")
    check(pre[0], g, eg, "G")
    check(pre[1], u, eu, "U")


def test_float32_products_past_the_type():
    """Products that fp16 cannot hold: float32 ones give their own gradients."""
    T, R, K = 70, 48, 64
    Wg, Wu = normal((R, K), 0.05, "f16", "Wg"), normal((R, K), 0.05, "f16", "Wu")
    Wg[:, 0] = 40000.0
    kg, ku = _ffn.kept(Wg, 2, 4), _ffn.kept(Wu, 2, 4)
    wg, wu = torch.where(kg, Wg, 0.0), torch.where(ku, Wu, 0.0)
    pg, pu = nm.pack(Wg, 2, 4), nm.pack(Wu, 2, 4)
    X = normal((T, K), 0.1, "f16", "X")
    X[:, 0] = torch.linspace(-8, 8, T)
    pre = torch.empty(2, T, R, device="cuda")
    nm.glu(pg, pu, X, pre=pre)
    assert bool(torch.isfinite(pre).all()) and float(pre[0].max()) > 3e5
    dH = normal((T, R), 0.0005, "f16", "dH")
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
    for a, b, e, what in zip(nm.glu_backward(pg, pu, X, pre, dH), want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


@pytest.mark.parametrize("T", [5, 70, 300])
def test_glu_backward_past_the_range_of_fp16(T):
    """dG or dU beyond 65504: the token's dX and the row of the weight gradient
    are not finite, nothing else changes; below 2^-25: zero."""
    R, K = 80, 136
    pg, _, kg = weights(R, K, 2, 4, "f16", "g")
    pu, _, ku = weights(R, K, 2, 4, "f16", "u")
    X, dH = normal((T, K), 1.0, "f16", "X", T), normal((T, R), 0.1, "f16", "dH", T)
    pre = normal((2 * T, R), 1.0, "f16", "pre", T).view(2, T, R)
    clean = nm.glu_backward(pg, pu, X, pre, dH)
    pre[:, 2, 7] = torch.tensor([30.0, 40.0], device="cuda")
    dH[2, 7] = 30000.0                                    # dG = 1.2e6, dU = 9e5
    dx, dwg, dwu = nm.glu_backward(pg, pu, X, pre, dH)
    t, r = torch.arange(T, device="cuda") != 2, torch.arange(R, device="cuda") != 7
    assert torch.equal(dx[t], clean[0][t]) and torch.equal(dwg[r], clean[1][r]) and torch.equal(dwu[r], clean[2][r])
    assert not bool(torch.isfinite(dx[2]).all())
    for d, k in ((dwg, kg), (dwu, ku)):
        assert not bool(torch.isfinite(d[7][k[7]]).any()) and bool((d[7][~k[7]] == 0).all())
    pre.fill_(0.25)
    dH.fill_(2.0 ** -24)                                  # dG, dU below 2^-26
    for d in nm.glu_backward(pg, pu, X, pre, dH):
        assert bool((d == 0).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [3, 70, 200])
def test_glu_backward_of_products_past_the_type(T, dt, act):
    """Products that 16 bits hold as infinities: H is finite, and the gradients
    are those of the type's largest value, finite in every row."""
    R, K = 48, 64
    top = torch.finfo(TORCH[dt]).max
    Wg = normal((R, K), 0.05, dt, "Wg")
    Wg[:, 0] = 0.0
    Wg[::3, 0] = 40000.0 if dt == "f16" else 0.0
    Wu = normal((R, K), 0.05, dt, "Wu")
    kg, ku = _ffn.kept(Wg, 2, 4), _ffn.kept(Wu, 2, 4)
    wg, wu = torch.where(kg, Wg, 0.0), torch.where(ku, Wu, 0.0)
    pg, pu = nm.pack(Wg, 2, 4), nm.pack(Wu, 2, 4)
    X = normal((T, K), 0.1, dt, "X", T)
    X[:, 0] = torch.tensor([2.0, -2.0, 0.5], device="cuda").repeat(T)[:T]
    pre = torch.empty((2, T, R), dtype=X.dtype, device="cuda")
    H = nm.glu(pg, pu, X, act=act, pre=pre)
    assert bool(torch.isfinite(H).all())
    if dt == "f16":
        assert bool((pre[0, 0::3, ::3] == float("inf")).all()) and bool((pre[0, 1::3, ::3] == float("-inf")).all())
    else:
        pre[0, 0, ::3], pre[0, 1, ::3] = float("inf"), float("-inf")
    pre[1, 2, 5::6] = float("inf")
    dH = normal((T, R), 0.0005, dt, "dH", T)
    if dt == "bf16":
        dH *= 2.0 ** -100                                 # outputs within the type
    else:
        dH[2, 5::6] = 2.0 ** -14
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre.clamp(-top, top), dH, act)
    for a, b, e, what in zip(nm.glu_backward(pg, pu, X, pre, dH, act=act), want, bound, ("dX", "dWg", "dWu")):
        assert bool(torch.isfinite(a).all()), what
        check(a, b, e, what)
    pre[0, 1, 1] = float("nan")                           # what is no number stays none
    dx, dwg, dwu = nm.glu_backward(pg, pu, X, pre, dH, act=act)
    assert bool(torch.isnan(dx[1]).any()) and bool(torch.isfinite(dx[[0, 2]]).all())
    assert bool(torch.isnan(dwg[1][kg[1]]).all()) and bool(torch.isnan(dwu[1][ku[1]]).all())


# ---------------------------------------------------------------- microscaled 4-bit format
def _check_mx(x):
    m = nm.mx_quantize(x)
    val, code, byte = _ffn.mx64(x.cpu())
    codes, bytes_ = _ffn.mx_read(m)
    K = x.shape[1]
    nb = byte.shape[1]
    assert torch.equal(bytes_[:, :nb], byte), "scales"
    fin = (byte != 255).repeat_interleave(32, dim=1)[:, :K]
    # a negative value that rounds to zero may carry either sign
    same = (codes[:, :K] == code) | ((codes[:, :K] & 7 == 0) & (code & 7 == 0))
    assert bool(same[fin].all()), f"codes differ at {(~same & fin).nonzero()[:4].tolist()}"
    assert bool((codes[:, K:] == 0).all()), "codes past K"
    for dt in (x.dtype, torch.float32):
        y = nm.mx_dequantize(m, out_dtype=dt).double().cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(val))
        assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(val)), dt
    return m


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("top", [0.0, 1.0, 1.9921875, 6.5, 2.0 ** -20])
def test_mx_quantize_every_16_bit_value(dt, top):
    """Every finite 16-bit pattern, below a block's largest magnitude in the
    first block of its row, among similar magnitudes in the second."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(TORCH[dt])
    v = v[torch.isfinite(v)]
    order = torch.argsort(v.abs().float())
    v = v[order]
    v = torch.cat((v, v[:-len(v) % 31])).view(-1, 31)
    lead = torch.full((v.shape[0], 1), top, dtype=v.dtype)
    x = torch.cat((lead, v), dim=1)
    _check_mx(x.cuda())


@pytest.mark.parametrize("rows,K", [(1, 1), (1, 31), (3, 32), (31, 33), (32, 255), (33, 256), (65, 257), (7, 770),
                                    (200, 1000)])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_mx_quantize_shapes(rows, K, dt):
    x = normal((rows, K), 1.0, dt, "x", rows, K)
    _check_mx(x)
    _, v = wide(x, 3, float("nan"))
    _check_mx(v)


def test_mx_quantize_float32_range():
    """binary32 blocks at both ends of the scale's range, subnormals among
    them, and values that round half way."""
    x = torch.randn(64, 64, generator=_gen("r"))
    e = torch.linspace(-149, 127, 64).round()
    x = torch.ldexp(x, e[:, None].to(torch.int32)).clamp(-3e38, 3e38)
    x[0] = 0.0
    x[1, ::2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]).repeat(4)
    x[1, 1::2] = -x[1, ::2]
    _check_mx(x.cuda())


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_mx_quantize_non_finite_blocks(dt, bad):
    x = normal((5, 100), 1.0, dt, "x")
    x[2, 40] = bad
    x[4, 99] = bad
    m = _check_mx(x)
    y = nm.mx_dequantize(m)
    assert bool(torch.isnan(y[2, 32:64]).all()) and bool(torch.isnan(y[4, 96:]).all())
    assert int(torch.isnan(y).sum()) == 32 + 4
    # a block without a value taints every sum it enters, and no other
    w = nm.mx_quantize(normal((48, 100), 1.0, dt, "w"))
    for X in (x, m):
        out = nm.mx_linear(w, X, out_dtype=torch.float32)
        assert bool(torch.isnan(out[[2, 4]]).all()) and bool(torch.isfinite(out[[0, 1, 3]]).all())


MX_SHAPES = [(1, 1, 1), (1, 8, 7), (1, 17, 40), (2, 100, 256), (3, 33, 9), (9, 20, 261), (15, 16, 264),
             (16, 40, 1027), (16, 48, 1000), (17, 40, 33), (33, 65, 512), (64, 33, 770), (65, 40, 32),
             (70, 129, 256), (129, 300, 520), (300, 257, 1288)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T", range(1, 17))
def test_mx_few_tokens_quantised_inside(T, dt):
    """Activations quantised inside the product and beforehand: the same bits,
    for every token count a load of token pairs can end at, one to several
    slabs a wave, the last one whole and short, inputs new to the caches."""
    for K, R in ((256, 40), (264, 33), (2560, 17), (8712, 100)):
        w, u = _mx_w(R, K, dt)[0], _mx_w(R, K, dt, "u")[0]
        for i in range(3):
            X = normal((T, K), 1.0, dt, "X", T, K, i)
            q = nm.mx_quantize(X)
            assert torch.equal(nm.mx_linear(w, X), nm.mx_linear(w, q, out_dtype=X.dtype)), (K, i)
            assert torch.equal(nm.mx_glu(w, u, X), nm.mx_glu(w, u, q, out_dtype=X.dtype)), (K, i)


def _mx_w(R, K, dt, *key):
    W = normal((R, K), 0.05, dt, "mw", R, K, *key)
    return nm.mx_quantize(W), _ffn.mx64(W)[0]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,R,K", MX_SHAPES)
def test_mx_linear_shapes(T, R, K, dt):
    w, W = _mx_w(R, K, dt)
    X = normal((T, K), 1.0, dt, "X", T, K)
    X[:, :: 7] *= 10
    x = _ffn.mx64(X)[0]
    b = normal((R,), 1.0, "f32", "b", R)
    y = x @ W.t()
    e = _ffn.sum_err(K, x.abs() @ W.abs().t())
    check(nm.mx_linear(w, X), y, e, "Y")
    yb = y + b.double()
    eb = e + 2.0 ** -23 * (yb.abs() + e)
    check(nm.mx_linear(w, X, bias=b, out_dtype=torch.float32), yb, eb, "Y + b")
    ya = _ffn.act64(yb, "gelu")
    check(nm.mx_linear(w, X, bias=b, act="gelu"), ya, 1.13 * eb + _ffn.act_err(yb, "gelu") + 1e-6 * eb, "gelu")
    # activations that come quantised: the same sums
    q = nm.mx_quantize(X)
    out = torch.empty(T, R, dtype=TORCH[dt], device="cuda")
    assert torch.equal(nm.mx_linear(w, q, out=out), nm.mx_linear(w, X))
    # a pitch that rules out wide accesses on both sides
    _, xv = wide(X, 3, float("nan"))
    ob, ov = wide(torch.zeros(T, R, dtype=TORCH[dt], device="cuda"), 3, 5.0)
    nm.mx_linear(w, xv, out=ov)
    check(ov, y, e, "strided")
    assert bool((ob[:, R:] == 5.0).all())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,R,K", MX_SHAPES + [(700, 4500, 300)])
def test_mx_glu_shapes(T, R, K, dt):
    wg, Wg = _mx_w(R, K, dt, "g")
    wu, Wu = _mx_w(R, K, dt, "u")
    X = normal((T, K), 1.0, dt, "X", T, K)
    x = _ffn.mx64(X)[0]
    for act in ("silu", "gelu"):
        h, _, _, eh, _, _ = _ffn.glu64(x, Wg, Wu, act)
        check(nm.mx_glu(wg, wu, X, act=act), h, eh, act)
    check(nm.mx_glu(wg, wu, nm.mx_quantize(X), act="gelu", out_dtype=torch.float32), h, eh, "quantised X")


@pytest.mark.parametrize("K", [32, 300, 1500])
@pytest.mark.parametrize("shape", [0, 1, 2, 3])
def test_mx_tile_shapes(tile, shape, K):
    """Every shape with more tiles than compute units, split and not."""
    T, R = {0: (2100, 8300), 1: (1100, 8300), 2: (1100, 4300), 3: (700, 3700)}[shape]
    w, W = _mx_w(R, K, "bf16")
    X = normal((T, K), 1.0, "bf16", "X", T, K)
    x = _ffn.mx64(X)[0]
    y, e = x @ W.t(), _ffn.sum_err(K, x.abs() @ W.abs().t())
    b = normal((R,), 1.0, "f32", "b", R)
    for split in (1, 2, 5):
        tile("tile", shape, split)
        check(nm.mx_linear(w, X), y, e, f"Y in {split}")
        yb = y + b.double()
        eb = e + 2.0 ** -23 * (yb.abs() + e) * split
        check(nm.mx_linear(w, X, bias=b, out_dtype=torch.float32), yb, eb, f"Y + b in {split}")
    u, U = _mx_w(R, K, "bf16", "u")
    h, _, _, eh, _, _ = _ffn.glu64(x, W, U, "silu")
    check(nm.mx_glu(w, u, X), h, eh, "H")


@pytest.mark.parametrize("split", [2, 7, 16])
@pytest.mark.parametrize("R", [1, 333, 642])
def test_mx_split_reductions(tile, R, split):
    """Parts of a long reduction added with the bias and the activation;
    outputs of an odd width, in rows of an odd pitch."""
    T, K = 70, 8200
    w, W = _mx_w(R, K, "bf16")
    X = normal((T, K), 0.05, "bf16", "X", R)
    b = normal((R,), 1.0, "f32", "b", R)
    x = _ffn.mx64(X)[0]
    y, e = x @ W.t() + b.double(), _ffn.sum_err(K, x.abs() @ W.abs().t()) + 2.0 ** -23 * split * b.double().abs()
    tile("tile", 3, split)
    ob, ov = wide(torch.zeros(T, R, dtype=torch.float16, device="cuda"), 3, 5.0)
    check(nm.mx_linear(w, X, bias=b, out=ov), y, e + 2.0 ** -23 * (y.abs() + e), "Y")
    assert bool((ob[:, R:] == 5.0).all())
    want = _ffn.act64(y, "gelu")
    err = 1.13 * (e + 2.0 ** -23 * (y.abs() + e)) + _ffn.act_err(y, "gelu") + 2.0 ** -22 * e
    check(nm.mx_linear(w, X, bias=b, act="gelu", out=ov), want, err, "gelu(Y)")
    assert bool((ob[:, R:] == 5.0).all())


@pytest.mark.parametrize("shape", [0, 1, 2, 3])
@pytest.mark.parametrize("split,K", [(5, 2560), (16, 8192), (16, 4096), (11, 8200)])
def test_mx_splits_that_divide(tile, shape, split, K):
    """The largest splits in every shape, one slab a slice and more; the
    workspace holds that many slices."""
    T, R = 130, 300
    w, W = _mx_w(R, K, "bf16")
    X = normal((T, K), 0.05, "bf16", "X", K)
    q = nm.mx_quantize(X)
    b = normal((R,), 1.0, "f32", "b", R)
    tile("tile", shape, split)
    quant = -(-T * (-(-K // 256) * 128) // 256) * 256 + -(-T // 32) * -(-K // 256) * 256
    assert nm.mx_workspace_size(w, T) == quant + -(-split * T * R * 4 // 256) * 256
    x = _ffn.mx64(X)[0]
    y, e = x @ W.t() + b.double(), _ffn.sum_err(K, x.abs() @ W.abs().t()) + 2.0 ** -23 * split * b.double().abs()
    Y = nm.mx_linear(w, X, bias=b)
    check(Y, y, e + 2.0 ** -23 * (y.abs() + e), "Y")
    assert torch.equal(nm.mx_linear(w, q, bias=b), Y)


def test_mx_offsets_past_32_bits():
    """Outputs, then quantised activations, of more than 2^32 bytes."""
    for T, R, K in ((70000, 32768, 64), (300000, 64, 32768)):
        w, W = _mx_w(R, K, "bf16")
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        X = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        m = nm.mx_quantize(X)
        Y = nm.mx_linear(w, m)
        for a in (0, T // 2, T - 3):
            x = _ffn.mx64(X[a:a + 3])[0]
            check(Y[a:a + 3], x @ W.t(), _ffn.sum_err(K, x.abs() @ W.abs().t()), f"Y from {a}")
        if T == 70000:
            y = nm.mx_dequantize(m, out_dtype=torch.bfloat16)
            assert torch.equal(y[-3:].double(), _ffn.mx64(X[-3:])[0])
        del X, Y, m


def test_mx_linear_large_tiles():
    T, R, K = 1500, 9000, 300
    w, W = _mx_w(R, K, "bf16")
    X = normal((T, K), 1.0, "bf16", "X")
    x = _ffn.mx64(X)[0]
    check(nm.mx_linear(w, X), x @ W.t(), _ffn.sum_err(K, x.abs() @ W.abs().t()), "Y")


# ---------------------------------------------------------------- in use
def test_pruned_block_end_to_end():
    """Gated block and down projection of a pruned model, forward and back
    down to the weights, on a stream of its own."""
    T, R, K, dt = 96, 256, 128, "bf16"
    pg, wg, kg = weights(R, K, 2, 4, dt, "g")
    pu, wu, ku = weights(R, K, 2, 4, dt, "u")
    pd, wd, _ = weights(K, R, 2, 4, dt, "d")
    X = normal((T, K), 1.0, dt, "X")
    pre = torch.empty(2, T, R, dtype=X.dtype, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        H = nm.glu(pg, pu, X, pre=pre)
        Y = nm.linear(pd, H)
        dH = (Y.float() @ wd.float()).to(H.dtype)         # dL/dY = Y
        grads = nm.glu_backward(pg, pu, X, pre, dH)
    s.synchronize()
    h, _, _, eh, _, _ = _ffn.glu64(X, wg, wu, "silu")
    check(H, h, eh, "H")
    check(Y, H.double() @ wd.double().t(), _ffn.sum_err(R, H.double().abs() @ wd.double().abs().t()), "Y")
    want, bound = _ffn.glu_grad64(X, wg, wu, kg, ku, pre, dH, "silu")
    for a, b, e, what in zip(grads, want, bound, ("dX", "dWg", "dWu")):
        check(a, b, e, what)


@pytest.mark.parametrize("T", [1, 20, 100])
def test_four_bit_block_in_a_graph(T):
    """Gated block and down projection at 4 bits, and the pruned block with
    its gradients, captured into one graph and replayed on new inputs with
    eager work in between: every replay gives the eager call's bits."""
    R, K, dt = 320, 264, "bf16"
    g4, u4 = _mx_w(R, K, dt, "g")[0], _mx_w(R, K, dt, "u")[0]
    d4 = _mx_w(K, R, dt, "d")[0]
    pg, pu = weights(R, K, 2, 4, dt, "g")[0], weights(R, K, 2, 4, dt, "u")[0]
    X = normal((T, K), 1.0, dt, "X")
    dH = normal((T, R), 0.1, dt, "dH")
    pre = torch.empty(2, T, R, dtype=X.dtype, device="cuda")

    def step():
        y4 = nm.mx_linear(d4, nm.mx_glu(g4, u4, X))
        h = nm.glu(pg, pu, X, pre=pre)
        return (y4, h, *nm.glu_backward(pg, pu, X, pre, dH))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        X.copy_(normal((T, K), 1.0, dt, "X", i))
        dH.copy_(normal((T, R), 0.1, dt, "dH", i))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), f"replay {i}"


def test_results_do_not_vary():
    """No result depends on the order in which workgroups finish."""
    T, R, K = 130, 600, 520
    pg, pu = weights(R, K, 4, 8, "f16", "g")[0], weights(R, K, 4, 8, "f16", "u")[0]
    X, dH = normal((T, K), 1.0, "f16", "X"), normal((T, R), 0.1, "f16", "dH")
    pre = torch.empty(2, T, R, dtype=X.dtype, device="cuda")
    w = _mx_w(R, K, "f16")[0]
    first = None
    for _ in range(3):
        out = (nm.glu(pg, pu, X, pre=pre), *nm.glu_backward(pg, pu, X, pre, dH), nm.mx_linear(w, X))
        if first is None:
            first = out
        for a, b in zip(first, out):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,R,K", [(20, 200, 264), (200, 1000, 520)])
def test_float32_products_in_a_graph(T, R, K):
    """A step with float32 products (in two parts and in one) on a stream of its
    own, then captured and replayed with eager work between."""
    dt = "bf16"
    pg, pu = weights(R, K, 2, 4, dt, "g")[0], weights(R, K, 2, 4, dt, "u")[0]
    X, dH = normal((T, K), 1.0, dt, "X"), normal((T, R), 0.1, dt, "dH")
    pre = torch.empty(2, T, R, device="cuda")
    ws = torch.empty(nm.glu_backward_workspace_size(pg, pu, T), dtype=torch.uint8, device="cuda")

    def step():
        h = nm.glu(pg, pu, X, pre=pre)
        return (h, *nm.glu_backward(pg, pu, X, pre, dH, workspace=ws))

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        X.copy_(normal((T, K), 1.0, dt, "X", i))
        dH.copy_(normal((T, R), 0.1, dt, "dH", i))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), f"replay {i}"
