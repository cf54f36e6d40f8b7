"""8-bit rows, their product, and products of rows grouped by expert: GPU
parity with 64-bit forms within derived bounds."""
import contextlib
import os

import pytest
import torch

import semi_structured_sparse_nm_amd as nm
from tests._ffn import TORCH, check
from tests._rows import (expert64, expert_grad64, experts_of, i8_64, i8_expert64, i8_product64, pruned)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SPARSE = [(2, 4), (1, 4), (1, 8), (2, 8)]             # as 2:4 blocks in the tile product; others as dense ones
PATTERNS = [(1, 4), (2, 4), (3, 4), (4, 4), (1, 8), (2, 8), (3, 8), (4, 8), (5, 8), (6, 8), (7, 8), (8, 8)]
# every pattern streamed, wide and in each shape of its tile product
PATHS = [(p, *nm_) for nm_ in PATTERNS
         for p in ["stream:1", "wide:0", "wide:1"] + [f"{'tile24' if nm_ in SPARSE else 'tile'}:{i}" for i in range(4)]]


@contextlib.contextmanager
def forced(path):
    """NM_FFN_TILE for the calls inside, as the tests of the tile products use it."""
    old = os.environ.get("NM_FFN_TILE")
    if path:
        os.environ["NM_FFN_TILE"] = path
    try:
        yield
    finally:
        if old is None:
            os.environ.pop("NM_FFN_TILE", None)
        else:
            os.environ["NM_FFN_TILE"] = old


def randn(*shape, seed=0, dt=torch.float32, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dt)


def strided(x, pad):
    """x's values in rows that lie `pad` elements apart, from an odd element on."""
    if not pad:
        return x
    wide = torch.full((x.shape[0], x.shape[1] + pad + 1), float("nan") if x.is_floating_point() else 0, device=DEV,
                      dtype=x.dtype)
    v = wide[:, 1:1 + x.shape[1]]
    v.copy_(x)
    return v


def counts(T, E, kind, seed=0):
    """Offsets of E experts over T rows, int32 on the GPU."""
    g = torch.Generator()
    g.manual_seed(seed)
    if kind == "even":
        ends = [(i + 1) * T // E for i in range(E)]
    elif kind == "one":                                   # every row goes to one expert
        ends = [T if i >= E // 2 else 0 for i in range(E)]
    else:                                                 # ragged, some without rows
        w = torch.rand(E, generator=g) * (torch.rand(E, generator=g) < 0.7)
        w[torch.randint(E, (1,), generator=g)] += 0.1
        ends = (w.cumsum(0) / w.sum() * T).round().long().tolist()
        ends[-1] = T
    return torch.tensor([0] + ends, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- quantiser
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,K,pad", [(1, 1, 0), (1, 7, 0), (3, 8, 3), (5, 129, 0), (197, 770, 0), (6, 1024, 5),
                                        (9, 2050, 1), (4, 4100, 0), (3, 11008, 0), (2, 16385, 0), (2, 20000, 3),
                                        (4099, 64, 0)])
def test_i8_quantize(dt, rows, K, pad):
    x = randn(rows, K, seed=rows + K, dt=TORCH[dt])
    x[:, ::7] *= 20
    x[:, K // 2] = x.abs().amax(dim=1) / 2               # near a border: 63.5
    if rows > 2:
        x[1] = 0
    X = strided(x, pad)
    q = nm.i8_quantize(X)
    want, s = i8_64(x)
    assert torch.equal(q.scales, s)
    assert torch.equal(q.values.long(), want)
    assert not q.codes[:, K:].any()
    for odt in (torch.float32, x.dtype):
        y = nm.i8_dequantize(q, odt)
        assert torch.equal(y, (want.float() * s[:, None]).to(odt))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_i8_quantize_extremes(dt):
    t = TORCH[dt]
    f = torch.finfo(t)
    x = torch.zeros(9, 300, dtype=t, device=DEV)
    x[0] = f.max
    x[0, 1] = -f.max
    x[1] = f.smallest_normal * f.eps                     # the smallest there is
    x[2, 5] = f.smallest_normal
    x[2, 6] = f.smallest_normal * f.eps
    x[3, 299] = float("inf")
    x[4, 0] = float("nan")
    x[5, 100:] = float("-inf")
    x[6] = torch.linspace(-1, 1, 300, device=DEV).to(t)
    x[7] = -0.0
    x[8, 0], x[8, 1] = f.max, f.tiny
    q = nm.i8_quantize(x)
    want, s = i8_64(x)
    assert torch.equal(q.scales.isnan(), s.isnan())
    assert torch.equal(q.scales.nan_to_num(), s.nan_to_num())
    assert torch.equal(q.values.long(), want)
    y = nm.i8_dequantize(q)
    assert y[3:6].isnan().all() and not y[[0, 1, 2, 6, 7, 8]].isnan().any()


def test_i8_quantize_ties():
    # scale 1: quotients that are whole numbers and halves
    x = torch.arange(-254, 255, device=DEV, dtype=torch.float32)[None] / 2
    q = nm.i8_quantize(x)
    assert float(q.scales) == 1.0
    assert torch.equal(q.values[0].float(), torch.round(x[0]))
    assert torch.equal(nm.i8_quantize(x.half()).values, q.values)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_i8_quantize_beside_the_quotient(dt):
    """How far the stored rows are from those of the rounded quotient amax / 127.  The
    scale is amax c rounded, c = 1/127 cut to 24 bits, within 2^-28 of it: it and the
    rounded quotient are off by at most (2^-28 + 2^-24) and 2^-24 of amax / 127, less
    than one and a half steps apart, so neighbours at most.  x over either is then the
    same within 127 (2^-23 + 2^-28 + 2^-46) < 2^-16 (2^-23 a step's most), so only elements
    that close to a border may differ, by one.  Every element is within half a scale of
    x, and 127 scales within 127 (2^-28 + 2^-24) < 2^-16 scales of amax."""
    x = randn(2000, 1000, seed=7, dt=TORCH[dt])
    x[::3] *= randn(667, 1, seed=8).exp().to(x.dtype)
    q = nm.i8_quantize(x)
    amax = x.double().abs().amax(dim=1)
    s = (amax / 127).float()
    assert ((q.scales.view(torch.int32) - s.view(torch.int32)).abs() <= 1).all()
    u = x.double() / s.double()[:, None]
    low = torch.floor(u)
    border = (u - low - 0.5).abs() <= 2.0 ** -16
    off = (q.values.double() - torch.round(u)).abs()
    assert not off[~border].any() and (off <= 1).all()
    scale = q.scales.double()[:, None]
    assert ((q.values.double() * scale - x.double()).abs() <= (0.5 + 2.0 ** -16) * scale).all()


# ---------------------------------------------------------------- 8-bit product
def i8_weight(R, K, N, M, seed, E=None):
    """(packed, scales, pruned whole numbers)."""
    W = randn(*((E or 1), R, K), seed=seed, scale=0.02)
    q, s = i8_64(W.reshape(-1, K))
    codes = q.to(torch.int8).reshape(W.shape)
    w, _ = pruned(codes, N, M)
    s = s.reshape(W.shape[:2])
    if E is None:
        return nm.pack(codes[0], N, M), s[0], w[0]
    return nm.pack_experts(codes, N, M), s, w


@pytest.mark.parametrize("path,N,M", PATHS)
def test_i8_linear_patterns(path, N, M):
    T, R, K = 70, 150, 392
    p, sw, w = i8_weight(R, K, N, M, 3)
    X = randn(T, K, seed=4, dt=torch.bfloat16)
    bias = randn(R, seed=5)
    with forced(path):
        Y = nm.i8_linear(p, sw, X, bias=bias, out_dtype=torch.float32)
    q, sx = i8_64(X)
    check(Y, *i8_product64(q, sx, w, sw, bias, "none"), f"{path} {N}:{M}")


@pytest.mark.parametrize("dt,odt", [("f16", None), ("bf16", None), ("f32", None), ("f16", "f32"), ("bf16", "f16"),
                                    ("f32", "bf16")])
@pytest.mark.parametrize("T,R,K,N,M", [(1, 1, 4, 2, 4), (1, 512, 4096, 2, 4), (2, 33, 132, 1, 4), (16, 100, 1000, 4, 8),
                                       (17, 64, 128, 2, 4), (33, 257, 640, 3, 4), (64, 16, 260, 4, 4),
                                       (65, 300, 520, 2, 8), (100, 1500, 1000, 5, 8), (129, 500, 384, 2, 4),
                                       (300, 700, 1284, 4, 4), (600, 520, 256, 2, 4)])
def test_i8_linear(dt, odt, T, R, K, N, M):
    p, sw, w = i8_weight(R, K, N, M, T + R)
    pad = 3 if R % 2 else 0
    X = strided(randn(T, K, seed=K, dt=TORCH[dt]), pad)
    bias = randn(R, seed=1) if T % 2 else None
    act = "gelu" if K % 8 == 4 else "none"
    Y = nm.i8_linear(p, sw, X, bias=bias, act=act, out_dtype=odt and TORCH[odt])
    assert Y.dtype == TORCH[odt or dt]
    q, sx = i8_64(X)
    want, bound = i8_product64(q, sx, w, sw, bias, act)
    check(Y, want, bound, "i8_linear")
    # the same rows quantised beforehand, into a wider output's columns
    wide = torch.full((T, R + 5), 7.0, device=DEV, dtype=Y.dtype)
    Z = nm.i8_linear(p, sw, nm.i8_quantize(X), bias=bias, act=act, out=wide[:, 2:2 + R])
    assert torch.equal(Z, Y)
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + R:] == 7).all()


def test_i8_linear_long_sums():
    # the longest reduction, every product the largest: 131068 x 127 x 127 is close to 2^31
    K = 131068
    w = torch.full((20, K), 127, dtype=torch.int8, device=DEV)
    w[1::2] = -127
    p = nm.pack(w, 4, 4)
    sw = torch.ones(20, device=DEV)
    for T in (3, 80):
        X = torch.ones(T, K, device=DEV, dtype=torch.float16)
        Y = nm.i8_linear(p, sw, X, out_dtype=torch.float32)
        q, sx = i8_64(X)
        check(Y, *i8_product64(q, sx, w, sw, None, "none"), "long sums")


# Rows that the streamed product quantises itself, longer than the 4096 columns that
# its threads have a piece each of: two to four pieces a thread, whose maximum is carried
# across them, and rows beyond the four pieces that a thread holds.
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,K,N,M", [(1, 4100, 2, 4), (1, 8192, 4, 8), (1, 11008, 2, 4), (1, 11008, 4, 8),
                                     (1, 12292, 3, 4), (1, 16384, 4, 8), (2, 8184, 5, 8), (3, 5376, 4, 8),
                                     (2, 4224, 4, 4)])
def test_i8_linear_long_rows_quantised_inside(dt, T, K, N, M):
    R = 90
    p, sw, w = i8_weight(R, K, N, M, K)
    assert nm.i8_linear_workspace_size(p, T) == 0         # (no launch of the quantiser)
    X = randn(T, K, seed=T, dt=TORCH[dt])
    # (each row's largest element in another piece of another thread)
    for t in range(T):
        X[t, (K - 1 - 700 * t) % K] = 9.0 + t
    X = strided(X, 5)
    Y = nm.i8_linear(p, sw, X, out_dtype=torch.float32)
    q, sx = i8_64(X)
    check(Y, *i8_product64(q, sx, w, sw, None, "none"), "i8_linear")
    assert torch.equal(nm.i8_linear(p, sw, nm.i8_quantize(X), out_dtype=torch.float32), Y)
    X[0, K - 1] = float("nan")                            # in the last piece
    Y2 = nm.i8_linear(p, sw, X, out_dtype=torch.float32)
    assert Y2[0].isnan().all() and torch.equal(Y2[1:], Y[1:])


# The rows of one expert, up to 48 KB of LDS beside the kernel's own 19: launches with
# more than 64 KB.
@pytest.mark.parametrize("kind", ["one", "ragged", "even"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,E,K,N,M", [(15, 32, 3200, 4, 8), (15, 32, 3136, 2, 4), (3, 3, 16200, 4, 8),
                                       (2, 7, 16384, 3, 4), (16, 16, 2944, 6, 8)])
def test_i8_expert_linear_rows_quantised_inside(T, E, K, N, M, dt, kind):
    R = 40
    x, sw, w = i8_weight(R, K, N, M, K, E=E)
    assert nm.i8_expert_linear_workspace_size(x, T) == 0
    X = randn(T, K, seed=T, dt=TORCH[dt])
    for t in range(T):
        X[t, (K - 1 - 900 * t) % K] = 9.0 + t
    o = counts(T, E, kind, seed=K)
    Y = nm.i8_expert_linear(x, sw, X, o, out_dtype=torch.float32)
    q, sx = i8_64(X)
    check(Y, *i8_expert64(q, sx, w, sw, None, "none", o), "i8_expert_linear")
    assert torch.equal(nm.i8_expert_linear(x, sw, nm.i8_quantize(X), o, out_dtype=torch.float32), Y)


def test_i8_linear_not_finite():
    p, sw, w = i8_weight(40, 256, 2, 4, 0)
    for T in (4, 90):
        X = randn(T, 256, dt=torch.bfloat16)
        X[1, 3] = float("inf")
        X[2, 200] = float("nan")
        Y = nm.i8_linear(p, sw, X)
        assert Y[1].isnan().all() and Y[2].isnan().all()
        ok = [t for t in range(T) if t not in (1, 2)]
        q, sx = i8_64(X[ok])
        check(Y[ok], *i8_product64(q, sx, w, sw, None, "none"), "other tokens")


# ---------------------------------------------------------------- grouped, 16 bits
@pytest.mark.parametrize("path,N,M", PATHS)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_expert_linear_patterns(path, N, M, dt):
    T, R, K, E = 210, 150, 328, 4
    W = randn(E, R, K, seed=1, dt=TORCH[dt], scale=0.1)
    X = randn(T, K, seed=2, dt=TORCH[dt])
    o = counts(T, E, "ragged", seed=3)
    w, _ = pruned(W, N, M)
    x = nm.pack_experts(W, N, M)
    with forced(path):
        Y = nm.expert_linear(x, X, o)
    check(Y, *expert64(X, w, o), f"{path} {N}:{M}")


CASES = [(1, 1, 8, 1), (1, 40, 4, 3), (5, 33, 100, 7), (16, 96, 256, 32), (40, 130, 72, 1), (64, 64, 64, 2),
         (200, 257, 132, 3), (300, 331, 500, 5), (700, 128, 320, 64), (1500, 300, 260, 4), (90, 20, 64, 70),
         (130, 48, 128, 1023)]


@pytest.mark.parametrize("kind", ["even", "one", "ragged"])
@pytest.mark.parametrize("T,R,K,E", CASES)
def test_expert_linear(T, R, K, E, kind):
    N, M = ((2, 4), (3, 4), (1, 4))[T % 3] if K % 8 else ((2, 4), (4, 8), (2, 8), (5, 8), (4, 4))[(T + R) % 5]
    dt = torch.float16 if R % 2 else torch.bfloat16
    W = randn(E, R, K, seed=T, dt=dt, scale=0.1)
    X = strided(randn(T, K, seed=R, dt=dt), 3 if T % 4 == 1 else 0)
    o = counts(T, E, kind, seed=K)
    if T % 2:
        o = o.long()
    w, _ = pruned(W, N, M)
    x = nm.pack_experts(W, N, M)
    check(nm.expert_linear(x, X, o), *expert64(X, w, o), "expert_linear")


@pytest.mark.parametrize("T", [24, 400])
@pytest.mark.parametrize("lo,hi", [(0, 7), (3, 0), (2, 5), (24, 0)])
def test_expert_rows_of_none(T, lo, hi):
    """Rows before the first expert's and behind the last one's: left alone in a
    given output, zero in a new one; in the gradients zero."""
    E, R, K = 3, 50, 136
    W = randn(E, R, K, seed=1, dt=torch.float16, scale=0.1)
    X = randn(T, K, seed=2, dt=torch.float16)
    o = torch.tensor([lo, max(lo, T // 3), max(lo, T // 2), max(lo, T - hi)], dtype=torch.int32, device=DEV)
    w, keep = pruned(W, 2, 4)
    x = nm.pack_experts(W, 2, 4)
    want, bound = expert64(X, w, o)
    rest = experts_of(o, T)[1]
    check(nm.expert_linear(x, X, o), want, bound, "new output")
    out = torch.full((T, R), 3.0, device=DEV, dtype=X.dtype)
    nm.expert_linear(x, X, o, out=out)
    assert (out[rest] == 3).all()
    taken = [r for r in range(T) if r not in rest]
    check(out[taken], want[taken], bound[taken], "given output")
    dY = randn(T, R, seed=3, dt=torch.float16)
    dY[rest] = float("nan")                              # nothing of these rows is used
    X[rest] = float("nan")
    (dX, dW), b = expert_grad64(X, w, keep, dY, o)
    got = nm.expert_linear_backward(x, X, o, dY)
    check(got[0], dX, b[0], "dX")
    check(got[1], dW, b[1], "dW")


def test_expert_bad_offsets():
    """Offsets that run backwards or outside the rows stay inside the buffers."""
    T, E, R, K = 60, 5, 40, 64
    W = randn(E, R, K, seed=1, dt=torch.bfloat16, scale=0.1)
    X = randn(T, K, seed=2, dt=torch.bfloat16)
    dY = randn(T, R, seed=3, dt=torch.bfloat16)
    w, keep = pruned(W, 4, 8)
    x = nm.pack_experts(W, 4, 8)
    for at in ([-7, 5, 3, 80, 20, 10], [0, 2 ** 40, 0, 0, 0, 0], [-2 ** 40, -1, -1, 10, 9, 2 ** 33], [70] * 6, [0] * 6):
        o = torch.tensor(at, dtype=torch.int64, device=DEV)
        check(nm.expert_linear(x, X, o), *expert64(X, w, o), f"{at}")
        want, b = expert_grad64(X, w, keep, dY, o)
        for got, wn, bn in zip(nm.expert_linear_backward(x, X, o, dY), want, b):
            check(got, wn, bn, f"{at}")


# ---------------------------------------------------------------- gradients
@pytest.mark.parametrize("kind", ["even", "one", "ragged"])
@pytest.mark.parametrize("T,R,K,E", CASES)
def test_expert_backward(T, R, K, E, kind):
    N, M = ((2, 4), (3, 4), (1, 4))[T % 3] if K % 8 else ((2, 4), (4, 8), (2, 8), (5, 8), (4, 4))[(T + R) % 5]
    dt = torch.float16 if R % 2 else torch.bfloat16
    W = randn(E, R, K, seed=T, dt=dt, scale=0.1)
    X = strided(randn(T, K, seed=R, dt=dt), 3 if T % 4 == 1 else 0)
    dY = strided(randn(T, R, seed=R + 1, dt=dt), 1 if T % 4 == 2 else 0)
    o = counts(T, E, kind, seed=K)
    w, keep = pruned(W, N, M)
    x = nm.pack_experts(W, N, M)
    (dX, dW), (bX, bW) = expert_grad64(X, w, keep, dY, o)
    gX, gW = nm.expert_linear_backward(x, X, o, dY)
    check(gX, dX, bX, "dX")
    check(gW, dW, bW, "dW")
    assert (gW[~keep] == 0).all()
    # each alone
    oX, none = nm.expert_linear_backward(x, X, o, dY, need_dw=False)
    assert none is None and torch.equal(oX, gX)
    none, oW = nm.expert_linear_backward(x, X, o, dY, need_dx=False)
    assert none is None and torch.equal(oW, gW)


@pytest.mark.parametrize("shape", [0, 1, 2, 3])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_expert_backward_shapes(shape, dt):
    T, R, K, E = 700, 300, 520, 3
    W = randn(E, R, K, seed=1, dt=TORCH[dt], scale=0.1)
    X = randn(T, K, seed=2, dt=TORCH[dt])
    dY = randn(T, R, seed=3, dt=TORCH[dt])
    o = counts(T, E, "ragged", seed=4)
    w, keep = pruned(W, 4, 8)
    x = nm.pack_experts(W, 4, 8)
    (dX, dW), (bX, bW) = expert_grad64(X, w, keep, dY, o)
    with forced(f"tile:{shape}"):
        gX, gW = nm.expert_linear_backward(x, X, o, dY)
    check(gX, dX, bX, "dX")
    check(gW, dW, bW, "dW")


# ---------------------------------------------------------------- grouped, 8 bits
@pytest.mark.parametrize("kind", ["even", "one", "ragged"])
@pytest.mark.parametrize("T,R,K,E", CASES)
def test_i8_expert_linear(T, R, K, E, kind):
    N, M = ((2, 4), (3, 4), (1, 4))[T % 3] if K % 8 else ((2, 4), (4, 8), (2, 8), (5, 8), (4, 4))[(T + R) % 5]
    x, sw, w = i8_weight(R, K, N, M, T, E=E)
    X = strided(randn(T, K, seed=R, dt=torch.float16), 3 if T % 4 == 1 else 0)
    bias = randn(E, R, seed=9) if T % 2 else None
    act = "gelu" if R % 2 else "none"
    o = counts(T, E, kind, seed=K)
    Y = nm.i8_expert_linear(x, sw, X, o, bias=bias, act=act, out_dtype=torch.float32)
    q, sx = i8_64(X)
    want, bound = i8_expert64(q, sx, w, sw, bias, act, o)
    check(Y, want, bound, "i8_expert_linear")
    out = torch.full((T, R), 2.0, device=DEV, dtype=torch.float32)
    o2 = o.clone()
    o2[-1] = o2[-2]                                      # the last expert's rows are no expert's now
    nm.i8_expert_linear(x, sw, nm.i8_quantize(X), o2, bias=bias, act=act, out=out)
    (spans, rest) = experts_of(o2, T)
    assert (out[rest] == 2).all()
    taken = [r for r in range(T) if r not in set(rest)]
    assert torch.equal(out[taken], Y[taken])
