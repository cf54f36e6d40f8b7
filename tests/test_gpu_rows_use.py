"""8-bit rows and products of rows grouped by expert as a program uses them: a
routed block's operators one after another, a training step's, captured graphs
whose offsets change, streams, workspaces that calls share, long buffers, rows
that are not finite."""
import copy
import pickle

import pytest
import torch

import semi_structured_sparse_nm_amd as nm
from tests._ffn import check, half_step
from tests._rows import expert64, expert_grad64, experts_of, i8_64, i8_expert64, i8_product64, pruned
from tests.test_gpu_rows import DEV, PATHS, counts, forced, i8_weight, randn

pytestmark = pytest.mark.gpu


def routed(T, E, top, seed):
    """(token of each row, offsets): `top` experts of E for each of T tokens, rows
    sorted by expert."""
    pick = torch.rand(T, E, generator=torch.Generator().manual_seed(seed)).topk(top, dim=1).indices.to(DEV)
    flat = pick.reshape(-1)
    order = flat.argsort(stable=True)
    at = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    at[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return order // top, at


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("T", [1, 37, 300])
def test_routed_block(T):
    """Tokens quantised once, for the weight that all of them share and for the
    experts': every operator within its bound of the 64-bit form on what the one
    before it returned."""
    K, R, E, top = 384, 200, 12, 3
    shared, ss, ws = i8_weight(R, K, 2, 4, 1)
    first, s1, w1 = i8_weight(R, K, 4, 8, 2, E=E)
    second, s2, w2 = i8_weight(K, R, 2, 4, 3, E=E)
    X = randn(T, K, seed=T, dt=torch.bfloat16)
    rows, o = routed(T, E, top, T)
    Q = nm.i8_quantize(X)
    q, sx = i8_64(X)
    check(nm.i8_linear(shared, ss, Q), *i8_product64(q, sx, ws, ss, None, "none"), "shared")
    G = nm.I8(T * top, K, Q.codes[rows], Q.scales[rows])
    H = nm.i8_expert_linear(first, s1, G, o, act="gelu")
    check(H, *i8_expert64(q[rows], sx[rows], w1, s1, None, "gelu", o), "first")
    Y = nm.i8_expert_linear(second, s2, H, o, out_dtype=torch.float32)
    qh, sh = i8_64(H)
    check(Y, *i8_expert64(qh, sh, w2, s2, None, "none", o), "second")


@pytest.mark.parametrize("T", [3, 140])
def test_training_step(T):
    """Two expert layers with a ReLU between them, forward and back."""
    K, R, E = 136, 96, 5
    W1 = randn(E, R, K, seed=1, dt=torch.bfloat16, scale=0.1)
    W2 = randn(E, K, R, seed=2, dt=torch.bfloat16, scale=0.1)
    w1, k1 = pruned(W1, 2, 4)
    w2, k2 = pruned(W2, 4, 8)
    x1, x2 = nm.pack_experts(W1, 2, 4), nm.pack_experts(W2, 4, 8)
    rows, o = routed(T, E, 2, T)
    X = randn(T, K, seed=T, dt=torch.bfloat16)[rows]
    H = nm.expert_linear(x1, X, o)
    check(H, *expert64(X, w1, o), "H")
    A = H.relu()
    check(nm.expert_linear(x2, A, o), *expert64(A, w2, o), "Y")
    dY = randn(2 * T, K, seed=9, dt=torch.bfloat16)
    dA, dW2 = nm.expert_linear_backward(x2, A, o, dY)
    want, b = expert_grad64(A, w2, k2, dY, o)
    check(dA, want[0], b[0], "dA")
    check(dW2, want[1], b[1], "dW2")
    dH = dA * (H > 0)
    dX, dW1 = nm.expert_linear_backward(x1, X, o, dH)
    want, b = expert_grad64(X, w1, k1, dH, o)
    check(dX, want[0], b[0], "dX")
    check(dW1, want[1], b[1], "dW1")


@pytest.mark.parametrize("N,M", [(2, 4), (3, 8)])
def test_gradients_against_differences(N, M):
    """The product is linear in X and in the kept weights, so a difference of two
    outputs is the gradient's whatever the step.  Whole numbers up to 8: inputs and
    steps are exact in fp16; sums of 64 products up to 64 in binary32 are too, so an
    output is off by its rounding only, and so are the gradients."""
    T, R, K, E = 90, 48, 64, 4
    g = torch.Generator().manual_seed(N)

    def whole(*shape):
        return torch.randint(-4, 5, shape, generator=g).to(DEV, torch.float16)

    W, X, dX, dY = whole(E, R, K), whole(T, K), whole(T, K), whole(T, R)
    W = W + W.sign()                                      # (the step below keeps every kept weight the larger one)
    o = counts(T, E, "ragged", seed=1)
    w, keep = pruned(W, N, M)
    x = nm.pack_experts(W, N, M)
    gX, gW = nm.expert_linear_backward(x, X, o, dY)

    def along(a, b):
        """(sum a b, what the rounding of a moves it by)"""
        p = a.double() * b.double()
        return float(p.sum()), float(half_step(a.dtype) * p.abs().sum())

    up, down = (nm.expert_linear(x, X + s * dX, o) for s in (1, -1))
    (a, ea), (b, eb), (c, ec) = along(up, dY), along(down, dY), along(gX, dX)
    assert abs((a - b) / 2 - c) <= (ea + eb) / 2 + ec
    dW = whole(E, R, K) * keep
    wu, wd = (nm.pack_experts(torch.where(keep, 16 * W + s * dW, torch.zeros_like(W)), N, M) for s in (1, -1))
    up, down = (nm.expert_linear(v, X, o) for v in (wu, wd))
    (a, ea), (b, eb), (c, ec) = along(up, dY), along(down, dY), along(gW, dW)
    assert abs((a - b) / 2 - c) <= (ea + eb) / 2 + ec


# ---------------------------------------------------------------- graphs and streams
def replayed(run, inputs, changes):
    """run() captured once; for each of `changes` (new values for `inputs`) a replay
    gives what an eager call gives."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for change in changes:
        for t, v in zip(inputs, change):
            t.copy_(v)
        for g in got:
            g.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for g, e in zip(got, run()):
            assert torch.equal(g, e)


@pytest.mark.parametrize("T", [20, 800])
def test_graphs_with_other_offsets(T):
    R, K, E = 136, 264, 6
    W = randn(E, R, K, seed=1, dt=torch.float16, scale=0.1)
    w, keep = pruned(W, 4, 8)
    x = nm.pack_experts(W, 4, 8)
    x8, s8, w8 = i8_weight(R, K, 2, 4, 2, E=E)
    X, dY = randn(T, K, dt=torch.float16), randn(T, R, seed=1, dt=torch.float16)
    o = counts(T, E, "even")
    changes = [(randn(T, K, seed=i, dt=torch.float16), randn(T, R, seed=9 + i, dt=torch.float16), at)
               for i, at in enumerate([counts(T, E, "ragged", 3), counts(T, E, "one"), counts(T, E, "ragged", 4) // 2,
                                       torch.zeros_like(o), counts(T, E, "even")])]

    def run():
        return (nm.expert_linear(x, X, o), *nm.expert_linear_backward(x, X, o, dY), nm.i8_expert_linear(x8, s8, X, o))

    replayed(run, (X, dY, o), changes)
    want, bound = expert64(X, w, o)
    check(run()[0], want, bound, "after the replays")


def test_graphs_share_a_workspace():
    """Two captured steps with one workspace, replayed in turn."""
    T, R, K, E = 500, 130, 200, 4
    W = randn(E, R, K, seed=1, dt=torch.bfloat16, scale=0.1)
    w, keep = pruned(W, 3, 8)
    x = nm.pack_experts(W, 3, 8)
    x8, s8, w8 = i8_weight(R, K, 5, 8, 2, E=E)
    X, dY, o = randn(T, K, dt=torch.bfloat16), randn(T, R, seed=1, dt=torch.bfloat16), counts(T, E, "ragged", 1)
    ws = torch.empty(max(nm.expert_linear_backward_workspace_size(x, T), nm.expert_linear_workspace_size(x, T),
                         nm.i8_expert_linear_workspace_size(x8, T)), dtype=torch.uint8, device=DEV)
    with forced("tile:1"):                                # (whose dense copies lie in the workspace)
        def one():
            return nm.expert_linear(x, X, o, workspace=ws), *nm.expert_linear_backward(x, X, o, dY, workspace=ws)

        def two():
            return (nm.i8_expert_linear(x8, s8, X, o, workspace=ws),)

        need = nm.expert_linear_workspace_size(x, T)
        assert 0 < need <= ws.numel() and nm.i8_expert_linear_workspace_size(x8, T) <= ws.numel()
        eager = [[t.clone() for t in f()] for f in (one, two)]
        graphs, got = [], []
        for f in (one, two):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                got.append(f())
            graphs.append(g)
        for i in (0, 1, 0, 1, 1, 0):
            for t in got[i]:
                t.fill_(float("nan"))
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got[i], eager[i]))
    check(eager[0][0], *expert64(X, w, o), "expert_linear")


def test_other_stream():
    """Calls go to the current stream, behind what it holds."""
    T, R, K, E = 300, 96, 512, 4
    x8, s8, w8 = i8_weight(R, K, 4, 8, 1, E=E)
    X0, o = randn(T, K, dt=torch.float16), counts(T, E, "ragged", 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        X = torch.zeros_like(X0)
        torch.cuda._sleep(20_000_000)
        X.copy_(X0)
        Y = nm.i8_expert_linear(x8, s8, X, o)
        Q = nm.i8_quantize(X)
        Z = nm.i8_dequantize(Q)
    s.synchronize()
    q, sx = i8_64(X0)
    check(Y, *i8_expert64(q, sx, w8, s8, None, "none", o), "i8_expert_linear")
    assert torch.equal(Z, q.float() * sx[:, None])


@pytest.mark.parametrize("T", [20, 600])
def test_two_streams_at_once(T):
    """Calls on two streams, side by side on the same weights, rows and offsets."""
    R, K, E = 200, 328, 5
    W = randn(E, R, K, seed=1, dt=torch.bfloat16, scale=0.1)
    x = nm.pack_experts(W, 5, 8)
    x8, s8, w8 = i8_weight(R, K, 3, 4, 2, E=E)
    X, dY, o = randn(T, K, dt=torch.bfloat16), randn(T, R, seed=1, dt=torch.bfloat16), counts(T, E, "ragged", 2)

    def run():
        return (nm.expert_linear(x, X, o), *nm.expert_linear_backward(x, X, o, dY), nm.i8_expert_linear(x8, s8, X, o),
                nm.i8_dequantize(nm.i8_quantize(X)))

    want = run()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_backward_reserves_what_it_uses():
    """The binding's own workspace: no dense weights without dX, no padded rows for whole
    ones."""
    T, R, K, E = 64, 256, 512, 8
    x = nm.pack_experts(randn(E, R, K, seed=1, dt=torch.bfloat16, scale=0.1), 2, 4)
    X, dY, o = randn(T, K, dt=torch.bfloat16), randn(T, R, seed=1, dt=torch.bfloat16), counts(T, E, "even")
    dense, rows, mask = E * R * K * 2, T * (K + R) * 2, E * (R // 128) * (K // 64) * 1024
    for dx, dw, most in ((True, True, dense + mask), (True, False, dense), (False, True, mask)):
        nm.expert_linear_backward(x, X, o, dY, need_dx=dx, need_dw=dw)
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        out = nm.expert_linear_backward(x, X, o, dY, need_dx=dx, need_dw=dw)
        peak = torch.cuda.max_memory_allocated() - before
        assert peak == sum(g.numel() * 2 for g in out if g is not None) + most, (dx, dw)
        del out
    assert nm.expert_linear_backward_workspace_size(x, T) == dense + mask + rows


def test_backward_takes_any_truth_value():
    T, R, K, E = 30, 40, 64, 2
    x = nm.pack_experts(randn(E, R, K, seed=1, dt=torch.float16, scale=0.1), 2, 4)
    X, dY, o = randn(T, K, dt=torch.float16), randn(T, R, seed=1, dt=torch.float16), counts(T, E, "even")
    dX, dW = nm.expert_linear_backward(x, X, o, dY)
    for no in (None, 0, []):
        a, b = nm.expert_linear_backward(x, X, o, dY, need_dx=1, need_dw=no)
        assert torch.equal(a, dX) and b is None
        a, b = nm.expert_linear_backward(x, X, o, dY, need_dx=no, need_dw="yes")
        assert a is None and torch.equal(b, dW)


# ---------------------------------------------------------------- copies, rows, lengths
def test_copies_and_pickles():
    x8, s8, w8 = i8_weight(40, 136, 2, 4, 1, E=3)
    X, o = randn(9, 136, dt=torch.float16), counts(9, 3, "even")
    Q = nm.i8_quantize(X)
    want = nm.i8_expert_linear(x8, s8, Q, o)
    for again in (copy.copy, copy.deepcopy, lambda v: pickle.loads(pickle.dumps(v))):
        assert torch.equal(nm.i8_expert_linear(again(x8), s8, again(Q), o), want)
    Q.codes, Q.scales = Q.codes.clone(), Q.scales * 2     # fields replaced between calls
    assert torch.equal(nm.i8_expert_linear(x8, s8, Q, o, out_dtype=torch.float32),
                       2 * nm.i8_expert_linear(x8, s8, X, o, out_dtype=torch.float32))


@pytest.mark.parametrize("path,N,M", [p for p in PATHS if p[1:] in ((2, 4), (4, 4), (1, 8), (5, 8))])
def test_rows_not_finite(path, N, M):
    """An infinite or NaN element reaches the outputs of its row only; the row's
    last columns too, behind which kernels fill up with zeros."""
    T, R, K, E = 150, 70, 136, 3
    W = randn(E, R, K, seed=1, dt=torch.bfloat16, scale=0.1)
    w, _ = pruned(W, N, M)
    x = nm.pack_experts(W, N, M)
    X, o = randn(T, K, seed=2, dt=torch.bfloat16), counts(T, E, "even")
    bad = {5: (3, float("inf")), 49: (K - 1, float("nan")), 50: (128, float("-inf")), 149: (K - 8, float("inf"))}
    for r, (k, v) in bad.items():
        X[r, k] = v
    with forced(path):
        Y = nm.expert_linear(x, X, o)
    fine = [r for r in range(T) if r not in bad]
    Xf = X.clone()
    Xf[list(bad)] = 0
    want, bound = expert64(Xf, w, o)
    check(Y[fine], want[fine], bound[fine], path)
    assert Y[49, w[0, :, K - 1] != 0].isnan().all()
    for r, (k, v) in bad.items():
        e = next(e for e, (a, b) in enumerate(experts_of(o, T)[0]) if a <= r < b)
        assert not Y[r, w[e, :, k] != 0].isfinite().any()


@pytest.mark.parametrize("path,E", [("tile24:0", 700), ("tile24:1", 511), ("tile24:2", 512), ("tile24:3", 1023),
                                    ("wide:0", 1023), ("stream:1", 1023)])
def test_many_experts(path, E):
    R, K, T = 24, 64, 2000
    X = randn(T, K, seed=1, dt=torch.float16)
    x8, s8, w8 = i8_weight(R, K, 2, 4, 1, E=E)
    W = randn(E, R, K, seed=2, dt=torch.float16, scale=0.1)
    x, (w, _) = nm.pack_experts(W, 2, 4), pruned(W, 2, 4)
    q, sx = i8_64(X)
    for kind in ("ragged", "one"):
        o = counts(T, E, kind, seed=E)
        with forced(path):
            check(nm.i8_expert_linear(x8, s8, X, o), *i8_expert64(q, sx, w8, s8, None, "none", o), "8 bits")
            check(nm.expert_linear(x, X, o), *expert64(X, w, o), "16 bits")


@pytest.mark.parametrize("path", ["stream:1", "wide:0", "wide:1", "tile24:1", "tile24:3"])
def test_rows_past_32_bits(path):
    """Rows whose byte offsets pass 2^32, in X and in the output."""
    T, R, K, E, last = (1 << 20) + 37, 2056, 2056, 2, 300
    ld = 2056
    W = randn(E, R, K, seed=1, dt=torch.bfloat16, scale=0.1)
    x, (w, _) = nm.pack_experts(W, 2, 4), pruned(W, 2, 4)
    X = torch.empty(T, ld, dtype=torch.bfloat16, device=DEV)
    X[-last:] = randn(last, K, seed=2, dt=torch.bfloat16)
    out = torch.empty(T, R, dtype=torch.bfloat16, device=DEV)
    out[-last - 50:] = 5
    assert (T - last) * ld * 2 > 1 << 32
    o = torch.tensor([T - last, T - 200, T - 10], device=DEV)
    with forced(path):
        nm.expert_linear(x, X, o, out=out)
    Y, B = expert64(X[-last:], w, o - (T - last))
    check(out[-last:-10], Y[:-10], B[:-10], path)
    assert (out[-10:] == 5).all() and (out[-last - 50:-last] == 5).all()


@pytest.mark.parametrize("path", ["stream:1", "wide:1", "tile:1"])
def test_codes_past_32_bits(path):
    T, R, K, last = (1 << 20) + 37, 40, 4200, 100
    p, sw, w = i8_weight(R, K, 4, 8, 1, E=1)
    Q = nm.I8(T, K, torch.empty(T, 4224, dtype=torch.int8, device=DEV), torch.ones(T, device=DEV))
    X = randn(last, K, seed=2, dt=torch.bfloat16)
    q, sx = i8_64(X)
    Q.codes[-last:, :K] = q.to(torch.int8)
    Q.codes[-last:, K:] = 0
    Q.scales[-last:] = sx
    o = torch.tensor([T - last, T], dtype=torch.int32, device=DEV)
    out = torch.empty(T, R, device=DEV)
    with forced(path):
        nm.i8_expert_linear(p, sw, Q, o, out=out)
    check(out[-last:], *i8_product64(q, sx, w[0], sw[0], None, "none"), path)


@pytest.mark.parametrize("path", ["stream:1", "wide:1", "tile24:1"])
def test_weights_past_32_bits(path):
    """The last of many large experts: its packed weight, gradient and transposed
    copy lie past 2^32 bytes."""
    E, R, K, T = 80, 7168, 8192, 150
    W = torch.zeros(E, R, K, dtype=torch.bfloat16, device=DEV)
    W[-1] = randn(R, K, seed=1, dt=torch.bfloat16, scale=0.1)
    w, keep = pruned(W[-1:], 2, 4)
    x = nm.pack_experts(W, 2, 4)
    assert x.values.numel() * (E - 1) // E > 1 << 32
    del W
    X = randn(T, K, seed=2, dt=torch.bfloat16)
    o = torch.tensor([0] * E + [T], device=DEV)
    one = torch.tensor([0, T])
    with forced(path):
        check(nm.expert_linear(x, X, o), *expert64(X, w, one), path)
    if path == "tile24:1":
        dY = randn(T, R, seed=3, dt=torch.bfloat16)
        dX, dW = nm.expert_linear_backward(x, X, o, dY)
        want, b = expert_grad64(X, w, keep, dY, one)
        check(dX, want[0], b[0], "dX")
        check(dW[-1:], want[1], b[1], "dW")
        assert not dW[:-1].any()


@pytest.mark.parametrize("T,R,K,N,M", [(2048, 11000, 640, 2, 4), (2000, 9001, 512, 1, 8), (1500, 14000, 384, 4, 4),
                                       (3000, 7300, 768, 6, 8)])
def test_long_prompts_in_two_shapes(T, R, K, N, M):
    """More tiles than compute units: whole rounds of large ones, the last outputs in
    smaller ones, each with its own scales and bias."""
    p, sw, w = i8_weight(R, K, N, M, R)
    X, bias = randn(T, K, seed=T, dt=torch.bfloat16), randn(R, seed=2)
    wide = torch.full((T, R + 24), 3.0, dtype=torch.bfloat16, device=DEV)
    nm.i8_linear(p, sw, X, bias=bias, act="gelu", out=wide[:, 8:8 + R])
    q, sx = i8_64(X)
    check(wide[:, 8:8 + R], *i8_product64(q, sx, w, sw, bias, "gelu"), "i8_linear")
    assert (wide[:, :8] == 3).all() and (wide[:, 8 + R:] == 3).all()
    W = randn(1, R, K, seed=1, dt=torch.float16, scale=0.1)
    x, (we, _) = nm.pack_experts(W, N, M), pruned(W, N, M)
    X = X.half()
    o = torch.tensor([5, T - 7], dtype=torch.int32, device=DEV)
    check(nm.expert_linear(x, X, o), *expert64(X, we, o), "expert_linear")
