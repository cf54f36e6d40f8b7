"""Cases, inputs and plain forms of the feed-forward operators.

Five operators of a language model's feed-forward block:

  glu          H = act(X Wg^T) * (X Wu^T), both weights N:M packed (the gated
               block of a pruned model; both projections, the activation and
               the product in one call)
  glu_train    the same with the two products kept, then its backward pass:
               dX and the gradients of the kept weights
  mx_quantize  16-bit values -> microscaled 4-bit floating point (blocks of 32
               E2M1 elements, one E8M0 scale each) and back
  mx_linear    Y = act(X W^T + b), weight and activations in that format
  mx_glu       the gated block with both weights in that format

X is [T, K], weights are [R, K], outputs [T, R], the reduction contiguous.
`run` computes them in their plain form with elementary torch operations in
32 bits, or, where `own` is set, by the package's calls.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, T, R, K, dtype, N=2, M=4, act="silu", pad=0, bias=False):
    c = {"op": op, "T": T, "R": R, "K": K, "dtype": dtype, "N": N, "M": M, "act": act, "pad": pad, "bias": bias}
    if name is not None:
        c = {"name": name, **c}
    return c


def listed():
    return [
        # one token of decoding through a pruned 7B-sized gated block: launch
        # and weight streaming
        _case("glu_decode_1", "glu", 1, 11008, 4096, "bf16"),
        # sixteen requests decoding together, the looser 4:8 pattern
        _case("glu_decode_16_4of8", "glu", 16, 11008, 4096, "fp16", N=4, M=8),
        # a short prompt through a small block whose sizes fit no tile, the
        # activations a slice of a wider buffer
        _case("glu_ragged", "glu", 77, 1500, 1000, "fp16", act="gelu", pad=24),
        # a prompt of 2048 tokens: bound by the matrix cores
        _case("glu_prompt_2048", "glu", 2048, 11008, 4096, "fp16"),
        # one small training step on an image's 197 tokens, 4:8
        _case("glu_train_197", "glu_train", 197, 1000, 768, "fp16", N=4, M=8, act="gelu"),
        # one training step of the 7B-sized block on 2048 tokens
        _case("glu_train_2048", "glu_train", 2048, 11008, 4096, "bf16"),
        # activations of one image, a width that ends inside a block
        _case("mx_quantize_197", "mx_quantize", 197, 0, 770, "bf16"),
        # a whole 7B-sized projection converted at load time
        _case("mx_quantize_weight", "mx_quantize", 11008, 0, 4096, "bf16"),
        # the down projection for one token
        _case("mx_linear_decode_1", "mx_linear", 1, 4096, 11008, "bf16", act="none"),
        # the down projection for a prompt of 2048 tokens, with bias
        _case("mx_linear_prompt_2048", "mx_linear", 2048, 4096, 11008, "bf16", act="none", bias=True),
        # sixteen requests decoding through the 4-bit gated block
        _case("mx_glu_decode_16", "mx_glu", 16, 11008, 4096, "bf16"),
        # a prompt through the 4-bit gated block, a ragged number of tokens
        _case("mx_glu_prompt_1900", "mx_glu", 1900, 11008, 4096, "fp16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: the tokens and both widths over their whole ranges."""
    op = rng.choice(["glu", "glu", "glu_train", "mx_quantize", "mx_linear", "mx_glu"])
    T = _log_int(rng, 1, 2048)
    R = _log_int(rng, 64, 11008)
    N, M = rng.choice([(2, 4), (2, 4), (4, 8), (1, 4), (2, 8), (4, 4), (3, 4)])
    K = _log_int(rng, 64, 4096)
    if op in ("glu", "glu_train"):
        K = max(M, K // M * M)
    act = rng.choice(["silu", "gelu"])
    if op == "mx_linear":
        act = rng.choice(["none", "gelu"])
    if op == "mx_quantize":
        T, R = _log_int(rng, 1, 11008), 0
    return _case(None, op, T, R, K, rng.choice(["fp16", "bf16"]), N=N, M=M, act=act,
                 pad=rng.choice([0, 0, 8, 5]), bias=op == "mx_linear" and rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _inputs(case, seed):
    """Activations ~ N(0, 1) with a few channels ten times as large, weights
    ~ N(0, 0.02), gradients ~ N(0, 0.1), from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, R, K = case["T"], case["R"], case["K"]
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    loud = 1.0 + 9.0 * (torch.rand(K, generator=gen, device="cuda") < 0.01)
    wide = torch.zeros(T, K + case["pad"], device="cuda", dtype=dt)
    X = wide[:, :K]
    X.copy_(normal(T, K) * loud)
    d = {"X": X}
    if case["op"] != "mx_quantize":
        d["W"] = [(normal(R, K) * 0.02).to(dt) for _ in range(1 if case["op"] == "mx_linear" else 2)]
    if case["op"] == "glu_train":
        d["dH"] = (normal(T, R) * 0.1).to(dt)
    if case["bias"]:
        d["bias"] = normal(R)
    return d


def _keep(W, N, M):
    """Truth values of the N largest magnitudes of every M along a row, equal
    ones going to the lower position."""
    a = W.float().abs().reshape(W.shape[0], -1, M)
    keep = torch.empty(a.shape, dtype=torch.bool, device=W.device)
    for i in range(M):
        rank = torch.zeros(a.shape[:2], dtype=torch.int32, device=W.device)
        for j in range(M):
            if j != i:
                rank += (a[..., j] > a[..., i]) if j > i else (a[..., j] >= a[..., i])
        keep[..., i] = rank < N
    return keep.reshape(W.shape)


def prepare(case, seed):
    """The call's operands as a program holds them: the activations, and the
    weights pruned (or quantised) once when the model was loaded."""
    d = _inputs(case, seed)
    state = {"case": case, "X": d["X"], "dH": d.get("dH"), "bias": d.get("bias")}
    op = case["op"]
    if op == "mx_quantize":
        return state
    if own:
        import semi_structured_sparse_nm_amd as nm
        if op in ("glu", "glu_train"):
            state["W"] = [nm.pack(W, case["N"], case["M"]) for W in d["W"]]
        else:
            state["W"] = [nm.mx_quantize(W) for W in d["W"]]
    elif op in ("glu", "glu_train"):
        state["keep"] = [_keep(W, case["N"], case["M"]) for W in d["W"]]
        state["W"] = [torch.where(k, W, torch.zeros_like(W)) for k, W in zip(state["keep"], d["W"])]
    else:
        state["W"] = [_mx_round(W).to(W.dtype) for W in d["W"]]
    return state


# ---------------------------------------------------------------- plain forms
def _gate(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))


def _gate_slope(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def _mx_round(x):
    """x rounded to E2M1 elements with one power-of-two scale for each block
    of 32 along the rows, in 32 bits: scale 2^(floor(log2 amax) - 2), round
    half to even, magnitudes above 6 become 6."""
    rows, K = x.shape
    nb = (K + 31) // 32
    v = torch.zeros(rows, nb * 32, dtype=torch.float32, device=x.device)
    v[:, :K] = x
    v = v.reshape(rows, nb, 32)
    e = (torch.frexp(v.abs().amax(dim=2, keepdim=True)).exponent - 3).clamp(-127, 127)
    u = torch.ldexp(v, -e)
    a = u.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.ldexp(torch.copysign(q, u), e).reshape(rows, nb * 32)[:, :K]


def _plain(state):
    case, X = state["case"], state["X"]
    op, act, dt = case["op"], case["act"], X.dtype
    if op == "mx_quantize":
        return _mx_round(X).to(dt)
    if op == "mx_linear":
        y = _mx_round(X) @ state["W"][0].float().t()
        if state["bias"] is not None:
            y = y + state["bias"]
        return (_gate(y, "gelu") if act == "gelu" else y).to(dt)
    x = _mx_round(X) if op == "mx_glu" else X.float()
    Wg, Wu = (W.float() for W in state["W"])
    g, u = x @ Wg.t(), x @ Wu.t()
    a = _gate(g, act)
    h = (a * u).to(dt)
    if op != "glu_train":
        return h
    dh = state["dH"].float()
    dg, du = dh * u * _gate_slope(g, act), dh * a
    dx = (dg @ Wg + du @ Wu).to(dt)
    kg, ku = state["keep"]
    dwg = torch.where(kg, dg.t() @ x, 0.0).to(dt)
    dwu = torch.where(ku, du.t() @ x, 0.0).to(dt)
    return h, dx, dwg, dwu


def _own(state):
    import semi_structured_sparse_nm_amd as nm
    case, X, W = state["case"], state["X"], state.get("W")
    op, act = case["op"], case["act"]
    if op == "glu":
        return nm.glu(W[0], W[1], X, act=act)
    if op == "glu_train":
        # the kept products in 32 bits, as the plain form has them
        pre = torch.empty(2, X.shape[0], W[0].rows, dtype=torch.float32, device=X.device)
        h = nm.glu(W[0], W[1], X, act=act, pre=pre)
        return (h, *nm.glu_backward(W[0], W[1], X, pre, state["dH"], act=act))
    if op == "mx_quantize":
        return nm.mx_dequantize(nm.mx_quantize(X), out_dtype=X.dtype)
    if op == "mx_linear":
        return nm.mx_linear(W[0], X, bias=state["bias"], act=act)
    return nm.mx_glu(W[0], W[1], X, act=act)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: inputs and outputs once, the weights
    in their packed form, products with kept weights only."""
    op, T, R, K = case["op"], case["T"], case["R"], case["K"]
    N, M = case["N"], case["M"]
    packed = R * K * N / M * (2 + (0 if N == M else (2 if M == 4 else 3) / 8))
    mx = 17 / 32                                      # bytes of an element with its share of the scale
    if op == "glu":
        return {"bytes": 2 * T * K + 2 * packed + 2 * T * R, "flops": 4 * T * R * K * N / M}
    if op == "glu_train":
        # forward and both directions of the backward pass; X, dH and the
        # weights in, H, dX and the two weight gradients out
        return {"bytes": 4 * T * K + 2 * packed + 4 * T * R + 4 * R * K, "flops": 12 * T * R * K * N / M}
    if op == "mx_quantize":
        return {"bytes": 4 * T * K, "flops": 0}
    n = 1 if op == "mx_linear" else 2
    return {"bytes": 2 * T * K + n * R * K * mx + 2 * T * R + (4 * R if case["bias"] else 0),
            "flops": 2 * n * T * R * K}


# ---------------------------------------------------------------- 64 bits
def _exact_mx(x):
    """The same rounding from the format's definition: the nearest of the
    eight magnitudes, the one with the even code where two are equally near."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for r in range(0, x.shape[0], 2048):
        for k in range(0, x.shape[1], 2048):          # whole blocks of 32
            v = x[r:r + 2048, k:k + 2048].double()
            short = -v.shape[1] % 32
            b = torch.nn.functional.pad(v, (0, short)).unflatten(1, (-1, 32))
            top = b.abs().amax(dim=2, keepdim=True)
            p = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
            # log2 rounded across a power of two
            p = p - (torch.exp2(p) > top).double() + (torch.exp2(p + 1) <= top).double()
            s = torch.exp2(torch.where(top > 0, p - 2, 0.0).clamp(-127, 127))
            m = (b.abs() / s).contiguous()
            down = torch.bucketize(m, mid)            # on a midpoint: the lower code
            up = torch.bucketize(m, mid, right=True)  # on a midpoint: the upper code
            code = torch.where(down % 2 == 0, down, up)
            q = (torch.sign(b) * grid[code] * s).flatten(1)
            out[r:r + 2048, k:k + 2048] = q[:, :v.shape[1]]
    return out


def _exact_keep(W, N, M):
    order = W.double().abs().unflatten(1, (-1, M)).sort(dim=2, descending=True, stable=True).indices
    keep = torch.zeros(order.shape, dtype=torch.bool, device=W.device)
    keep.scatter_(2, order[..., :N], True)
    return keep.flatten(1)


def exact(case, seed):
    d = _inputs(case, seed)
    op, act = case["op"], case["act"]
    if op == "mx_quantize":
        return _exact_mx(d["X"])
    if op.startswith("mx"):
        x, W = _exact_mx(d["X"]), [_exact_mx(w) for w in d["W"]]
    else:
        keep = [_exact_keep(w, case["N"], case["M"]) for w in d["W"]]
        x, W = d["X"].double(), [w.double() * k for w, k in zip(d["W"], keep)]
    g = x @ W[0].t()
    if op == "mx_linear":
        if "bias" in d:
            g = g + d["bias"].double()
        return g * 0.5 * torch.erfc(-g / math.sqrt(2.0)) if act == "gelu" else g
    u = x @ W[1].t()
    if act == "silu":
        cdf = torch.sigmoid(g)
        slope = cdf + g * cdf * torch.sigmoid(-g)
    else:
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        slope = cdf + g * torch.exp(-g * g / 2) / math.sqrt(2.0 * math.pi)
    h = g * cdf * u
    if op != "glu_train":
        return h
    dh = d["dH"].double()
    dg, du = dh * u * slope, dh * g * cdf
    return h, dg @ W[0] + du @ W[1], (dg.t() @ x) * keep[0], (du.t() @ x) * keep[1]
